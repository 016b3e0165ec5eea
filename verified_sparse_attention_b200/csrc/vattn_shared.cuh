// Kernels of the shared-prefix decode (vattn_shared_dense_decode), in launch
// order:
//
//   k_shared_prep     validates lengths, groups and pages; the work of the
//                     prefix kernel and of the gather as prefix sums
//   k_shared_prefix(_tc)  every group's prefix against all of its queries
//   k_gather(_tc)<kModeSuffix>  every sequence's own positions
//   k_shared_combine  merges the records of both parts
//
// A group's G * (its sequences) query rows of one KV head meet the same keys,
// so the prefix is a matrix product with the rows of a block of RB on one side
// and tiles of KT keys on the other. Work is flattened as [group][row block]
// [KV head][key tile] and cut evenly over a persistent grid; each (CTA, block,
// head) segment leaves one record (maximum, weight sum, weighted values) per
// row. Only groups of which two sequences at least reach the end of the prefix
// are shared: the others, and sequences shorter than their prefix, are left to
// the gather whole, so that no row of a segment is masked and every key of a
// tile counts for every row.
#pragma once

#include "vattn_ctx.h"
#include "vattn_kernels.cuh"

namespace vattn {

constexpr unsigned kDevBadSeqlen = VATTN_DEV_BAD_SEQLEN, kDevBadPage = VATTN_DEV_BAD_PAGE,
                   kDevBadGroup = VATTN_DEV_BAD_GROUP;

struct SharedParams {
  // tensor-core prefix kernel: the caches in boxes of `box` rows by 64 columns,
  // the queries [batch][Hq][d] in boxes of 128 rows (128 / G sequences, the G
  // heads of a KV head) by 64 columns, 128-byte swizzle
  CUtensorMap tmk_t, tmv_t, tmq;
  DevParams D;
  SharedWork W;
  const int* group_start;
  const int* prefix_lens;
  int groups;
  int RB, KT;  // rows of a block, keys of a tile
  int box;     // rows of a cache box: a power of two that divides the page size, at most KT
};

// ---------------------------------------------------------------- groups
// Record rows of a whole group's query rows are its query rows per KV head;
// a block's records of KV head h start behind those of the blocks and heads
// before it.
__device__ __forceinline__ long long block_row0(const SharedParams& P, int mb, int h, int rows) {
  return static_cast<long long>(mb) * P.RB * P.D.Hkv + static_cast<long long>(h) * rows;
}

// ============================================================ k_shared_prep
constexpr int kSharedPrepThreads = 256;

__device__ __forceinline__ int checked_len(const SharedParams& P, int b) {
  const int n = P.D.seq_lens[b];
  return n < 0 || n > P.D.max_ctx ? -1 : n;
}

// Whether any of the page ids of row `b` in slots [s0, s1) is out of range.
__device__ __forceinline__ int bad_pages(const SharedParams& P, int b, int s0, int s1) {
  int bad = 0;
  for (int i0 = s0 + threadIdx.x; i0 < s1; i0 += 8 * blockDim.x) {  // eight independent loads in flight
    int pid[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int i = i0 + j * blockDim.x;
      pid[j] = i < s1 ? P.D.page_table[static_cast<size_t>(b) * P.D.pps + i] : 0;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (pid[j] < 0 || pid[j] >= P.D.num_pages) bad = 1;
  }
  return __syncthreads_or(bad);
}

// Sequences of [b0, b1) that reach position `prefix` (the whole block).
__device__ __forceinline__ int count_reach(const SharedParams& P, int b0, int b1, int prefix) {
  int cnt = 0;
  for (int base = b0; base < b1; base += blockDim.x) {
    const int b = base + threadIdx.x;
    cnt += __syncthreads_count(b < b1 && prefix > 0 && checked_len(P, b) >= prefix);
  }
  return cnt;
}

// CTA b < batch: sequence b; CTA batch + g: group g (its pages and count); the
// last CTA: the prefix sums.
static __global__ void __launch_bounds__(kSharedPrepThreads) k_shared_prep(const __grid_constant__ SharedParams P) {
  __shared__ unsigned s_warp[32];
  __shared__ int s_g, s_bad;
  const int tid = threadIdx.x, cta = blockIdx.x;
  const DevParams& D = P.D;
  if (tid == 0) {
    s_g = -1;
    s_bad = 0;
  }
  grid_dependency_wait();
  __syncthreads();
  // the bounds ascend from 0 to batch, or nothing is decoded; with ascending
  // bounds at most one group holds a sequence
  for (int g = tid; g < P.groups; g += blockDim.x) {
    const int lo = P.group_start[g], hi = P.group_start[g + 1];
    if (hi < lo || (g == 0 && lo != 0) || (g == P.groups - 1 && hi != D.batch)) s_bad = 1;
    if (cta < D.batch && lo <= cta && cta < hi) s_g = g;
  }
  __syncthreads();
  const bool bad_bounds = s_bad != 0;

  if (cta < D.batch) {
    const int b = cta, g = s_g;
    int n = checked_len(P, b), start = 0;
    if (tid == 0 && n < 0) atomicOr(D.err, kDevBadSeqlen);
    if (n < 0 || bad_bounds || g < 0) n = 0;
    if (n > 0) {
      const int prefix = P.prefix_lens[g];
      if (prefix < 0 || prefix > D.max_ctx) {
        n = 0;
      } else if (n >= prefix && prefix > 0) {
        if (count_reach(P, P.group_start[g], P.group_start[g + 1], prefix) >= 2) start = prefix;
      }
    }
    if (bad_pages(P, b, start / D.ps, (n + D.ps - 1) / D.ps)) {
      // only the positions behind the prefix are read through this row
      if (n > start) {
        if (tid == 0) atomicOr(D.err, kDevBadPage);
        n = 0;
      }
    }
    for (int h = tid; h < D.Hkv; h += blockDim.x) {
      UnitInfo inf = {};
      inf.n = n;
      inf.s1 = start;
      inf.k = g;
      D.info[static_cast<size_t>(b) * D.Hkv + h] = inf;
    }
    return;
  }
  if (cta < D.batch + P.groups) {
    const int g = cta - D.batch;
    int reach = 0, ok = 0;
    if (!bad_bounds) {
      const int prefix = P.prefix_lens[g], b0 = P.group_start[g], b1 = P.group_start[g + 1];
      if (prefix < 0 || prefix > D.max_ctx) {
        if (tid == 0) atomicOr(D.err, kDevBadGroup);
      } else {
        reach = count_reach(P, b0, b1, prefix);
        ok = 1;
        if (reach >= 2 && bad_pages(P, b0, 0, (prefix + D.ps - 1) / D.ps)) {
          if (tid == 0) atomicOr(D.err, kDevBadPage);
          ok = 0;
        }
      }
    }
    if (tid == 0) P.W.pages_ok[g] = ok;
    return;
  }
  // prefix sums: key tiles and record rows over groups, the gather's slices
  if (bad_bounds && tid == 0) atomicOr(D.err, kDevBadGroup);
  for (int g = tid; g < P.groups; g += blockDim.x) P.W.reach[g] = 0;
  __syncthreads();
  if (!bad_bounds) {
    for (int b = tid; b < D.batch; b += blockDim.x) {
      int lo = 0, hi = P.groups;  // the last g with group_start[g] <= b
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (P.group_start[mid] <= b) lo = mid;
        else hi = mid;
      }
      const int prefix = P.prefix_lens[lo];
      if (prefix > 0 && prefix <= D.max_ctx && checked_len(P, b) >= prefix) atomicAdd(&P.W.reach[lo], 1);
    }
  }
  __threadfence_block();
  __syncthreads();
  __shared__ long long s_sum[2];
  long long tiles = 0, rows = 0;
  for (int base = 0; base < P.groups; base += blockDim.x) {
    const int g = base + tid;
    long long t = 0, r = 0;
    SharedGroup rec = {};
    if (g < P.groups && !bad_bounds) {
      const int reach = *static_cast<volatile int*>(&P.W.reach[g]);
      rec.b0 = P.group_start[g];
      rec.size = P.group_start[g + 1] - rec.b0;
      rec.prefix = P.prefix_lens[g];
      if (reach >= 2) {
        const int nrow = rec.size * D.G;
        rec.tiles = (rec.prefix + P.KT - 1) / P.KT;
        t = static_cast<long long>(rec.tiles) * ((nrow + P.RB - 1) / P.RB) * D.Hkv;
        r = static_cast<long long>(nrow) * D.Hkv;
      }
    }
    // both sums of 256 groups: tiles < 2^24 / KT * batch rows..., kept in 64 bits by a serial scan of warp 0
    __shared__ long long s_t[kSharedPrepThreads], s_r[kSharedPrepThreads];
    s_t[tid] = t;
    s_r[tid] = r;
    __syncthreads();
    for (int o = 1; o < kSharedPrepThreads; o <<= 1) {
      const long long a = tid >= o ? s_t[tid - o] : 0, c = tid >= o ? s_r[tid - o] : 0;
      __syncthreads();
      s_t[tid] += a;
      s_r[tid] += c;
      __syncthreads();
    }
    if (g < P.groups) {
      rec.tile0 = tiles + s_t[tid] - t;
      rec.row0 = rows + s_r[tid] - r;
      P.W.group[g] = rec;
    }
    tiles += s_t[kSharedPrepThreads - 1];
    rows += s_r[kSharedPrepThreads - 1];
    __syncthreads();
  }
  if (tid == 0) {
    SharedGroup rec = {};
    rec.tile0 = tiles;
    rec.row0 = rows;
    P.W.group[P.groups] = rec;
    s_sum[0] = 0;
  }
  __syncthreads();
  // slices of the gather: sequence b's own positions, once per KV head (a
  // sequence whose pages fail keeps its items here and is skipped there)
  for (int base = 0; base < D.batch; base += blockDim.x) {
    const int b = base + tid;
    unsigned cnt = 0;
    if (b < D.batch && !bad_bounds) {
      int lo = 0, hi = P.groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (P.group_start[mid] <= b) lo = mid;
        else hi = mid;
      }
      const int n = checked_len(P, b), prefix = P.prefix_lens[lo];
      const bool shared = prefix > 0 && prefix <= D.max_ctx && n >= prefix &&
                          *static_cast<volatile int*>(&P.W.reach[lo]) >= 2;
      if (n > 0 && prefix >= 0 && prefix <= D.max_ctx) cnt = static_cast<unsigned>(shared ? n - prefix : n);
    }
    const long long carry = s_sum[0];
    const unsigned incl = block_inclusive_scan(cnt, s_warp);  // 256 x 2^24 fits 32 bits unsigned
    if (b < D.batch) {
      const long long at = (carry + (incl - cnt)) * D.Hkv;
      for (int h = 0; h < D.Hkv; h++) {
        const size_t s = 2 * (static_cast<size_t>(b) * D.Hkv + h);
        D.pre_det[s] = at + static_cast<long long>(h) * cnt;
        D.pre_det[s + 1] = at + static_cast<long long>(h + 1) * cnt;
      }
    }
    __syncthreads();
    if (tid == blockDim.x - 1) s_sum[0] = carry + incl;
    __syncthreads();
  }
  if (tid == 0) D.pre_det[2 * static_cast<size_t>(D.units)] = s_sum[0] * D.Hkv;
}

// ---------------------------------------------------------------- segments
// One CTA's part of a (row block, KV head): key tiles [t0, t1).
struct Segment {
  int b0, prefix;       // the group's first sequence and prefix length
  int gi, mb, h, t0, t1;
  int row0, rows;       // the block's query rows within the group
  long long rec;        // its first record row
  long long next;       // flattened tile behind it
};
// The segment that starts at flattened tile x of a CTA with tiles up to `end`;
// gi: the group searched from. `group`: the records, in global or shared memory.
__device__ __forceinline__ Segment segment_at(const SharedParams& P, const SharedGroup* group, long long x,
                                              long long end, int gi) {
  while (group[gi + 1].tile0 <= x) gi++;
  const SharedGroup g = group[gi];
  Segment s;
  s.gi = gi;
  s.b0 = g.b0;
  s.prefix = g.prefix;
  const long long y = x - g.tile0;
  const int per = g.tiles * P.D.Hkv;
  s.mb = static_cast<int>(div_nonneg(y, per));
  const int z = static_cast<int>(y - static_cast<long long>(s.mb) * per);
  s.h = z / g.tiles;
  s.t0 = z - s.h * g.tiles;
  s.t1 = static_cast<int>(min(static_cast<long long>(g.tiles), s.t0 + (end - x)));
  s.next = x + (s.t1 - s.t0);
  s.row0 = s.mb * P.RB;
  s.rows = min(P.RB, g.size * P.D.G - s.row0);
  s.rec = static_cast<long long>(blockIdx.x) * P.RB + g.row0 + block_row0(P, s.mb, s.h, s.rows);
  return s;
}
// Group of flattened tile x (every warp by itself).
__device__ __forceinline__ int group_at(const SharedParams& P, const SharedGroup* group, long long x) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < P.groups; base += 32) {
    const int g = base + lane;
    const unsigned hit =
        __ballot_sync(0xffffffffu, g < P.groups && group[g].tile0 <= x && x < group[g + 1].tile0);
    if (hit) return base + __ffs(hit) - 1;
  }
  return 0;
}

// ============================================================ k_shared_prefix
// fp32 caches, and caches in host memory: fp32 FMAs. Blocks of 64 rows against
// tiles of 64 keys; 256 threads as 16 x 16, each with 4 x 4 scores and 4 rows
// of D / 16 outputs, all operands in shared memory as fp32.
template <int D>
struct PrefixShape {
  static constexpr int RB = 64, KT = 64;
  static constexpr int LD = D + 4;    // row pitch of Q and K: 16-byte rows that start in different banks
  static constexpr int LP = KT + 4;
  static constexpr size_t SMEM = static_cast<size_t>(RB * LD + KT * LD + KT * D + RB * LP) * 4;
};

template <typename T, int D>
__global__ void __launch_bounds__(256, 1) k_shared_prefix(const __grid_constant__ SharedParams P) {
  using S = PrefixShape<D>;
  constexpr int RB = S::RB, KT = S::KT, LD = S::LD, LP = S::LP, E = Elem<T>::kPer16, VPR = D / E;
  extern __shared__ __align__(16) float sm[];
  float* s_q = sm;
  float* s_k = s_q + RB * LD;
  float* s_v = s_k + KT * LD;
  float* s_p = s_v + KT * D;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  grid_dependency_wait();
  const long long Tt = P.W.group[P.groups].tile0;
  long long cur = div_nonneg(Tt * blockIdx.x, gridDim.x);
  const long long end = div_nonneg(Tt * (blockIdx.x + 1), gridDim.x);
  int gi = group_at(P, P.W.group, cur);
  const float c = P.D.scale * 1.4426950408889634f;  // scores in log2 units

  while (cur < end) {
    const Segment s = segment_at(P, P.W.group, cur, end, gi);
    gi = s.gi;
    cur = s.next;
    if (!P.W.pages_ok[s.gi]) continue;  // the combine does not read its records
    const T* q = static_cast<const T*>(P.D.q);
    for (int i = tid; i < RB * VPR; i += 256) {
      const int r = i / VPR, e = i % VPR * E;
      float x[E];
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (r < s.rows) {
        const int row = s.row0 + r, b = s.b0 + row / P.D.G;
        raw = *reinterpret_cast<const uint4*>(
            q + (static_cast<size_t>(b) * P.D.Hq + s.h * P.D.G + row % P.D.G) * D + e);
      }
      Elem<T>::unpack(raw, x);
#pragma unroll
      for (int j = 0; j < E; j++) s_q[r * LD + e + j] = x[j];
    }
    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 16; j++) o[i][j] = 0.0f;
    }
    for (int t = s.t0; t < s.t1; t++) {
      const int k0 = t * KT, nk = min(KT, s.prefix - k0);
      __syncthreads();
      for (int i = tid; i < KT * VPR; i += 256) {
        const int r = i / VPR, e = i % VPR * E;
        uint4 kr = make_uint4(0u, 0u, 0u, 0u), vr = kr;
        if (r < nk) {
          const size_t off = row_off(P.D, s.b0, s.h, k0 + r, D) + e;
          kr = ld_gather(static_cast<const T*>(P.D.k) + off);
          vr = ld_gather(static_cast<const T*>(P.D.v) + off);
        }
        float x[E], y[E];
        Elem<T>::unpack(kr, x);
        Elem<T>::unpack(vr, y);
#pragma unroll
        for (int j = 0; j < E; j++) {
          s_k[r * LD + e + j] = x[j];
          s_v[r * D + e + j] = y[j];
        }
      }
      __syncthreads();
      float sc[4][4];
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) sc[i][j] = 0.0f;
#pragma unroll 4
      for (int e = 0; e < D; e += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; i++) a[i] = *reinterpret_cast<const float4*>(s_q + (4 * ty + i) * LD + e);
#pragma unroll
        for (int j = 0; j < 4; j++) b[j] = *reinterpret_cast<const float4*>(s_k + (tx + 16 * j) * LD + e);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            sc[i][j] = fmaf(a[i].x, b[j].x, sc[i][j]);
            sc[i][j] = fmaf(a[i].y, b[j].y, sc[i][j]);
            sc[i][j] = fmaf(a[i].z, b[j].z, sc[i][j]);
            sc[i][j] = fmaf(a[i].w, b[j].w, sc[i][j]);
          }
      }
      // online softmax; the 16 lanes of a half warp share four rows
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          sc[i][j] = tx + 16 * j < nk ? sc[i][j] * c : -INFINITY;
          mx = fmaxf(mx, sc[i][j]);
        }
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(fmaxf(m[i], mx), -1e30f);  // finite: scores of -inf weigh exactly 0
        const float f = exp2f(m[i] - mn);
        m[i] = mn;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float p = exp2f(sc[i][j] - mn);
          sum += p;
          s_p[(4 * ty + i) * LP + tx + 16 * j] = p;
        }
        l[i] = l[i] * f + sum;
#pragma unroll
        for (int j = 0; j < D / 16; j++) o[i][j] *= f;
      }
      __syncwarp();  // a row's weights come from its own half warp
#pragma unroll 2
      for (int k = 0; k < KT; k += 4) {
        float pw[4][4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float4 w = *reinterpret_cast<const float4*>(s_p + (4 * ty + i) * LP + k);
          pw[i][0] = w.x;
          pw[i][1] = w.y;
          pw[i][2] = w.z;
          pw[i][3] = w.w;
        }
#pragma unroll
        for (int kk = 0; kk < 4; kk++)
#pragma unroll
          for (int jj = 0; jj < D / 64; jj++) {
            const float4 v = *reinterpret_cast<const float4*>(s_v + (k + kk) * D + jj * 64 + tx * 4);
#pragma unroll
            for (int i = 0; i < 4; i++) {
              o[i][4 * jj] = fmaf(pw[i][kk], v.x, o[i][4 * jj]);
              o[i][4 * jj + 1] = fmaf(pw[i][kk], v.y, o[i][4 * jj + 1]);
              o[i][4 * jj + 2] = fmaf(pw[i][kk], v.z, o[i][4 * jj + 2]);
              o[i][4 * jj + 3] = fmaf(pw[i][kk], v.w, o[i][4 * jj + 3]);
            }
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float sum = l[i];
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      const int r = 4 * ty + i;
      if (r >= s.rows) continue;
      const long long row = s.rec + r;
      if (tx == 0) P.W.ml[row] = make_float2(m[i], sum);
#pragma unroll
      for (int jj = 0; jj < D / 64; jj++)
        *reinterpret_cast<float4*>(P.W.rec + row * D + jj * 64 + tx * 4) =
            make_float4(o[i][4 * jj], o[i][4 * jj + 1], o[i][4 * jj + 2], o[i][4 * jj + 3]);
    }
    __syncthreads();
  }
  grid_dependents_launch();
}

// ============================================================ k_shared_combine
// One CTA per (sequence, KV head, query head of the group): folds the records
// of the prefix segments and of the gather.
constexpr int kSharedCombWarps = 4;

template <int D>
__global__ void __launch_bounds__(kSharedCombWarps * 32) k_shared_combine(const __grid_constant__ SharedParams P) {
  constexpr int PL = D / 32;
  __shared__ float s_acc[kSharedCombWarps][D];
  __shared__ float2 s_ml[kSharedCombWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  const DevParams& Q = P.D;
  const int u = blockIdx.x, gh = blockIdx.y;
  const int b = u / Q.Hkv, h = u % Q.Hkv;
  const UnitInfo inf = Q.info[u];
  float* out = Q.out + (static_cast<size_t>(b) * Q.Hq + h * Q.G + gh) * D;
  const bool shared = inf.s1 > 0;
  if (inf.n <= 0 || (shared && !P.W.pages_ok[inf.k])) {
    for (int e = threadIdx.x; e < D; e += blockDim.x) out[e] = 0.0f;
    return;
  }
  // records of the gather
  const long long To = Q.pre_det[2 * Q.units];
  const SliceRecs own = slice_recs(Q.pre_det, 2 * u, To, Q.CD);
  // records of the prefix
  SliceRecs pre{0, 0, 0, false};
  long long Tp = 0, base = 0;
  const int C = P.W.grid;
  if (shared) {
    const SharedGroup g = P.W.group[inf.k];
    Tp = P.W.group[P.groups].tile0;
    const int row = (b - g.b0) * Q.G + gh, mb = row / P.RB;
    const int rows = min(P.RB, g.size * Q.G - mb * P.RB);
    base = g.row0 + block_row0(P, mb, h, rows) + (row - mb * P.RB);
    pre.x0 = g.tile0 + (static_cast<long long>(mb) * Q.Hkv + h) * g.tiles;
    pre.per_item = Tp < C;
    pre.cf = pre.per_item ? 0 : cta_of(pre.x0, Tp, C);
    pre.n = pre.per_item ? g.tiles : cta_of(pre.x0 + g.tiles - 1, Tp, C) - pre.cf + 1;
  }
  const int np = pre.n, N = np + own.n;
  float m = -INFINITY, l = 0.0f, a[PL];
#pragma unroll
  for (int i = 0; i < PL; i++) a[i] = 0.0f;
  for (int j = warp; j < N; j += kSharedCombWarps) {
    float rm, rl;
    const float* src;
    if (j < np) {
      const long long row = static_cast<long long>(slice_rec(pre, Tp, C, j)) * P.RB + base;
      const float2 v = P.W.ml[row];
      rm = v.x;
      rl = v.y;
      src = P.W.rec + row * D;
    } else {
      const long long id = slice_rec(own, To, Q.CD, j - np) + 2LL * u;
      const float* r = Q.rec_det + static_cast<size_t>(id) * (Q.G * (2 + D)) + gh * (2 + D);
      rm = r[0] * 1.4426950408889634f;  // the gather keeps natural units
      rl = r[1];
      src = r + 2;
    }
    if (rl == 0.0f) continue;  // no key, or weights of zero alone
    const float nm = fmaxf(m, rm);
    const float fo = exp2f(m - nm), fn = exp2f(rm - nm);
    l = l * fo + rl * fn;
#pragma unroll
    for (int i = 0; i < PL; i++) a[i] = a[i] * fo + src[lane + 32 * i] * fn;
    m = nm;
  }
#pragma unroll
  for (int i = 0; i < PL; i++) s_acc[warp][lane + 32 * i] = a[i];
  if (lane == 0) s_ml[warp] = make_float2(m, l);
  __syncthreads();
  const int e = threadIdx.x;
  if (e >= D) return;
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kSharedCombWarps; w++) M = fmaxf(M, s_ml[w].x);
  float A = 0.0f, L = 0.0f;
#pragma unroll
  for (int w = 0; w < kSharedCombWarps; w++) {
    const float f = s_ml[w].x == -INFINITY ? 0.0f : exp2f(s_ml[w].x - M);
    L += s_ml[w].y * f;
    A += s_acc[w][e] * f;
  }
  out[e] = A / L;
}

}  // namespace vattn
