// Kernels of the shared-prefix decode (vattn_shared_dense_decode), in launch
// order:
//
//   k_shared_prep     validates lengths, groups and pages; the work of the two
//                     kernels behind it as prefix sums
//   k_shared_prefix(_tc)  every group's prefix against all of its queries
//   k_shared_own      every sequence's own positions (bf16 caches in device
//                     memory; others: k_gather<kModeSuffix>)
//   k_shared_combine  merges the records of both parts
//
// A group's G * (its sequences) query rows of one KV head meet the same keys,
// so the prefix is a matrix product with the rows of a block of RB on one side
// and tiles of KT keys on the other. Work is flattened as [group][row block]
// [KV head][key tile] and cut evenly over a persistent grid; each (CTA, block,
// head) segment leaves one record (maximum, weight sum, weighted values) per
// row. Only groups of which min_reach sequences reach the end of the prefix are
// shared: the others, and sequences shorter than their prefix, are left to
// the own part whole, so that no row of a segment is masked and every key of a
// tile counts for every row. The prefix of a sequence that reaches its end is
// read through the pages of the group's first sequence in every case: the
// gather looks each position up in the one row or the other; k_shared_own reads
// one row per sequence, so for it a single sequence behind a first one that is
// shorter makes a group shared.
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
  CUtensorMap tmk_16, tmv_16;  // the caches in boxes of 16 rows (k_shared_own)
  DevParams D;
  SharedWork W;
  const int* group_start;
  const int* prefix_lens;
  int groups;
  int RB, KT;  // rows of a block, keys of a tile
  int box;     // rows of a cache box: a power of two that divides the page size, at most KT
  int own_warps;  // k_shared_own's warps; 0: the gather takes the own positions
  int min_reach;  // sequences that have to reach a prefix's end for it to be shared, at least 2 (but see is_shared)
};

// ---------------------------------------------------------------- groups
// Record rows of a whole group's query rows are its query rows per KV head;
// a block's records of KV head h start behind those of the blocks and heads
// before it.
__device__ __forceinline__ long long block_row0(const SharedParams& P, int mb, int h, int rows) {
  return static_cast<long long>(mb) * P.RB * P.D.Hkv + static_cast<long long>(h) * rows;
}

// Key tiles and record rows of a shared group (its sequences and prefix given).
__device__ __forceinline__ void group_work(const SharedParams& P, SharedGroup& g, long long& tiles, long long& rows) {
  const int nrow = g.size * P.D.G;
  g.tiles = (g.prefix + P.KT - 1) / P.KT;
  tiles = static_cast<long long>(g.tiles) * ((nrow + P.RB - 1) / P.RB) * P.D.Hkv;
  rows = static_cast<long long>(nrow) * P.D.Hkv;
}

// How far a group's sequences reach: a count of those that reach the prefix's
// end, plus kFirstShort if the first sequence does not.
constexpr int kFirstShort = 1 << 30;
__device__ __forceinline__ bool is_shared(const SharedParams& P, int reach) {
  const int cnt = reach & (kFirstShort - 1);
  return cnt >= P.min_reach || (P.own_warps > 0 && cnt > 0 && cnt != reach);
}

// The running maxima start here: finite, so that scores of -inf weigh exactly 0,
// and below every finite score.
constexpr float kLowest = -3.402823466e38f;

// Chunks of k_shared_own that cover positions [start, n): kOwnChunk positions
// each from the 16-position block that holds `start`. Warps take them in pieces
// of at least kOwnPiece chunks of one (sequence, KV head), about kOwnPieces a
// warp when there are many.
constexpr int kOwnPiece = 6, kOwnPieces = 6;
// Chunks after which a piece's accumulator is added to its fp32 sum: the tensor
// core truncates with every product added (see kFlush in vattn_prefix_tc.cuh).
constexpr int kOwnFlush = 32;
constexpr int kOwnChunk = 16;
__device__ __forceinline__ int own_chunks(int start, int n) {
  return n > start ? (n - (start & ~15) + kOwnChunk - 1) / kOwnChunk : 0;
}

// ============================================================ k_shared_prep
constexpr int kSharedPrepThreads = 256;
constexpr int kSharedPrepKeep = 1024;  // sequences and groups kept in shared memory by the last CTA

__device__ __forceinline__ int checked_len(const SharedParams& P, int b) {
  const int n = __ldcg(P.D.seq_lens + b);
  return n < 0 || n > P.D.max_ctx ? -1 : n;
}

// Whether any of the page ids of row `b` in slots [s0, s1) is out of range (a warp).
__device__ __forceinline__ bool bad_pages(const SharedParams& P, int b, int s0, int s1) {
  int bad = 0;
  for (int i0 = s0 + (threadIdx.x & 31); i0 < s1; i0 += 8 * 32) {  // eight independent loads in flight
    int pid[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int i = i0 + j * 32;
      pid[j] = i < s1 ? P.D.page_table[static_cast<size_t>(b) * P.D.pps + i] : 0;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (pid[j] < 0 || pid[j] >= P.D.num_pages) bad = 1;
  }
  return __any_sync(0xffffffffu, bad);
}

// How far the sequences [b0, b1) reach with a prefix of `prefix` (a warp).
__device__ __forceinline__ int count_reach(const SharedParams& P, int b0, int b1, int prefix) {
  int cnt = 0;
  for (int base = b0; base < b1; base += 32) {
    const int b = base + (threadIdx.x & 31);
    const unsigned reach = __ballot_sync(0xffffffffu, b < b1 && prefix > 0 && checked_len(P, b) >= prefix);
    if (base == b0 && prefix > 0 && !(reach & 1u)) cnt = kFirstShort;
    cnt += __popc(reach);
  }
  return cnt;
}

// Inclusive 64-bit prefix sum over the block's 256 threads.
__device__ __forceinline__ long long block_scan_ll(long long v, long long* s_w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) s_w[warp] = v;  // the warps' sums stay there
  __syncthreads();
  for (int w = 0; w < warp; w++) v += s_w[w];
  __syncthreads();
  return v;
}

// The last two CTAs find the prefix kernel's work and the own parts' as prefix
// sums; every warp of the others one sequence or one group (its pages). Few
// CTAs, because the prefix kernel, which runs beside them, has to wait for the
// SMs that they are on.
static __global__ void __launch_bounds__(kSharedPrepThreads) k_shared_prep(const __grid_constant__ SharedParams P) {
  const int tid = threadIdx.x;
  const DevParams& D = P.D;
  // (the tensor-core prefix kernel starts on this signal, before this kernel's
  // end: everything before the call has to have ended)
  grid_dependency_wait();
  grid_dependents_launch();

  if (blockIdx.x < gridDim.x - 2) {
    const int job = blockIdx.x * (kSharedPrepThreads / 32) + (tid >> 5), lane = tid & 31;
    if (job >= D.batch + P.groups) return;
    // the bounds ascend from 0 to batch, or nothing is decoded; with ascending
    // bounds at most one group holds a sequence
    int bad = 0, own = -1;
    for (int g = lane; g < P.groups; g += 32) {
      const int lo = P.group_start[g], hi = P.group_start[g + 1];
      if (hi < lo || (g == 0 && lo != 0) || (g == P.groups - 1 && hi != D.batch)) bad = 1;
      if (job < D.batch && lo <= job && job < hi) own = g;
    }
    const bool bad_bounds = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int o = 16; o; o >>= 1) own = max(own, __shfl_xor_sync(0xffffffffu, own, o));
    if (job < D.batch) {
      const int b = job, g = own;
      // positions [0, start) are left to the prefix kernel, [start, first) are read
      // through the pages of the group's first sequence b0, the rest through its own
      int n = checked_len(P, b), start = 0, first = 0, b0 = 0;
      if (lane == 0 && n < 0) atomicOr(D.err, kDevBadSeqlen);
      if (n < 0 || bad_bounds || g < 0) n = 0;
      if (n > 0) {
        const int prefix = P.prefix_lens[g];
        if (prefix < 0 || prefix > D.max_ctx) {
          n = 0;
        } else if (n >= prefix && prefix > 0) {
          b0 = P.group_start[g];
          if (is_shared(P, count_reach(P, b0, P.group_start[g + 1], prefix))) start = prefix;
          else if (b != b0) first = prefix;
        }
      }
      const int own0 = max(start, first);
      if ((n > own0 && bad_pages(P, b, own0 / D.ps, (n + D.ps - 1) / D.ps)) ||
          (n > 0 && first > 0 && bad_pages(P, b0, 0, (first + D.ps - 1) / D.ps))) {
        if (lane == 0) atomicOr(D.err, kDevBadPage);
        n = 0;
      }
      for (int h = lane; h < D.Hkv; h += 32) {
        UnitInfo inf = {};
        inf.n = n;
        inf.s1 = start;
        inf.wst = first;
        inf.k = g;
        inf.p = b0;
        D.info[static_cast<size_t>(b) * D.Hkv + h] = inf;
      }
      return;
    }
    const int g = job - D.batch;
    int ok = 0;
    if (!bad_bounds) {
      const int prefix = P.prefix_lens[g], b0 = P.group_start[g], b1 = P.group_start[g + 1];
      if (prefix < 0 || prefix > D.max_ctx) {
        if (lane == 0) atomicOr(D.err, kDevBadGroup);
      } else {
        ok = 1;
        if (is_shared(P, count_reach(P, b0, b1, prefix)) && bad_pages(P, b0, 0, (prefix + D.ps - 1) / D.ps)) {
          if (lane == 0) atomicOr(D.err, kDevBadPage);
          ok = 0;
        }
      }
    }
    if (lane == 0) P.W.pages_ok[g] = ok;
    return;
  }

  // ---- prefix sums. The inputs come into shared memory in one round of loads
  // (what does not fit is read where it is).
  const bool own_cta = blockIdx.x == gridDim.x - 1;
  int* g_reach = P.W.reach + (own_cta ? P.groups : 0);
  __shared__ int s_len[kSharedPrepKeep], s_prefix[kSharedPrepKeep], s_reach[kSharedPrepKeep];
  __shared__ int s_start[kSharedPrepKeep + 1];
  __shared__ long long s_w[kSharedPrepThreads / 32], s_carry[2];
  __shared__ int s_bad;
  for (int b = tid; b < min(D.batch, kSharedPrepKeep); b += blockDim.x) s_len[b] = checked_len(P, b);
  for (int g = tid; g < min(P.groups, kSharedPrepKeep); g += blockDim.x) {
    s_prefix[g] = P.prefix_lens[g];
    s_reach[g] = 0;
  }
  for (int g = tid; g < min(P.groups, kSharedPrepKeep) + 1; g += blockDim.x) s_start[g] = P.group_start[g];
  for (int g = kSharedPrepKeep + tid; g < P.groups; g += blockDim.x) g_reach[g] = 0;
  if (tid == 0) {
    s_bad = 0;
    s_carry[0] = s_carry[1] = 0;
  }
  __syncthreads();
  auto len = [&](int b) -> int { return b < kSharedPrepKeep ? s_len[b] : checked_len(P, b); };
  auto start_of = [&](int g) -> int { return g <= kSharedPrepKeep ? s_start[g] : P.group_start[g]; };
  auto prefix_of = [&](int g) -> int { return g < kSharedPrepKeep ? s_prefix[g] : P.prefix_lens[g]; };
  auto reach_of = [&](int g) -> int {
    return g < kSharedPrepKeep ? s_reach[g] : *static_cast<volatile int*>(&g_reach[g]);
  };
  auto group_of = [&](int b) -> int {  // the last g with group_start[g] <= b
    int lo = 0, hi = P.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (start_of(mid) <= b) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  for (int g = tid; g < P.groups; g += blockDim.x) {
    const int lo = start_of(g), hi = start_of(g + 1);
    if (hi < lo || (g == 0 && lo != 0) || (g == P.groups - 1 && hi != D.batch)) s_bad = 1;
  }
  __syncthreads();
  const bool bad_bounds = s_bad != 0;
  if (bad_bounds && tid == 0 && !own_cta) atomicOr(D.err, kDevBadGroup);
  if (!bad_bounds) {
    for (int b = tid; b < D.batch; b += blockDim.x) {
      const int g = group_of(b), prefix = prefix_of(g);
      if (prefix <= 0 || prefix > D.max_ctx) continue;
      const int add = len(b) >= prefix ? 1 : b == start_of(g) ? kFirstShort : 0;
      if (add) atomicAdd(g < kSharedPrepKeep ? &s_reach[g] : &g_reach[g], add);
    }
  }
  __threadfence_block();
  __syncthreads();
  if (!own_cta) {
    // key tiles and record rows over groups
    long long tiles = 0, rows = 0;
    for (int base = 0; base < P.groups; base += blockDim.x) {
      const int g = base + tid;
      long long t = 0, r = 0;
      SharedGroup rec = {};
      if (g < P.groups && !bad_bounds) {
        rec.b0 = start_of(g);
        rec.size = start_of(g + 1) - rec.b0;
        rec.prefix = prefix_of(g);
        if (is_shared(P, reach_of(g))) group_work(P, rec, t, r);
      }
      const long long it = block_scan_ll(t, s_w), ir = block_scan_ll(r, s_w);
      if (g < P.groups) {
        rec.tile0 = tiles + it - t;
        rec.row0 = rows + ir - r;
        P.W.group[g] = rec;
      }
      if (tid == blockDim.x - 1) {
        s_carry[0] += it;
        s_carry[1] += ir;
      }
      __syncthreads();
      tiles = s_carry[0];
      rows = s_carry[1];
      __syncthreads();
    }
    if (tid == 0) {
      SharedGroup rec = {};
      rec.tile0 = tiles;
      rec.row0 = rows;
      P.W.group[P.groups] = rec;
    }
    return;
  }
  // the own parts: a sequence whose pages fail keeps its part here and is
  // skipped by its kernel
  auto own_start = [&](int b) -> int {  // -1: no own part
    if (b >= D.batch || bad_bounds) return -1;
    const int g = group_of(b), n = len(b), prefix = prefix_of(g);
    if (n <= 0 || prefix < 0 || prefix > D.max_ctx) return -1;
    return prefix > 0 && n >= prefix && is_shared(P, reach_of(g)) ? prefix : 0;
  };
  if (P.own_warps) {
    long long sum = 0;  // chunks of one KV head
    for (int b = tid; b < D.batch; b += blockDim.x) {
      const int start = own_start(b);
      if (start >= 0) sum += own_chunks(start, len(b));
    }
    block_scan_ll(sum, s_w);
    if (tid < 32) {
      long long v = tid < kSharedPrepThreads / 32 ? s_w[tid] : 0;
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (tid == 0) s_carry[1] = v;
    }
    __syncthreads();
    const long long most = static_cast<long long>(kOwnPieces) * P.own_warps;
    const int piece = static_cast<int>(max(static_cast<long long>(kOwnPiece), (s_carry[1] * D.Hkv + most - 1) / most));
    __shared__ int s_pre[kSharedPrepKeep + 1];
    for (int base = 0; base < D.batch; base += blockDim.x) {
      const int b = base + tid, start = own_start(b);
      const int cnt = start >= 0 ? (own_chunks(start, len(b)) + piece - 1) / piece : 0;
      const long long carry = s_carry[0], incl = block_scan_ll(cnt, s_w);
      if (b < D.batch) {
        const int pre = static_cast<int>(carry + incl - cnt);
        if (b < kSharedPrepKeep) s_pre[b] = pre;
        P.W.own_pre[b] = pre;
      }
      __syncthreads();
      if (tid == blockDim.x - 1) s_carry[0] = carry + incl;
      __syncthreads();
    }
    const int total = static_cast<int>(s_carry[0]);
    if (tid == 0) {
      P.W.own_pre[D.batch] = total;
      P.W.own_next[0] = 0;
    }
    __threadfence_block();
    __syncthreads();
    auto pre_of = [&](int b) -> int {
      return b < kSharedPrepKeep ? s_pre[b] : *static_cast<volatile int*>(&P.W.own_pre[b]);
    };
    // the pieces themselves
    for (int j = tid; j < total; j += blockDim.x) {
      int lo = 0, hi = D.batch;  // the last sequence whose pieces begin at or before j
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (pre_of(mid) <= j) lo = mid;
        else hi = mid;
      }
      const int first = (j - pre_of(lo)) * piece, start = own_start(lo), n = len(lo);
      OwnPiece e = {};
      e.b = lo;
      e.pos = (start & ~15) + kOwnChunk * first;
      e.chunks = min(piece, own_chunks(start, n) - first);
      e.start = start;
      e.n = n;
      P.W.own_piece[j] = e;
    }
    return;
  }
  for (int base = 0; base < D.batch; base += blockDim.x) {
    const int b = base + tid, start = own_start(b), cnt = start >= 0 ? len(b) - start : 0;
    const long long carry = s_carry[0], incl = block_scan_ll(cnt, s_w);
    if (b < D.batch) {
      const long long at = (carry + incl - cnt) * D.Hkv;
      for (int h = 0; h < D.Hkv; h++) {
        const size_t s = 2 * (static_cast<size_t>(b) * D.Hkv + h);
        D.pre_det[s] = at + static_cast<long long>(h) * cnt;
        D.pre_det[s + 1] = at + static_cast<long long>(h + 1) * cnt;
      }
    }
    __syncthreads();
    if (tid == blockDim.x - 1) s_carry[0] = carry + incl;
    __syncthreads();
  }
  if (tid == 0) D.pre_det[2 * static_cast<size_t>(D.units)] = s_carry[0] * D.Hkv;
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
  s.rec = static_cast<long long>(blockIdx.x) * P.W.stride + g.row0 + block_row0(P, s.mb, s.h, s.rows);
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

// 16 bytes global -> shared past L1; zeros instead when !in
__device__ __forceinline__ void cp_async16_or_zero(float* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
               "l"(__cvta_generic_to_global(src)), "r"(in ? 16 : 0)
               : "memory");
}

// ============================================================ k_shared_prefix
// fp32 caches, and caches in host memory: fp32 FMAs, bound by them from a few
// sequences on (32 sequences x 4 heads over 16384 keys, d = 128: 8.6 GFLOP in
// 0.25 ms, 34 TFLOP/s). Blocks of 64 rows against tiles of 64 keys; 256 threads as
// 16 x 16, each with 4 x 4 scores and 4 rows of D / 16 outputs, all operands in
// shared memory as fp32.
template <int D>
struct PrefixShape {
  static constexpr int RB = 64, KT = 64;
  static constexpr int LD = D + 4;    // row pitch of Q and K: 16-byte rows that start in different banks
  static constexpr int LP = KT + 4;
  static constexpr int TILE = KT * LD + KT * D;  // K and V of a tile
  static constexpr size_t SMEM = static_cast<size_t>(RB * LD + 2 * TILE + RB * LP) * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory of the prefix kernel");
};

template <typename T, int D, bool HOST>
__global__ void __launch_bounds__(256, 1) k_shared_prefix(const __grid_constant__ SharedParams P) {
  using S = PrefixShape<D>;
  constexpr int RB = S::RB, KT = S::KT, LD = S::LD, LP = S::LP, E = Elem<T>::kPer16, VPR = D / E;
  extern __shared__ __align__(16) float sm[];
  float* s_q = sm;
  float* s_kv = s_q + RB * LD;  // two tiles
  float* s_p = s_kv + 2 * S::TILE;
  // fp32 rows in device memory are copied asynchronously, a tile ahead
  constexpr bool kAhead = sizeof(T) == 4 && !HOST;
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
    // K and V of tile t into buffer t % 2; rows behind the prefix are zeros
    auto load = [&](int t) {
      const int k0 = t * KT, nk = min(KT, s.prefix - k0);
      float* s_k = s_kv + (t & 1) * S::TILE;
      float* s_v = s_k + KT * LD;
      for (int i = tid; i < KT * VPR; i += 256) {
        const int r = i / VPR, e = i % VPR * E;
        const size_t off = r < nk ? row_off(P.D, s.b0, s.h, k0 + r, D) + e : 0;
        if constexpr (kAhead) {
          cp_async16_or_zero(s_k + r * LD + e, static_cast<const T*>(P.D.k) + off, r < nk);
          cp_async16_or_zero(s_v + r * D + e, static_cast<const T*>(P.D.v) + off, r < nk);
        } else {
          uint4 kr = make_uint4(0u, 0u, 0u, 0u), vr = kr;
          if (r < nk) {
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
      }
      if constexpr (kAhead) cp_async_commit();
    };
    const bool busy = 4 * (ty & ~1) < s.rows;  // the warp has query rows
    if constexpr (kAhead) load(s.t0);
    for (int t = s.t0; t < s.t1; t++) {
      const int nk = min(KT, s.prefix - t * KT);
      const float* s_k = s_kv + (t & 1) * S::TILE;
      const float* s_v = s_k + KT * LD;
      if constexpr (kAhead) {
        cp_async_wait<0>();
        __syncthreads();
        if (t + 1 < s.t1) load(t + 1);  // into the buffer that the tile before left
      } else {
        load(t);
        __syncthreads();
      }
      if (!busy) continue;
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
        const float mn = fmaxf(fmaxf(m[i], mx), kLowest);
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

// ============================================================ k_shared_own
// Every sequence's positions behind its shared prefix (all of them where
// nothing is shared), for bf16 caches in device memory. They come in many short
// runs, so a warp's chunks (16 positions inside one page: 4 KB of K and of V in
// a row at d = 128) form one stream: a ring of NS chunks in shared memory is
// filled NS - 1 chunks ahead of the one being computed, across the ends of
// runs, by two or four tensor copies a chunk. SMs stream at rates that differ
// by a third, and the prefix kernel leaves them at different times, so warps
// take pieces of runs from a counter (the first by their index; the KV heads of
// a piece follow one another); a piece has the record of its index. The arithmetic of a chunk is k_gather_tc's: S = K q
// as m16n8k16 products, the online softmax in the accumulator layout,
// O^T += V^T P with the weights as two bf16 terms.
// The kernel needs k_shared_prep's results alone: it starts while the prefix
// kernel's last CTAs run (which start after k_shared_prep's end) and waits
// for them only before it ends, so that its own end means both. What
// k_shared_prep wrote is therefore read past L1.
// 256 sequences x 150 positions, 8 heads, d = 128 (165 MB): 30 us, 5.5 TB/s; as
// slices of k_gather_tc, whose rings drain at every end, 73 us, and with the
// pieces cut statically 55 us.
template <int D>
struct OwnShape {
  static constexpr int H = D / 64, KT = D / 16;
  static constexpr int HALF = 16 * 128;              // 16 rows of a 64-column half
  static constexpr int MAT = H * HALF;
  static constexpr int STAGE = 2 * MAT;              // a chunk: K, then V
  static constexpr int NW = 7, THREADS = NW * 32;
  static constexpr int NS = D == 128 ? 4 : 6;
  static constexpr int QUEUE = 8;                    // pieces between the copies and the arithmetic: at most NS + 1
  static constexpr size_t RING = static_cast<size_t>(NW) * NS * STAGE;
  static constexpr size_t SMEM = RING + static_cast<size_t>(NW) * (NS * 8 + QUEUE * sizeof(OwnPiece));
  static_assert(NS + 1 <= QUEUE && SMEM <= 227 * 1024, "shared memory of the own part");
};

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

template <int D, int G>
__global__ void __launch_bounds__(OwnShape<D>::THREADS, 1) k_shared_own(const __grid_constant__ SharedParams P) {
  using S = OwnShape<D>;
  constexpr int H = S::H, KT = S::KT, HALF = S::HALF, NS = S::NS, STAGE = S::STAGE, MAT = S::MAT;
  extern __shared__ __align__(1024) unsigned char s_tiles[];
  const DevParams& Q = P.D;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = P.own_warps, gw = blockIdx.x * S::NW + warp;
  unsigned char* ring = s_tiles + warp * NS * STAGE;
  const unsigned ring_s = smem_u32(ring);
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_tiles + S::RING) + warp * NS;
  OwnPiece* queue = reinterpret_cast<OwnPiece*>(s_tiles + S::RING + S::NW * NS * 8) + warp * S::QUEUE;
  if (lane < NS) mbar_init(&bars[lane], 1);
  mbar_init_fence();
  __syncwarp();
  grid_dependents_launch();  // k_shared_combine fills the SMs that this kernel leaves
  // (the array holds more entries than there are warps, used or not)
  const int4* first = reinterpret_cast<const int4*>(&P.W.own_piece[gw / Q.Hkv]);
  const int4 first_a = __ldcg(first), first_b = __ldcg(first + 1);
  const int total = __ldcg(&P.W.own_pre[Q.batch]) * Q.Hkv;
  const float c = Q.scale * 1.4426950408889634f;  // scores in log2 units

  if (gw < total) {
    // Producer: the piece being copied (pp), its next chunk and that chunk's
    // page, and the piece after it (pn), which is fetched in three dependent
    // steps, one with every chunk copied: its index, its entry, its state and
    // first page.
    OwnPiece pp, pn;
    int px = 0, page = 0, id_n = gw, page_n = 0, n_n = 0, step = 2;
    unsigned nq = 0, dq = 0;  // pieces queued and taken
    unsigned ni = 0, nc = 0;  // chunks copied and computed (stage and phase follow)
    auto page_of = [&](const OwnPiece& p, int x) -> int {
      return __ldcg(Q.page_table + static_cast<size_t>(p.b) * Q.pps + page_slot(Q, p.pos + kOwnChunk * x));
    };
    auto take = [&](const int4& a, const int4& b) {
      pn.b = a.x;
      pn.pos = a.y;
      pn.chunks = a.z;
      pn.start = a.w;
      pn.n = b.x;
      pn.id = id_n;
    };
    take(first_a, first_b);
    auto fetch_step = [&]() {  // 0 -> 3; 4: no piece is left
      if (step == 0) {
        if (lane == 0) id_n = W + atomicAdd(&P.W.own_next[0], 1);
        step = 1;
      } else if (step == 1) {
        id_n = __shfl_sync(0xffffffffu, id_n, 0);
        step = id_n < total ? 2 : 4;
        if (step == 2) {
          const int4* e = reinterpret_cast<const int4*>(&P.W.own_piece[id_n / Q.Hkv]);
          take(__ldcg(e), __ldcg(e + 1));
        }
      } else if (step == 2) {
        n_n = __ldcg(&Q.info[static_cast<size_t>(pn.b) * Q.Hkv].n);
        page_n = page_of(pn, 0);
        step = 3;
      }
    };
    // the next piece that can be read becomes the one being copied
    auto advance = [&]() -> bool {
      do {
        while (step < 3) fetch_step();
        if (step == 4) return false;
        pp = pn;
        step = 0;
      } while (n_n <= 0);  // a sequence whose pages failed
      px = 0;
      page = page_n;
      if (lane == 0) queue[nq % S::QUEUE] = pp;
      __syncwarp();
      nq++;
      return true;
    };
    bool left = advance();
    auto issue = [&]() {  // one chunk, if there is one and a stage is free
      if (ni - nc >= NS) return;
      if (left && px >= pp.chunks) left = advance();
      if (!left) return;
      const int pos = pp.pos + kOwnChunk * px;
      const int row = (page * Q.Hkv + pp.id % Q.Hkv) * Q.ps + (pos - page_slot(Q, pos) * Q.ps);
      const int st = static_cast<int>(ni % NS);
      fence_proxy_async();  // the stage's earlier reads come before the copy's writes
      if (lane == 0) mbar_arrive_expect_tx(&bars[st], STAGE);
      __syncwarp();
      if (lane < 2 * H)
        tma_2d(ring + st * STAGE + lane * HALF, lane < H ? &P.tmk_16 : &P.tmv_16, (lane % H) * 64, row, &bars[st]);
      ni++;
      px++;
      if (px < pp.chunks) page = page_of(pp, px);
      if (step < 3) fetch_step();
    };
#pragma unroll 1
    for (int i = 0; i < NS - 1; i++) issue();

    const int fj = lane >> 3, fr = lane & 7;  // ldmatrix.x4: matrix lane / 8, row lane % 8
    const int hc = 2 * (lane & 3), ra = lane >> 2;
    bool ok = true;
    while (dq < nq && ok) {
      const OwnPiece cu = queue[dq % S::QUEUE];
      dq++;
      // the query operand: lane holds head lane / 4, dims 16 kt + 2 (lane % 4)
      // + {0, 1} and those + 8 (zero columns past G)
      unsigned qf[KT][2];
      {
        const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(Q.q) +
                                  (static_cast<size_t>(cu.b) * Q.Hq + (cu.id % Q.Hkv) * G + (ra < G ? ra : 0)) * D + hc;
#pragma unroll
        for (int kt = 0; kt < KT; kt++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const unsigned v = __ldcg(reinterpret_cast<const unsigned*>(qp + 16 * kt + 8 * e));
            qf[kt][e] = ra < G ? v : 0u;
          }
      }
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, o[KT][4], sum[KT][4];
#pragma unroll
      for (int mt = 0; mt < KT; mt++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[mt][e] = sum[mt][e] = 0.0f;
      auto flush = [&]() {
#pragma unroll
        for (int mt = 0; mt < KT; mt++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            sum[mt][e] += o[mt][e];
            o[mt][e] = 0.0f;
          }
      };
#pragma unroll 1
      for (int x = 0; x < cu.chunks; x++) {
        issue();  // into the stage that the chunk before left
        const int st = static_cast<int>(nc % NS);
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[st], (nc / NS) & 1u));
        if (!ok) break;
        nc++;
        const int pos = cu.pos + kOwnChunk * x;
        const int r0 = max(cu.start - pos, 0), r1 = min(cu.n - pos, 16);  // own rows of the block
        const unsigned kb = ring_s + st * STAGE, vb = kb + MAT;
        const bool part = r1 - r0 < 16;
        if (part) {
          // V rows of no own key: zeros, whatever the cache holds there
          for (int i = lane; i < 16 * 8; i += 32)
            if (i / 8 < r0 || i / 8 >= r1)
#pragma unroll
              for (int hf = 0; hf < H; hf++)
                *reinterpret_cast<uint4*>(ring + st * STAGE + MAT + hf * HALF + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          __syncwarp();
        }
        // two chains of products: even and odd k-steps
        float sc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kt = 0; kt < KT; kt += 2) {
          unsigned a[4], b[4];
          ldsm_x4(kb + tc_off(((fj & 1) << 3) | fr, 2 * kt + (fj >> 1)), a);
          ldsm_x4(kb + tc_off(((fj & 1) << 3) | fr, 2 * kt + 2 + (fj >> 1)), b);
          mma_bf16(sc, a, qf[kt][0], qf[kt][1]);
          mma_bf16(sd, b, qf[kt + 1][0], qf[kt + 1][1]);
        }
        // online softmax: rows lane / 4 (values 0, 1) and lane / 4 + 8 (2, 3)
        float sv[4];
#pragma unroll
        for (int e = 0; e < 4; e++) sv[e] = (sc[e] + sd[e]) * c;
        if (part) {
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int r = ra + (e >> 1) * 8;
            if (r < r0 || r >= r1) sv[e] = -INFINITY;
          }
        }
        float bm[2] = {fmaxf(sv[0], sv[2]), fmaxf(sv[1], sv[3])};
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
#pragma unroll
          for (int k = 0; k < 2; k++) bm[k] = fmaxf(bm[k], __shfl_xor_sync(0xffffffffu, bm[k], off));
        if (__any_sync(0xffffffffu, bm[0] > m[0] || bm[1] > m[1])) {
          float f[2];
#pragma unroll
          for (int k = 0; k < 2; k++) {
            const float nm = fmaxf(fmaxf(m[k], bm[k]), kLowest);
            f[k] = exp2f(m[k] - nm);
            m[k] = nm;
            l[k] *= f[k];
          }
#pragma unroll
          for (int mt = 0; mt < KT; mt++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              o[mt][e] *= f[e & 1];
              sum[mt][e] *= f[e & 1];
            }
        }
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; e++) pv[e] = exp2f(sv[e] - m[e & 1]);
#pragma unroll
        for (int k = 0; k < 2; k++) l[k] += pv[k] + pv[2 + k];
        // the weights as the B operand: transposes of the [row][head pair] fragments
        unsigned ph0, pl0, ph1, pl1;
        split_bf16x2(pv[0], pv[1], ph0, pl0);
        split_bf16x2(pv[2], pv[3], ph1, pl1);
        ph0 = movm_t(ph0);
        pl0 = movm_t(pl0);
        ph1 = movm_t(ph1);
        pl1 = movm_t(pl1);
#pragma unroll
        for (int mt = 0; mt < KT; mt++) {
          unsigned a[4];
          ldsm_x4_t(vb + tc_off(((fj >> 1) << 3) | fr, 2 * mt + (fj & 1)), a);
          mma_bf16(o[mt], a, ph0, ph1);
          mma_bf16(o[mt], a, pl0, pl1);
        }
        if ((x + 1) % kOwnFlush == 0) flush();
        __syncwarp();  // the stage is free again
      }
      if (!ok) break;
      flush();
      // the piece's record: lane holds dims 16 mt + lane / 4 (+ 8)
      // of heads hc, hc + 1
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int k = 0; k < 2; k++) l[k] += __shfl_xor_sync(0xffffffffu, l[k], off);
      const size_t rec = static_cast<size_t>(cu.id) * G;
#pragma unroll
      for (int k = 0; k < 2; k++) {
        if (hc + k >= G) continue;
        if (ra == 0) P.W.own_ml[rec + hc + k] = make_float2(m[k], l[k]);
        float* r = P.W.own_rec + (rec + hc + k) * D + ra;
#pragma unroll
        for (int mt = 0; mt < KT; mt++) {
          r[16 * mt] = sum[mt][k];
          r[16 * mt + 8] = sum[mt][2 + k];
        }
      }
    }
    if (!ok) {
      if (lane == 0) atomicOr(Q.err, kDevTimeout);
      for (; nc != ni; nc++) mbar_wait(&bars[nc % NS], (nc / NS) & 1u);  // no copy lands after the warp has moved on
    }
  }
  grid_dependency_wait();
}

// ============================================================ k_shared_combine
// WR warps per (sequence, query head): fold the records of the prefix segments
// and of the own parts, 32 at a time: a lane reads one record's maximum and
// weight sum, then every lane adds its columns of each record under weights
// that are all known, so that the loads of several records are in flight. Bound
// by latency: 6 us behind the last record for 8192 rows of 7 records (30 MB).
constexpr int kSharedCombWarps = 8;

template <int D, int WR>
__global__ void __launch_bounds__(kSharedCombWarps * 32) k_shared_combine(const __grid_constant__ SharedParams P) {
  constexpr int PL = D / 64;  // float2 columns per lane
  __shared__ float2 s_acc[WR > 1 ? kSharedCombWarps : 1][PL][32];
  __shared__ float2 s_ml[kSharedCombWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const DevParams& Q = P.D;
  const int row_out = blockIdx.x * (kSharedCombWarps / WR) + warp / WR, part = warp % WR;
  // With k_shared_own before it the kernel starts after k_shared_prep's end, and
  // finds where its records are while the last of them are written; what
  // k_shared_prep wrote is read past L1. Behind the gather it waits first.
  if (!P.own_warps) grid_dependency_wait();
  grid_dependents_launch();
  const bool real = row_out < Q.batch * Q.Hq;
  const int b = real ? row_out / Q.Hq : 0, hq = row_out % Q.Hq, h = hq / Q.G, gh = hq % Q.G, u = b * Q.Hkv + h;
  const int4 i0 = __ldcg(reinterpret_cast<const int4*>(Q.info + u));  // n, s1, wst, k
  const int n_pos = i0.x, start = i0.y, gi = i0.w;
  float* out = Q.out + static_cast<size_t>(row_out) * D;
  const bool shared = start > 0;
  const bool none = n_pos <= 0 || (shared && !__ldcg(P.W.pages_ok + gi));
  // records of the own part
  long long To = 0, own0 = 0;
  SliceRecs own{0, 0, 0, false};
  if (P.own_warps) {
    own0 = __ldcg(P.W.own_pre + b);
    own.n = __ldcg(P.W.own_pre + b + 1) - static_cast<int>(own0);
  } else {
    To = Q.pre_det[2 * Q.units];
    own = slice_recs(Q.pre_det, 2 * u, To, Q.CD);
  }
  // records of the prefix
  SliceRecs pre{0, 0, 0, false};
  long long Tp = 0, base = 0;
  const int C = P.W.grid;
  if (shared) {
    SharedGroup g;
    const int4* gp = reinterpret_cast<const int4*>(P.W.group + gi);
    reinterpret_cast<int4*>(&g)[0] = __ldcg(gp);
    reinterpret_cast<int4*>(&g)[1] = __ldcg(gp + 1);
    Tp = __ldcg(&P.W.group[P.groups].tile0);
    const int row = (b - g.b0) * Q.G + gh, mb = row / P.RB;
    const int rows = min(P.RB, g.size * Q.G - mb * P.RB);
    base = g.row0 + block_row0(P, mb, h, rows) + (row - mb * P.RB);
    pre.x0 = g.tile0 + (static_cast<long long>(mb) * Q.Hkv + h) * g.tiles;
    pre.per_item = Tp < C;
    pre.cf = pre.per_item ? 0 : cta_of(pre.x0, Tp, C);
    pre.n = pre.per_item ? g.tiles : cta_of(pre.x0 + g.tiles - 1, Tp, C) - pre.cf + 1;
  }
  const int np = pre.n, N = real && !none ? np + own.n : 0;
  if (P.own_warps) grid_dependency_wait();
  float m = -INFINITY, l = 0.0f;
  float2 a[PL];
#pragma unroll
  for (int i = 0; i < PL; i++) a[i] = make_float2(0.0f, 0.0f);
  const int mine = (N - part + WR - 1) / WR;  // records part, part + WR, ...
  for (int j0 = 0; j0 < mine; j0 += 32) {
    const int j = j0 + lane < mine ? part + WR * (j0 + lane) : N;
    float rm = -INFINITY, rl = 0.0f;
    const float* src = nullptr;
    if (j < np) {
      const long long row = static_cast<long long>(slice_rec(pre, Tp, C, j)) * P.W.stride + base;
      const float2 v = P.W.ml[row];
      rm = v.x;
      rl = v.y;
      src = P.W.rec + row * D;
    } else if (j < N) {
      if (P.own_warps) {
        const long long id = ((own0 + j - np) * Q.Hkv + h) * Q.G + gh;
        const float2 v = P.W.own_ml[id];
        rm = v.x;
        rl = v.y;
        src = P.W.own_rec + id * D;
      } else {
        const long long id = slice_rec(own, To, Q.CD, j - np);
        const float* r = Q.rec_det + (id + 2LL * u) * (Q.G * (2 + D)) + gh * (2 + D);
        rm = r[0] * 1.4426950408889634f;  // the gather keeps natural units
        rl = r[1];
        src = r + 2;
      }
    }
    if (rl == 0.0f) rm = -INFINITY;  // no key, or weights of zero alone
    float top = rm;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == -INFINITY) continue;
    const float nm = fmaxf(m, top), f = exp2f(m - nm);
    m = nm;
    const float w = rm == -INFINITY ? 0.0f : exp2f(rm - nm);
    float sum = rl * w;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * f + sum;
#pragma unroll
    for (int i = 0; i < PL; i++) {
      a[i].x *= f;
      a[i].y *= f;
    }
    const int cnt = min(32, mine - j0);
    constexpr int B = 4;  // records whose loads are in flight together (8: slower by 1 to 6 us, fewer warps fit)
    for (int k0 = 0; k0 < cnt; k0 += B) {
      float2 x[B][PL];
      float wk[B];
#pragma unroll
      for (int k = 0; k < B; k++) {
        wk[k] = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
        const float* p = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), (k0 + k) & 31));
#pragma unroll
        for (int i = 0; i < PL; i++)
          x[k][i] = k0 + k < cnt && wk[k] != 0.0f ? reinterpret_cast<const float2*>(p)[lane + 32 * i]
                                                  : make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int k = 0; k < B; k++)
#pragma unroll
        for (int i = 0; i < PL; i++) {
          a[i].x += x[k][i].x * wk[k];
          a[i].y += x[k][i].y * wk[k];
        }
    }
  }
  if constexpr (WR > 1) {
    if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
    for (int i = 0; i < PL; i++) s_acc[warp][i][lane] = a[i];
    __syncthreads();
    if (part != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < WR; w++) top = fmaxf(top, s_ml[warp + w].x);
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; i++) a[i] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < WR; w++) {
      const float f = s_ml[warp + w].x == -INFINITY ? 0.0f : exp2f(s_ml[warp + w].x - top);
      l += s_ml[warp + w].y * f;
#pragma unroll
      for (int i = 0; i < PL; i++) {
        a[i].x += s_acc[warp + w][i][lane].x * f;
        a[i].y += s_acc[warp + w][i][lane].y * f;
      }
    }
  }
  if (!real) return;
#pragma unroll
  for (int i = 0; i < PL; i++) {
    const float2 v = none ? make_float2(0.0f, 0.0f) : make_float2(a[i].x / l, a[i].y / l);
    float* p = out + 2 * (lane + 32 * i);
    if ((reinterpret_cast<uintptr_t>(Q.out) & 7u) == 0) {
      *reinterpret_cast<float2*>(p) = v;
    } else {  // the caller's array may start at any float
      p[0] = v.x;
      p[1] = v.y;
    }
  }
}

}  // namespace vattn
