// k_shared_prefix_tc: the shared prefix of bf16 caches in device memory on the
// tensor cores (tcgen05), one CTA per SM.
//
// A segment (vattn_shared.cuh) is up to two tiles of 128 query rows against a
// run of 128-key tiles. Its work is a sequence of steps, each S = Q K^T
// (128 x 128 scores), the online softmax of S, and O += P V:
//   two query tiles: step 2j + i is query tile i against key tile j, so a K or
//                    V tile in shared memory serves both;
//   one query tile:  step t is key tile t, into accumulator t % 2; the two
//                    accumulators leave two records per row.
// Steps alternate between two stages (S, O and a softmax warpgroup each), so
// that the tensor cores work on one stage while the other's softmax runs.
//   warps 0-3, 4-7  softmax of stage 0 and 1: thread = row (TMEM lane)
//   warp 8          producer: Q, K and V tiles by TMA, 128-byte swizzle, K and
//                   V through a ring of NST tiles; K and V blocks of `box` rows,
//                   each inside one page
//   warp 9          issues the MMAs (one thread) and clears the V rows behind
//                   the prefix's last key, so that whatever the cache holds
//                   there meets its zero weights as zeros
// TMEM (512 columns): S0, S1, O0, O1 of 128 each. The weights overwrite their
// scores as two bf16 terms (hi = bf16(p), lo = bf16(p - hi), 2^-17 relative),
// the A operand of two products with V: fp32 outputs keep fp32's accuracy from
// bf16 products. The running maximum moves only when a tile exceeds it by more
// than 2^8 (weights stay below 2^8, far inside fp32 and bf16), so O is rarely
// rescaled; by the time a tile's scores are read, the stage's previous product
// is complete (both are issued in order), so the softmax threads may rescale O.
#pragma once

#include "vattn_ctx.h"
#include "vattn_kernels.cuh"

namespace vattn {

template <int D>
struct PrefixTcShape {
  static constexpr int M = 128, KT = 128, H = D / 64;
  static constexpr int HALF = 128 * 128;             // bytes of 128 rows of a 64-column half
  static constexpr int TILE = H * HALF;              // a Q, K or V tile
  static constexpr int NST = 160 * 1024 / TILE;      // ring tiles
  static constexpr int THREADS = 320;
  static constexpr size_t SMEM = 1024 + static_cast<size_t>(2 + NST) * TILE;
  static_assert(SMEM <= 226 * 1024, "shared memory of the prefix kernel");
};

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// D[tmem] (+)= A[smem] B[smem], bf16 operands, fp32 accumulation
__device__ __forceinline__ void tc_mma_ss(unsigned d, uint64_t a, uint64_t b, unsigned idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_ts(unsigned d, unsigned a, uint64_t b, unsigned idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// this warp's 32 lanes x 32 columns from `t`: one row's columns per thread
__device__ __forceinline__ void tc_ld32(unsigned t, unsigned (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tc_st32(unsigned t, const unsigned (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_st16(unsigned t, const unsigned (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory descriptor of a 128-byte-swizzled tile: 8-row groups 1024 bytes
// apart; `lead`: bytes between 64-column blocks of an operand whose columns are
// its M or N side (unused where they are its K side).
__device__ __forceinline__ uint64_t tc_desc(unsigned addr, unsigned lead) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// Instruction descriptor: bf16 x bf16 -> fp32, M = 128, A by rows (K-major), B
// by rows (K-major) or, with b_cols, with N contiguous.
__host__ __device__ constexpr unsigned tc_idesc(int n, bool b_cols) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_cols ? 1u << 16 : 0u) | (static_cast<unsigned>(n >> 3) << 17) |
         (static_cast<unsigned>(128 >> 4) << 24);
}

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Steps of stage `st` in a segment.
__device__ __forceinline__ int stage_steps(bool two, int nt, int st) { return two ? nt : (nt + 1 - st) / 2; }

constexpr float kRescale = 8.0f;  // log2 of the weights' bound before the maximum moves

template <int D>
__global__ void __launch_bounds__(PrefixTcShape<D>::THREADS, 1)
    k_shared_prefix_tc(const __grid_constant__ SharedParams P) {
  using S = PrefixTcShape<D>;
  constexpr int H = S::H, HALF = S::HALF, TILE = S::TILE, NST = S::NST, KT = S::KT;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* s_q = smem;
  unsigned char* s_ring = smem + 2 * TILE;
  __shared__ __align__(8) uint64_t b_full[NST], b_empty[NST], b_qfull, b_qfree, b_s[2], b_p[2], b_o[2], b_ofree[2],
      b_done;
  __shared__ unsigned s_tmem;
  __shared__ int s_g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; i++) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    mbar_init(&b_qfull, 1);
    mbar_init(&b_qfree, 1);
    mbar_init(&b_done, 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(&b_s[i], 1);
      mbar_init(&b_p[i], 4);
      mbar_init(&b_o[i], 1);
      mbar_init(&b_ofree[i], 4);
    }
    s_g = 0;
    mbar_init_fence();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = s_tmem;
  grid_dependency_wait();

  const long long Tt = P.W.tiles[P.groups];
  const long long beg = div_nonneg(Tt * blockIdx.x, gridDim.x), end = div_nonneg(Tt * (blockIdx.x + 1), gridDim.x);
  const int gi0 = beg < end ? first_group(P, beg, &s_g) : 0;
  bool ok = true;

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    const int box = P.box, per = KT / box * H;  // copies of a whole tile: one per lane
    const int blk = lane / H, hf = lane % H;
    unsigned li = 0;
    int seg = 0;
    int gi = gi0;
    for (long long cur = beg; cur < end && ok;) {
      const Segment s = segment_at(P, cur, end, gi);
      gi = s.gi;
      cur = s.next;
      if (!P.W.pages_ok[s.gi]) continue;
      const bool two = s.rows > 128;
      // page of this lane's block of key tile t (position behind the prefix: no block)
      const int* pages = P.D.page_table + static_cast<size_t>(s.g.b0) * P.D.pps;
      auto row_of = [&](int t) -> int {
        const int pos = t * KT + blk * box;
        if (t >= s.t1 || lane >= per || pos >= s.g.prefix) return -1;
        const int slot = page_slot(P.D, pos);
        return (pages[slot] * P.D.Hkv + s.h) * P.D.ps + (pos - slot * P.D.ps);
      };
      int row = row_of(s.t0);
      if (seg > 0) ok = __all_sync(0xffffffffu, mbar_wait(&b_qfree, (seg - 1) & 1));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&b_qfull, static_cast<unsigned>((two ? 2 : 1) * TILE));
        const int b0 = s.g.b0 + s.row0 / P.D.G;
        for (int t = 0; t < (two ? 2 : 1); t++)
          for (int x = 0; x < H; x++)
            tma_3d(s_q + t * TILE + x * HALF, &P.tmq, x * 64, s.h * P.D.G, b0 + t * (128 / P.D.G), &b_qfull);
      }
      seg++;
      for (int t = s.t0; t < s.t1 && ok; t++) {
        const int next = row_of(t + 1);
        const int nblk = min(KT / box, (s.g.prefix - t * KT + box - 1) / box);
        for (int kv = 0; kv < 2; kv++, li++) {
          const unsigned st = li % NST;
          if (li >= NST) ok = __all_sync(0xffffffffu, mbar_wait(&b_empty[st], (li / NST - 1) & 1u));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&b_full[st], static_cast<unsigned>(nblk * box * D * 2));
          __syncwarp();
          if (row >= 0)
            tma_2d(s_ring + st * TILE + hf * HALF + blk * box * 128, kv ? &P.tmv_t : &P.tmk_t, hf * 64, row,
                   &b_full[st]);
        }
        row = next;
      }
    }
    // no copy may land after the CTA has moved on (only after a failed wait are some still in flight)
    if (!ok)
      for (unsigned i = li > NST ? li - NST : 0; i < li; i++) mbar_wait(&b_full[i % NST], (i / NST) & 1u);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMAs
    constexpr unsigned kQK = tc_idesc(KT, false), kPV = tc_idesc(D, true);
    const unsigned q_a = smem_u32(s_q), r_a = smem_u32(s_ring);
    unsigned li0 = 0, np[2] = {0, 0}, no[2] = {0, 0};
    int seg = 0, gi = gi0;
    for (long long cur = beg; cur < end && ok;) {
      const Segment s = segment_at(P, cur, end, gi);
      gi = s.gi;
      cur = s.next;
      if (!P.W.pages_ok[s.gi]) continue;
      const bool two = s.rows > 128;
      const int nt = s.t1 - s.t0, n = two ? 2 * nt : nt;
      auto qk = [&](int i) {
        const int st = i & 1, kt = two ? i >> 1 : i;
        const unsigned idx = li0 + 2u * kt, slot = idx % NST;
        if (!two || st == 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&b_full[slot], (idx / NST) & 1u));
        if (!ok) return;
        tc_fence_after();
        if (lane == 0) {
          const unsigned a = q_a + (two ? st * TILE : 0), b = r_a + slot * TILE;
#pragma unroll
          for (int k = 0; k < D / 16; k++) {
            const unsigned off = (k / 4) * HALF + (k % 4) * 32;
            tc_mma_ss(tmem + st * 128, tc_desc(a + off, 16), tc_desc(b + off, 16), kQK, k > 0);
          }
          tc_commit(&b_s[st]);
          if (!two || st == 1) tc_commit(&b_empty[slot]);
        }
        __syncwarp();
      };
      auto pv = [&](int i) {
        const int st = i & 1, kt = two ? i >> 1 : i;
        const unsigned idx = li0 + 2u * kt + 1u, slot = idx % NST;
        const bool first = two ? i < 2 : i == st;  // the stage's first step of the segment
        const bool last = two ? i >= n - 2 : i + 2 >= n;
        if (!two || st == 0) {
          ok = ok && __all_sync(0xffffffffu, mbar_wait(&b_full[slot], (idx / NST) & 1u));
          if (!ok) return;
          const int nk = s.g.prefix - (s.t0 + kt) * KT;
          if (nk < KT) {
            for (int x = nk * 8 + lane; x < KT * 8; x += 32)
#pragma unroll
              for (int hf = 0; hf < H; hf++)
                *reinterpret_cast<uint4*>(s_ring + slot * TILE + hf * HALF + x * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async();
            __syncwarp();
          }
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&b_p[st], np[st] & 1u));
        np[st]++;
        if (first && no[st] > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&b_ofree[st], (no[st] - 1) & 1u));
        if (!ok) return;
        tc_fence_after();
        if (lane == 0) {
          const unsigned b = r_a + slot * TILE, p = tmem + st * 128, o = tmem + 256 + st * 128;
#pragma unroll
          for (int term = 0; term < 2; term++)
#pragma unroll
            for (int k = 0; k < KT / 16; k++)
              tc_mma_ts(o, p + term * 64 + k * 8, tc_desc(b + k * 2048, H > 1 ? HALF : 1024), kPV, !(first && term == 0 && k == 0));
          if (!two || st == 1) tc_commit(&b_empty[slot]);
          if (last) tc_commit(&b_o[st]);
        }
        __syncwarp();
        if (last) no[st]++;
      };
      ok = __all_sync(0xffffffffu, mbar_wait(&b_qfull, seg & 1));
      seg++;
      if (!ok) break;
      qk(0);
      if (n > 1) qk(1);
      for (int i = 0; i < n && ok; i++) {
        pv(i);
        if (i + 2 < n) qk(i + 2);
        // the queries are free once the segment's last scores are computed
        if (i == max(n - 3, 0) && ok && lane == 0) tc_commit(&b_qfree);
      }
      li0 += 2u * nt;
    }
    // every MMA and every arrival of a commit is complete before the CTA ends
    if (lane == 0) tc_commit(&b_done);
    __syncwarp();
    ok = __all_sync(0xffffffffu, mbar_wait(&b_done, 0)) && ok;
  } else {
    // ------------------------------------------------------------ softmax
    const int st = warp >> 2, quarter = warp & 3;
    const unsigned sa = tmem + st * 128 + (static_cast<unsigned>(quarter * 32) << 16);
    const unsigned oa = sa + 256;
    const float c = P.D.scale * 1.4426950408889634f;  // scores in log2 units
    unsigned ns = 0, no = 0;
    int gi = gi0;
    for (long long cur = beg; cur < end && ok;) {
      const Segment s = segment_at(P, cur, end, gi);
      gi = s.gi;
      cur = s.next;
      if (!P.W.pages_ok[s.gi]) continue;
      const bool two = s.rows > 128;
      const int steps = stage_steps(two, s.t1 - s.t0, st);
      const int r = quarter * 32 + lane;                     // row of the query tile
      const int valid = two ? s.rows - st * 128 : s.rows;    // its query rows
      const bool idle = quarter * 32 >= valid;               // no query row in this warp
      const long long row = s.rec + (two ? st * 128 : st * s.rows) + r;
      float m = -INFINITY, l = 0.0f;
      for (int i = 0; i < steps && ok; i++) {
        ok = __all_sync(0xffffffffu, mbar_wait(&b_s[st], ns & 1u));
        ns++;
        if (!ok) break;
        tc_fence_after();
        if (!idle) {
          unsigned x[4][32];
#pragma unroll
          for (int k = 0; k < 4; k++) tc_ld32(sa + 32 * k, x[k]);
          tc_wait_ld();
          const int nk = s.g.prefix - (two ? s.t0 + i : s.t0 + 2 * i + st) * KT;
          if (nk < KT) {
#pragma unroll
            for (int k = 0; k < 4; k++)
#pragma unroll
              for (int j = 0; j < 32; j++)
                if (32 * k + j >= nk) x[k][j] = __float_as_uint(-INFINITY);
          }
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            mx[k] = __uint_as_float(x[k][0]);
#pragma unroll
            for (int j = 1; j < 32; j++) mx[k] = fmaxf(mx[k], __uint_as_float(x[k][j]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          if (i == 0) {
            m = fmaxf(top, -1e30f);  // finite: scores of -inf weigh exactly 0
          } else if (__any_sync(0xffffffffu, top > m + kRescale)) {
            const float mn = top > m + kRescale ? top : m;
            const float f = ex2(m - mn);
            m = mn;
            l *= f;
#pragma unroll 1
            for (int k = 0; k < D / 32; k++) {
              unsigned o[32];
              tc_ld32(oa + 32 * k, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tc_st32(oa + 32 * k, o);
            }
          }
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < 4; k++) {
            unsigned hi[16], lo[16];
#pragma unroll
            for (int j = 0; j < 16; j++) {
              const float p0 = ex2(fmaf(__uint_as_float(x[k][2 * j]), c, -m));
              const float p1 = ex2(fmaf(__uint_as_float(x[k][2 * j + 1]), c, -m));
              sum[j & 3] += p0 + p1;
              hi[j] = pack_bf16x2(p0, p1);
              lo[j] = pack_bf16x2(p0 - __uint_as_float(hi[j] << 16), p1 - __uint_as_float(hi[j] & 0xFFFF0000u));
            }
            tc_st16(sa + 16 * k, hi);
            tc_st16(sa + 64 + 16 * k, lo);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tc_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_p[st]);
      }
      if (!ok) break;
      if (r < valid) P.W.ml[row] = make_float2(m, l);
      if (steps == 0) continue;
      ok = __all_sync(0xffffffffu, mbar_wait(&b_o[st], no & 1u));
      no++;
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
#pragma unroll 1
        for (int k = 0; k < D / 32; k++) {
          unsigned o[32];
          tc_ld32(oa + 32 * k, o);
          tc_wait_ld();
          if (r < valid) {
            float4* dst = reinterpret_cast<float4*>(P.W.rec + row * D + 32 * k);
#pragma unroll
            for (int j = 0; j < 8; j++)
              dst[j] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                   __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b_ofree[st]);
    }
  }
  if (!ok && lane == 0) atomicOr(P.D.err, kDevTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependents_launch();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace vattn
