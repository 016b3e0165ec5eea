// k_shared_prefix_tc: the shared prefix of bf16 caches in device memory on the
// tensor cores (tcgen05), one CTA per SM.
//
// A segment (vattn_shared.cuh) is up to two tiles of 128 query rows against a
// run of 128-key tiles. Its work is a sequence of steps, each S = Q K^T
// (128 x 128 scores), the online softmax of S, and O += P V:
//   two query tiles: step 2j + i is query tile i against key tile j, so a K or
//                    V tile in shared memory serves both;
//   one query tile:  step t is key tile t, into accumulator t % 2; the two
//                    accumulators are merged into one record at the end.
// Steps alternate between two stages (S, O and a softmax warpgroup each), so
// that the tensor cores work on one stage while the other's softmax runs.
//   warps 0-3, 4-7  softmax of stage 0 and 1: thread = row (TMEM lane); they
//                   also clear the V rows behind the prefix's last key, so that
//                   whatever the cache holds there meets its zero weights as
//                   zeros, and write the records
//   warp 8          producer: Q, K and V tiles by TMA, 128-byte swizzle, K and
//                   V through a ring of NST tiles; K and V blocks of `box` rows,
//                   each inside one page
//   warp 9          one thread issues the MMAs. Few of them queue up in the
//                   tensor core, so every cycle between two products of this
//                   thread idles it: no warp-wide step stands there, and the
//                   weights are handed over in two halves of 64 keys
//   warp 10         lets the next kernel start
// TMEM (512 columns): S0, S1, O0, O1 of 128 each. The weights of 32 keys
// overwrite their scores as two bf16 terms (hi = bf16(p), lo = bf16(p - hi),
// 2^-16 relative; 16 columns each), the A operand of two products with V: the
// outputs are fp32, and one term would leave 2^-8. The running maximum moves only
// when a tile exceeds it by more than 2^8 (weights stay below 2^8, far inside
// fp32 and bf16), so O is rarely rescaled; by the time a tile's scores are read, the stage's previous product
// is complete (both are issued in order), so the softmax threads may rescale O.
//
// d = 128, 8 KV heads, 4 query heads each. 32 sequences over 32768 keys (one
// query tile): 134 MB in about 36 us of a 62 us call, bound by HBM (5.5 TB/s
// between the first tile and the records, 3.5 TB/s with them). 256 sequences
// over 8192 keys (two tiles, four blocks per head): 52 GFLOP with both terms in
// about 45 us of a 99 us call, 1.2 PFLOP/s with the tensor pipe active half the
// time: bound by the chain scores, softmax, weights, product of each stage.
// Without the second term's products it takes 3 us less, without the
// exponentials 2 us, so neither bounds it by itself. Two softmax threads per row
// (16 warps) made it 4 us slower.
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
  static constexpr int THREADS = 352;
  static constexpr int GROUPS = 16;                  // groups whose records fit shared memory (below a warp)
  struct Tail {
    uint64_t full[NST], empty[NST], qfull, qfree, s[2], p[2][2], o[2], ofree, done, all;
    unsigned tmem;
    int start[GROUPS + 1], prefix[GROUPS], reach[GROUPS];
    SharedGroup group[GROUPS + 1];
    float2 ml[2][128];
  };
  static constexpr size_t SMEM = static_cast<size_t>(2 + NST) * TILE + sizeof(Tail);
  static_assert(SMEM <= 227 * 1024, "shared memory of the prefix kernel");
};

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// One thread of a converged warp, the same one every time (commits track the
// MMAs of the thread that issues them).
__device__ __forceinline__ bool elect_one() {
  unsigned p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// Shared-memory descriptors of 128-byte-swizzled tiles: the low word holds the
// address and `lead`, the bytes between 64-column blocks of an operand whose
// columns are its M or N side (unused where they are its K side); the high
// word the 1024 bytes between 8-row groups, the version and the swizzle.
__device__ __forceinline__ unsigned tc_desc_lo(unsigned addr, unsigned lead) {
  return ((addr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}
constexpr unsigned kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// D[tmem] (+)= A[smem] B[smem], bf16 operands, fp32 accumulation
__device__ __forceinline__ void tc_mma_ss(unsigned d, unsigned a, unsigned b, unsigned idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(kDescHi)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_ts(unsigned d, unsigned a, unsigned b, unsigned idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.u32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(kDescHi)
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
__device__ __forceinline__ void tc_ld16(unsigned t, unsigned (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
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

// Instruction descriptor: bf16 x bf16 -> fp32, M = 128, A by rows (K-major), B
// by rows (K-major) or, with b_cols, with N contiguous.
__host__ __device__ constexpr unsigned tc_idesc(int n, bool b_cols) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_cols ? 1u << 16 : 0u) | (static_cast<unsigned>(n >> 3) << 17) |
         (static_cast<unsigned>(128 >> 4) << 24);
}

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ float2 unpack_bf16x2(unsigned h) {
  return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
}
// 32 bytes in one store
__device__ __forceinline__ void st_global_v8(float* p, const float (&x)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(p)), "f"(x[0]),
               "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

__device__ __forceinline__ void ld_global_v8(const float* p, float (&x)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(__cvta_generic_to_global(p))
               : "memory");
}
// Scores from column nk on (of 64) become -inf.
__device__ __forceinline__ void mask_tail(unsigned (&x)[2][32], int nk) {
#pragma unroll
  for (int k = 0; k < 2; k++)
#pragma unroll
    for (int j = 0; j < 32; j++)
      if (32 * k + j >= nk) x[k][j] = __float_as_uint(-INFINITY);
}
__device__ __forceinline__ float max64(const unsigned (&x)[2][32]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; i++) m[i] = __uint_as_float(x[0][i]);
#pragma unroll
  for (int j = 4; j < 64; j++) m[j & 3] = fmaxf(m[j & 3], __uint_as_float(x[j / 32][j % 32]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// 16 columns of a record: scaled; plus an accumulator's (or just these).
__device__ __forceinline__ void scale_record(float* p, float f) {
  float x[2][8];
  ld_global_v8(p, x[0]);
  ld_global_v8(p + 8, x[1]);
#pragma unroll
  for (int j = 0; j < 16; j++) x[j / 8][j % 8] *= f;
  st_global_v8(p, x[0]);
  st_global_v8(p + 8, x[1]);
}
__device__ __forceinline__ void add_record(float* p, const unsigned (&o)[16], bool more) {
  float x[2][8] = {};
  if (more) {
    ld_global_v8(p, x[0]);
    ld_global_v8(p + 8, x[1]);
  }
#pragma unroll
  for (int j = 0; j < 16; j++) x[j / 8][j % 8] += __uint_as_float(o[j]);
  st_global_v8(p, x[0]);
  st_global_v8(p + 8, x[1]);
}

// A barrier of several warps with a bounded wait: false if it ran out. `phase`
// counts the warp's passes.
__device__ __forceinline__ bool meet(uint64_t* bar, unsigned& phase) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, phase & 1u));
  phase++;
  return ok;
}

constexpr float kRescale = 8.0f;  // log2 of the weights' bound before the maximum moves
// The tensor core truncates when it adds to an accumulator: 0.8 to 1.7e-8 of the
// output is lost with every product, always towards zero (measured on constant
// and on random values). After kFlush steps a stage adds its accumulator to the
// segment's record in fp32 and starts a new one: the loss stays below 6.5e-6 at
// any length (1.3e-5 over 55 steps without). Each time moves 19 MB to the
// records and takes about 9 us of 62 for the steps between; every 16 steps made
// segments of 55 steps 13% longer, every 8 steps those of 14 steps 10%.
constexpr int kFlush = 24;

template <int D>
__global__ void __launch_bounds__(PrefixTcShape<D>::THREADS, 1)
    k_shared_prefix_tc(const __grid_constant__ SharedParams P) {
  using S = PrefixTcShape<D>;
  constexpr int H = S::H, HALF = S::HALF, TILE = S::TILE, NST = S::NST, KT = S::KT;
  extern __shared__ __align__(1024) unsigned char s_tiles[];  // the swizzle's pattern repeats every 1024 bytes
  unsigned char* s_q = s_tiles;
  unsigned char* s_ring = s_tiles + 2 * TILE;
  typename S::Tail& tail = *reinterpret_cast<typename S::Tail*>(s_tiles + (2 + NST) * TILE);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; i++) {
      mbar_init(&tail.full[i], 1);
      mbar_init(&tail.empty[i], 1);
    }
    mbar_init(&tail.qfull, 1);
    mbar_init(&tail.qfree, 1);
    mbar_init(&tail.ofree, 8);
    mbar_init(&tail.all, 8);
    mbar_init(&tail.done, 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(&tail.s[i], 1);
      mbar_init(&tail.p[i][0], 4);
      mbar_init(&tail.p[i][1], 4);
      mbar_init(&tail.o[i], 1);
    }
    mbar_init_fence();
  }
  if (warp == 8 && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &P.tmk_t : lane == 1 ? &P.tmv_t : &P.tmq) : "memory");
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tail.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  // The groups' records. With few groups every CTA finds them itself, from what
  // the caller gave, and starts while k_shared_prep runs (which lets this kernel
  // start once everything before the call has ended): that takes its 4 us out of
  // the way. It needs nothing else of k_shared_prep: for pages that are out of
  // range it reads others, and k_shared_combine does not read the records.
  const bool cached = P.groups <= S::GROUPS;
  if (cached) {
    const int mine = threadIdx.x < P.D.batch ? checked_len(P, threadIdx.x) : -1;
    if (threadIdx.x <= P.groups) tail.start[threadIdx.x] = __ldcg(P.group_start + threadIdx.x);
    if (threadIdx.x < P.groups) {
      tail.prefix[threadIdx.x] = __ldcg(P.prefix_lens + threadIdx.x);
      tail.reach[threadIdx.x] = 0;
    }
    __syncthreads();
    bool bad = tail.start[0] != 0 || tail.start[P.groups] != P.D.batch;
    for (int g = 0; g < P.groups; g++) bad |= tail.start[g + 1] < tail.start[g];
    for (int b = threadIdx.x; b < P.D.batch && !bad; b += S::THREADS) {
      const int n = b < S::THREADS ? mine : checked_len(P, b);
      int g = 0;
      while (tail.start[g + 1] <= b) g++;
      const int prefix = tail.prefix[g];
      if (prefix <= 0 || prefix > P.D.max_ctx) continue;
      const int add = n >= prefix ? 1 : b == tail.start[g] ? kFirstShort : 0;
      if (add) atomicAdd(&tail.reach[g], add);
    }
    __syncthreads();
    if (warp == 0) {  // lane g: group g; lane `groups`: the totals
      SharedGroup r = {};
      long long tiles = 0, rows = 0;
      if (lane < P.groups) {
        r.b0 = tail.start[lane];
        r.size = tail.start[lane + 1] - r.b0;
        r.prefix = tail.prefix[lane];
        if (!bad && is_shared(P, tail.reach[lane])) group_work(P, r, tiles, rows);
      }
      long long it = tiles, ir = rows;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, it, o), y = __shfl_up_sync(0xffffffffu, ir, o);
        if (lane >= o) {
          it += x;
          ir += y;
        }
      }
      r.tile0 = it - tiles;
      r.row0 = ir - rows;
      if (lane <= P.groups) tail.group[lane] = r;
    }
  } else {
    grid_dependency_wait();
  }
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = tail.tmem;
  const SharedGroup* group = cached ? tail.group : P.W.group;
  const long long Tt = group[P.groups].tile0;
  const long long beg = div_nonneg(Tt * blockIdx.x, gridDim.x), end = div_nonneg(Tt * (blockIdx.x + 1), gridDim.x);
  int gi = group_at(P, group, beg);
  bool ok = true;

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    const int box = P.box, per = KT / box * H;  // copies of a whole tile: one per lane
    const int blk = lane / H, hf = lane % H;
    unsigned li = 0;
    int seg = 0;
    for (long long cur = beg; cur < end && ok;) {
      const Segment s = segment_at(P, group, cur, end, gi);
      gi = s.gi;
      cur = s.next;
      const int tiles_q = s.rows > 128 ? 2 : 1;
      // first row of this lane's block of key tile t (-1: behind the prefix)
      const int* pages = P.D.page_table + static_cast<size_t>(s.b0) * P.D.pps;
      auto row_of = [&](int t) -> int {
        const int pos = t * KT + blk * box;
        if (t >= s.t1 || lane >= per || pos >= s.prefix) return -1;
        const int slot = page_slot(P.D, pos);
        int page = __ldcg(pages + slot);
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(P.D.num_pages)) page = 0;  // reported by k_shared_prep
        return (page * P.D.Hkv + s.h) * P.D.ps + (pos - slot * P.D.ps);
      };
      int row = row_of(s.t0);
      for (int t = s.t0; t < s.t1 && ok; t++) {
        const int next = row_of(t + 1);
        const int nblk = min(KT / box, (s.prefix - t * KT + box - 1) / box);
        for (int kv = 0; kv < 2; kv++, li++) {
          const unsigned st = li % NST;
          if (li >= NST) ok = __all_sync(0xffffffffu, mbar_wait(&tail.empty[st], (li / NST - 1) & 1u));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&tail.full[st], static_cast<unsigned>(nblk * box * D * 2));
          __syncwarp();
          if (row >= 0)
            tma_2d(s_ring + st * TILE + hf * HALF + blk * box * 128, kv ? &P.tmv_t : &P.tmk_t, hf * 64, row,
                   &tail.full[st]);
        }
        row = next;
        if (t == s.t0 && ok) {
          // the queries, once the segment before has computed its last scores
          if (seg > 0) ok = __all_sync(0xffffffffu, mbar_wait(&tail.qfree, (seg - 1) & 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&tail.qfull, static_cast<unsigned>(tiles_q * TILE));
          __syncwarp();
          const int qt = lane / H;
          if (qt < tiles_q)
            tma_3d(s_q + qt * TILE + hf * HALF, &P.tmq, hf * 64, s.h * P.D.G,
                   s.b0 + s.row0 / P.D.G + qt * (128 / P.D.G), &tail.qfull);
          seg++;
        }
      }
    }
    // no copy may land after the CTA has moved on (only after a failed wait are some still in flight)
    if (!ok) {
      for (unsigned i = li > NST ? li - NST : 0; i < li; i++) mbar_wait(&tail.full[i % NST], (i / NST) & 1u);
      if (seg > 0) mbar_wait(&tail.qfull, (seg - 1) & 1);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMAs, one thread
    if (elect_one()) {
      constexpr unsigned kQK = tc_idesc(KT, false), kPV = tc_idesc(D, true);
      const unsigned q_d = tc_desc_lo(smem_u32(s_q), 16), k_d = tc_desc_lo(smem_u32(s_ring), 16),
                     v_d = tc_desc_lo(smem_u32(s_ring), H > 1 ? HALF : 1024);
      unsigned li0 = 0, np[2] = {0, 0};
      int seg = 0;
      for (long long cur = beg; cur < end && ok;) {
        const Segment s = segment_at(P, group, cur, end, gi);
        gi = s.gi;
        cur = s.next;
        const bool two = s.rows > 128;
        const int nt = s.t1 - s.t0, n = two ? 2 * nt : nt;
        auto qk = [&](int i) {
          const int st = i & 1, kt = two ? i >> 1 : i;
          const unsigned idx = li0 + 2u * kt, slot = idx % NST;
          if (!two || st == 0) ok = ok && mbar_wait(&tail.full[slot], (idx / NST) & 1u);
          if (!ok) return;
          tc_fence_after();
          const unsigned a = q_d + (two ? st * (TILE >> 4) : 0), b = k_d + slot * (TILE >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; k++) {
            const unsigned off = ((k / 4) * HALF + (k % 4) * 32) >> 4;
            tc_mma_ss(tmem + st * 128, a + off, b + off, kQK, k > 0);
          }
          tc_commit(&tail.s[st]);
          if (!two || st == 1) tc_commit(&tail.empty[slot]);
        };
        auto pv = [&](int i) {
          const int st = i & 1, kt = two ? i >> 1 : i;
          const unsigned idx = li0 + 2u * kt + 1u, slot = idx % NST;
          const bool first = (i >> 1) % kFlush == 0;  // a new accumulator
          if (!two || st == 0) ok = ok && mbar_wait(&tail.full[slot], (idx / NST) & 1u);
          // the accumulators of the segment before have been read
          if (i == 0 && seg > 0) ok = ok && mbar_wait(&tail.ofree, (seg - 1) & 1);
          const unsigned b = v_d + slot * (TILE >> 4), p = tmem + st * 128, o = tmem + 256 + st * 128;
#pragma unroll
          for (int half = 0; half < 2; half++) {
            ok = ok && mbar_wait(&tail.p[st][half], np[st] & 1u);
            if (!ok) return;
            tc_fence_after();
#pragma unroll
            for (int term = 0; term < 2; term++)
#pragma unroll
              for (int k = 4 * half; k < 4 * half + 4; k++)
                tc_mma_ts(o, p + 32 * (k / 2) + 16 * term + 8 * (k % 2), b + (k * 2048 >> 4), kPV, k + term > 0 || !first);
          }
          np[st]++;
          if (!two || st == 1) tc_commit(&tail.empty[slot]);
          if (i + 2 >= n) tc_commit(&tail.o[st]);  // the stage's last step
        };
        ok = mbar_wait(&tail.qfull, seg & 1);
        if (!ok) break;
        qk(0);
        if (n > 1) qk(1);
        if (n <= 2 && ok) tc_commit(&tail.qfree);
        for (int i = 0; i < n && ok; i++) {
          pv(i);
          if (i + 2 < n && ok) qk(i + 2);
          if (i + 3 == n && ok) tc_commit(&tail.qfree);  // the segment's last scores
        }
        seg++;
        li0 += 2u * nt;
      }
      // every MMA and every arrival of a commit is complete before the CTA ends
      tc_commit(&tail.done);
      ok = mbar_wait(&tail.done, 0) && ok;
      if (!ok) atomicOr(P.D.err, kDevTimeout);
    }
    __syncwarp();
  } else if (warp == 10) {
    // k_shared_own may start once k_shared_prep has ended; it takes each SM as
    // this kernel leaves it
    grid_dependency_wait();
    grid_dependents_launch();
  } else {
    // ------------------------------------------------------------ softmax
    const int st = warp >> 2, quarter = warp & 3;
    const unsigned lanes = static_cast<unsigned>(quarter * 32) << 16;
    const unsigned sa = tmem + st * 128 + lanes, oa = tmem + 256 + lanes;
    const float c = P.D.scale * 1.4426950408889634f;  // scores in log2 units
    const int r = quarter * 32 + lane;                // row of the query tile
    unsigned ns = 0, no[2] = {0, 0}, li0 = 0, alls = 0;
    for (long long cur = beg; cur < end && ok;) {
      const Segment s = segment_at(P, group, cur, end, gi);
      gi = s.gi;
      cur = s.next;
      const bool two = s.rows > 128;
      const int nt = s.t1 - s.t0, steps = two ? nt : (nt + 1 - st) / 2;
      const int valid = two ? s.rows - st * 128 : s.rows;  // query rows of the stage's tile
      const bool idle = quarter * 32 >= valid;             // none in this warp
      // the stage's record row (with one query tile, stage 1's is scratch behind
      // the records, within the rows that are the CTA's at this point)
      const int behind = two ? 128 : s.rows;
      float* mine = P.W.rec + (s.rec + st * behind + r) * D;
      float m = -INFINITY, l = 0.0f;
      // Before its first scores can be there, a warp runs a step on whatever its
      // TMEM holds, without storing, waiting or signalling: the instructions are
      // then in the SM's cache when the scores arrive (they are several KB, and
      // came from L2 at the first tile's expense).
      for (int i = ns == 0 ? -1 : 0; i < steps && ok; i++) {
        const bool real = i >= 0;
        const int kt = two ? i : 2 * i + st;
        const int nk = real ? s.prefix - (s.t0 + kt) * KT : KT;
        if (real) {
          ok = __all_sync(0xffffffffu, mbar_wait(&tail.s[st], ns & 1u));
          ns++;
          if (!ok) break;
        }
        if (nk < KT && (!two || st == 0)) {
          // the V rows behind the prefix's last key: zero, whatever the cache holds.
          // (The tile's scores are there, so every earlier use of V's ring tile is
          // over and its barrier is in the phase waited for, or past it.)
          const unsigned idx = li0 + 2u * kt + 1u, slot = idx % NST;
          ok = __all_sync(0xffffffffu, mbar_wait(&tail.full[slot], (idx / NST) & 1u));
          if (!ok) break;
          for (int x = nk * 8 + r; x < KT * 8; x += 128)
#pragma unroll
            for (int hf = 0; hf < H; hf++)
              *reinterpret_cast<uint4*>(s_ring + slot * TILE + hf * HALF + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async();
        }
        tc_fence_after();
        // the row's 128 scores in four chunks of 32: the maximum over all; the
        // first two stay in registers, the others are read again (their weights
        // replace each chunk in place)
        unsigned x[2][32];
        float neg = 0.0f;
        if (!idle) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 1; k >= 0; k--) {
            tc_ld32(sa + 64 * k, x[0]);
            tc_ld32(sa + 64 * k + 32, x[1]);
            tc_wait_ld();
            if (nk < KT) mask_tail(x, nk - 64 * k);
            top = fmaxf(top, max64(x));
          }
          top *= c;
          if (i <= 0) {
            m = fmaxf(top, kLowest);
          } else if (__any_sync(0xffffffffu, top > m + kRescale)) {
            const float mn = top > m + kRescale ? top : m;
            const float f = ex2(m - mn);
            m = mn;
            l *= f;
#pragma unroll 1
            for (int k = 0; k < D / 16; k++) {
              unsigned o[16];
              tc_ld16(oa + st * 128 + 16 * k, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tc_st16(oa + st * 128 + 16 * k, o);
              if (i > kFlush && r < valid) scale_record(mine + 16 * k, f);
            }
          }
          if (i > 0 && i % kFlush == 0) {
            tc_wait_st();
#pragma unroll 1
            for (int k = 0; k < D / 16; k++) {
              unsigned o[16];
              tc_ld16(oa + st * 128 + 16 * k, o);
              tc_wait_ld();
              if (r < valid) add_record(mine + 16 * k, o, i > kFlush);
            }
          }
          neg = -m;
        }
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int half = 0; half < 2; half++) {
          if (!idle) {
            if (half == 1) {
              tc_wait_ld();
              if (nk < KT) mask_tail(x, nk - 64);
            }
#pragma unroll
            for (int k = 0; k < 2; k++) {
              unsigned w[32];  // hi terms, then lo terms
#pragma unroll
              for (int j = 0; j < 16; j++) {
                // (product and difference rounded apart, as the maximum's product is: fused, scores of
                // 2^31 and more would leave their own maximum by more than fp32's range of exponents)
                const float2 y = __fadd2_rn(
                    __fmul2_rn(make_float2(__uint_as_float(x[k][2 * j]), __uint_as_float(x[k][2 * j + 1])), make_float2(c, c)),
                    make_float2(neg, neg));
                const float2 p = make_float2(ex2(y.x), ex2(y.y));
                sum = __fadd2_rn(sum, p);
                w[j] = pack_bf16x2(p.x, p.y);
                const float2 h = unpack_bf16x2(w[j]);
                const float2 d = __fadd2_rn(p, make_float2(-h.x, -h.y));
                w[16 + j] = pack_bf16x2(d.x, d.y);
              }
              if (real) tc_st32(sa + 64 * half + 32 * k, w);
              if (half == 0) tc_ld32(sa + 64 + 32 * k, x[k]);
            }
            tc_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (real && lane == 0) mbar_arrive(&tail.p[st][half]);
        }
        l = i <= 0 ? sum.x + sum.y : l + (sum.x + sum.y);
      }
      li0 += 2u * nt;
      if (!ok) break;
      // records. Two query tiles: each stage its own. One: the two stages'
      // accumulators merged, every warpgroup one half of the columns
      const bool merge = !two && nt > 1;
      float f0 = 1.0f, f1 = 0.0f;
      if (merge) {
        tail.ml[st][r] = make_float2(m, l);
        ok = meet(&tail.all, alls);
        const float2 a = tail.ml[0][r], b = tail.ml[1][r];
        m = fmaxf(a.x, b.x);
        f0 = ex2(a.x - m);
        f1 = ex2(b.x - m);
        l = a.y * f0 + b.y * f1;
        ok = meet(&tail.all, alls) && ok;  // before the next segment's write
        if (!ok) break;
      }
      const bool has = two || merge || st == 0;  // columns to write
      const int s0 = two ? st : 0;               // the (first) accumulator
      const int steps0 = two ? nt : (nt + 1) / 2, steps1 = nt / 2;  // of it, and of the second in a merge
      // (a stage without a step waits too: it would run ahead otherwise, and
      // arrive at `ofree` for segments whose accumulators are still being read)
      ok = __all_sync(0xffffffffu, mbar_wait(&tail.o[s0], no[s0] & 1u));
      if (merge && ok) ok = __all_sync(0xffffffffu, mbar_wait(&tail.o[1], no[1] & 1u));
      no[0]++;
      if (two || merge) no[1]++;
      if (!ok) break;
      tc_fence_after();
      const long long row = s.rec + (two ? st * 128 : 0) + r;
      if (!idle && has) {
        const int c0 = merge ? st * (D / 2) : 0, c1 = merge ? c0 + D / 2 : D;
#pragma unroll 1
        for (int k = c0; k < c1; k += 16) {
          unsigned a[16], b[16];
          tc_ld16(oa + s0 * 128 + k, a);
          if (merge) tc_ld16(oa + 128 + k, b);
          tc_wait_ld();
          if (r < valid) {
            float* rec = P.W.rec + row * D + k;
            float o[2][8] = {}, e[2][8] = {};
            // (written by this row's thread of either stage, before their merge)
            if (steps0 > kFlush) {
              ld_global_v8(rec, o[0]);
              ld_global_v8(rec + 8, o[1]);
            }
            if (merge && steps1 > kFlush) {
              ld_global_v8(rec + behind * D, e[0]);
              ld_global_v8(rec + behind * D + 8, e[1]);
            }
#pragma unroll
            for (int j = 0; j < 16; j++) {
              float& x = o[j / 8][j % 8];
              x += __uint_as_float(a[j]);
              if (merge) x = x * f0 + (e[j / 8][j % 8] + __uint_as_float(b[j])) * f1;
            }
            st_global_v8(rec, o[0]);
            st_global_v8(rec + 8, o[1]);
          }
        }
        if (r < valid && (two || st == 0)) P.W.ml[row] = make_float2(m, l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail.ofree);
    }
  }
  if (!ok && lane == 0 && warp < 9) atomicOr(P.D.err, kDevTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace vattn
