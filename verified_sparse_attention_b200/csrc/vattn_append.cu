// Rotary positions and appending to the cache (vattn_rope_init, vattn_rotate,
// vattn_append).
//
// Both kernels stream rows of d components: every thread owns one chunk pair
// (2 x 16 bytes) of a token's heads and walks over some of the heads, kUnroll
// rows at a time. A block computes the cosines and sines of its tokens once,
// while its first rows are in flight (each thread for itself: 28.0 us instead of
// 26.0 for 8192 tokens x 32 heads, d = 128, bf16). Bound by HBM for prompts
// (8192 x 32 heads: 134 MB, 5.2 TB/s; 12001 tokens of 32 + 8 + 8 heads appended:
// 295 MB in 54 us, 5.5 TB/s) and by the launch for single tokens (3 us).
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "vattn_ctx.h"

namespace {

using vattn::aligned16;
using vattn::aligned_to;
using vattn::Elem;

constexpr int kThreads = 256;
constexpr int kMaxTok = 64;   // tokens of a block at most
constexpr int kMaxTokens = 1 << 30, kMaxHeads = 1 << 16;  // of a call
constexpr int kRank = 32;     // components of a projected key (Loki)
constexpr unsigned kDevBadSeqlen = VATTN_DEV_BAD_SEQLEN, kDevBadPage = VATTN_DEV_BAD_PAGE;

__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cos and sin of pair i at position pos: the position times the pair's turns
// wraps modulo one turn in 64-bit integers; the nearest quarter turn is taken
// out of the upper 32 bits exactly, and the rest, within an eighth of a turn
// (2^-32 of a turn exact, 2^-25 relative as fp32), goes through sincospif.
__device__ __forceinline__ void pair_turn(const vattn_rope& R, int i, int pos, bool transpose, float& c, float& s) {
  const unsigned t =
      static_cast<unsigned>((R.turns[i] * static_cast<unsigned long long>(static_cast<long long>(pos))) >> 32);
  const unsigned quarter = (t + 0x20000000u) >> 30;
  const int rest = static_cast<int>(t - (quarter << 30));
  float sr, cr;
  sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &sr, &cr);  // 2^-31: half turns
  s = (quarter & 1u) ? cr : sr;
  c = (quarter & 1u) ? sr : cr;
  if (quarter & 2u) s = -s;
  if ((quarter + 1u) & 2u) c = -c;
  if (transpose) s = -s;
  c *= R.amplitude;
  s *= R.amplitude;
}

// E elements as one load and store (16 bytes, or a single element).
template <typename T, int E>
struct Chunk {
  uint4 raw;
  __device__ __forceinline__ void load(const T* p) { raw = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = raw; }
  // into shared memory: 16-byte or 4-byte aligned
  template <bool ALIGNED>
  __device__ __forceinline__ void put(T* p) const {
    if constexpr (ALIGNED) {
      *reinterpret_cast<uint4*>(p) = raw;
    } else {
      unsigned* q = reinterpret_cast<unsigned*>(p);
      q[0] = raw.x;
      q[1] = raw.y;
      q[2] = raw.z;
      q[3] = raw.w;
    }
  }
  __device__ __forceinline__ void get(float (&x)[E]) const { Elem<T>::unpack(raw, x); }
  __device__ __forceinline__ void set(const float (&x)[E]) {
    if constexpr (sizeof(T) == 4) {
      raw = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
      unsigned w[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const unsigned*>(&v);
      }
      raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};
template <typename T>
struct Chunk<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T* p) { raw = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = raw; }
  template <bool ALIGNED>
  __device__ __forceinline__ void put(T* p) const {
    *p = raw;
  }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = static_cast<float>(raw); }
  __device__ __forceinline__ void set(const float (&x)[1]) { raw = static_cast<T>(x[0]); }
};

// A thread's two chunks of a row and the turns of its E pairs. Chunk pair p of
// the D / 2E of a row: in the half layout chunks p and p + rot / 2E while these
// rotate, else two neighbours behind rot_dim; in the interleaved layout chunks
// 2p and 2p + 1. E divides rot_dim / 2.
template <typename T, int D, int E>
struct Pair {
  int a, b;      // first elements of the two chunks
  bool turned, half;
  float c[E], s[E];
  __device__ __forceinline__ void place(const vattn_rope& R, int p) {
    half = R.layout == VATTN_ROPE_HALF;
    turned = p * E < R.rot_dim / 2;
    a = half && turned ? p * E : 2 * p * E;
    b = half && turned ? R.rot_dim / 2 + p * E : a + E;
  }
  __device__ __forceinline__ void turn(const vattn_rope& R, int p, int pos, bool transpose) {
    if (!turned) return;
#pragma unroll
    for (int e = 0; e < E; e++) pair_turn(R, p * E + e, pos, transpose, c[e], s[e]);
  }
  // one rounding per product and sum, the same in every variant
  __device__ static __forceinline__ void turn_pair(float& u, float& v, float c, float s) {
    const float w = __fmaf_rn(u, c, -__fmul_rn(v, s));
    v = __fmaf_rn(v, c, __fmul_rn(u, s));
    u = w;
  }
  __device__ __forceinline__ void apply(Chunk<T, E>& ca, Chunk<T, E>& cb) const {
    float x[E], y[E];
    ca.get(x);
    cb.get(y);
    if (half || E == 1) {
#pragma unroll
      for (int e = 0; e < E; e++) turn_pair(x[e], y[e], c[e], s[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E / 2; e++) {
        turn_pair(x[2 * e], x[2 * e + 1], c[e], s[e]);
        turn_pair(y[2 * e], y[2 * e + 1], c[E / 2 + e], s[E / 2 + e]);
      }
    }
    ca.set(x);
    cb.set(y);
  }
};

// Cosines and sines of a block's tokens, each computed once: thread by thread
// over (token, pair), then read back by the lanes that share the token.
template <typename T, int D, int E>
struct TurnTable {
  static constexpr int NP = D / (2 * E);
  static constexpr int SIZE = kThreads / NP * (D / 2);  // pairs of the tokens of a block
  float2 cs[SIZE];
  template <typename PosOf>
  __device__ __forceinline__ void fill(const vattn_rope& R, int tokens, bool transpose, PosOf pos) {
    const int half = R.rot_dim / 2;
    for (int x = threadIdx.x; x < tokens * (D / 2); x += kThreads) {
      const int t = x / (D / 2), i = x % (D / 2);
      if (i >= half) continue;
      float2 v;
      pair_turn(R, i, pos(t), transpose, v.x, v.y);
      cs[x] = v;
    }
  }
  __device__ __forceinline__ void read(Pair<T, D, E>& P, int t, int p) const {
    if (!P.turned) return;
#pragma unroll
    for (int e = 0; e < E; e++) {
      const float2 v = cs[t * (D / 2) + p * E + e];
      P.c[e] = v.x;
      P.s[e] = v.y;
    }
  }
};

// ---------------------------------------------------------------- rotate
struct RotateArgs {
  vattn_rope rope;
  const void* x;
  void* out;
  const int* positions;
  int tokens, heads, transpose;
  int lanes, tok_block;  // threads that share a token's heads (per chunk pair); tokens of a block
  long long xt, xh, ot, oh;
};

constexpr int kUnroll = 4;  // rows whose loads a thread issues together

template <typename T, int D, int E>
__global__ void __launch_bounds__(kThreads) k_rotate(const __grid_constant__ RotateArgs A) {
  constexpr int NP = D / (2 * E);
  __shared__ TurnTable<T, D, E> table;
  const int p = threadIdx.x % NP, rest = threadIdx.x / NP;
  const int hl = kThreads / NP / A.tok_block;  // head lanes of a block
  const int t0 = blockIdx.x * A.tok_block, i = rest / hl, t = t0 + i;
  const int r0 = t < A.tokens ? blockIdx.y * hl + rest % hl : A.heads;
  Pair<T, D, E> P;
  P.place(A.rope, p);
  dependency_wait();
  const T* x = static_cast<const T*>(A.x) + t * A.xt;
  T* out = static_cast<T*>(A.out) + t * A.ot;
  Chunk<T, E> ca[kUnroll], cb[kUnroll];
  auto load = [&](int r) {
#pragma unroll
    for (int k = 0; k < kUnroll; k++) {
      const int h = r + k * A.lanes;
      if (h >= A.heads) break;
      ca[k].load(x + h * A.xh + P.a);
      cb[k].load(x + h * A.xh + P.b);
    }
  };
  load(r0);  // in flight while the cosines are computed
  table.fill(A.rope, min(A.tok_block, A.tokens - t0), A.transpose != 0, [&](int j) { return A.positions[t0 + j]; });
  __syncthreads();
  if (r0 < A.heads) table.read(P, i, p);
  for (int r = r0; r < A.heads;) {
#pragma unroll
    for (int k = 0; k < kUnroll; k++) {
      const int h = r + k * A.lanes;
      if (h >= A.heads) break;
      if (P.turned) P.apply(ca[k], cb[k]);
      ca[k].store(out + h * A.oh + P.a);
      cb[k].store(out + h * A.oh + P.b);
    }
    r += kUnroll * A.lanes;
    load(r);
  }
}

// ---------------------------------------------------------------- append
struct AppendArgs {
  vattn_rope rope;   // rot_dim = 0: no rotation
  const void *k, *v, *q;
  long long ks, vs, qs;
  void *q_out, *k_cache, *v_cache, *k_t, *k_proj;
  const float* basis;
  const int *page_table, *seq_lens, *cu;
  unsigned* err;
  int tokens, batch, Hq, Hkv, ps, pps, max_ctx, num_pages;
  int key_blocks;        // proxies: blocks that take the keys and values
  int lanes, tok_block;  // as in RotateArgs
  int row_y;             // blocks that share a token's rows
};

// Position and cache row (page * Hkv * ps + slot; -1: nothing to write) of
// tokens [t0, t0 + n) into shared memory, by the whole block. Every sequence
// marks its own tokens of the range, in one round of loads. Only bounds that
// descend can give a token to several: then the first of these has it, found in
// a second round.
__device__ void resolve(const AppendArgs& A, int t0, int n, int* s_seq, int* s_pos, int* s_row) {
  constexpr int kNone = 0x7FFFFFFF;
  if (A.cu != nullptr) {
    // calls take(b, first, last, position of token 0) for every sequence with tokens of the range
    auto sequences = [&](bool report, auto take) -> bool {
      bool bad = false;
      for (int b = threadIdx.x; b < A.batch; b += blockDim.x) {
        const int lo = A.cu[b], hi = A.cu[b + 1];
        if (lo < 0 || hi < lo || hi > A.tokens) {
          if (report && t0 == 0) atomicOr(A.err, kDevBadSeqlen);
          bad = true;
          continue;
        }
        const int e = min(hi, t0 + n);
        // (the first tokens' block checks the lengths of sequences without new tokens too)
        const bool any = e > max(lo, t0);
        if (!any && t0 > 0) continue;
        const int len = A.seq_lens[b];  // any int: compared before anything is subtracted from it
        if (len < hi - lo || len > A.max_ctx) {
          if (report) atomicOr(A.err, kDevBadSeqlen);
          continue;
        }
        if (any) take(b, max(lo, t0), e, len - hi);
      }
      return bad;
    };
    for (int i = threadIdx.x; i < n; i += blockDim.x) s_seq[i] = kNone;
    __syncthreads();
    const bool bad = sequences(true, [&](int b, int t, int e, int base) {
      for (; t < e; t++) {
        s_seq[t - t0] = b;
        s_pos[t - t0] = base + t;
      }
    });
    if (__syncthreads_or(bad)) {
      for (int i = threadIdx.x; i < n; i += blockDim.x) s_seq[i] = kNone;
      __syncthreads();
      sequences(false, [&](int b, int t, int e, int) {
        for (; t < e; t++) atomicMin(&s_seq[t - t0], b);
      });
      __syncthreads();
      sequences(false, [&](int b, int t, int e, int base) {
        for (; t < e; t++)
          if (s_seq[t - t0] == b) s_pos[t - t0] = base + t;
      });
      __syncthreads();
    }
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int row = -1;  // below 2^31, as the host checked
    int b, pos;
    if (A.cu != nullptr) {
      b = s_seq[i];
      pos = b == kNone ? -1 : s_pos[i];
    } else {
      b = t0 + i;
      int len = A.seq_lens[b];
      if (len < 0 || len > A.max_ctx) {
        atomicOr(A.err, kDevBadSeqlen);
        len = 0;
      }
      pos = len - 1;
      s_pos[i] = pos;
    }
    if (pos >= 0) {
      const int slot = pos / A.ps;
      const int page = A.page_table[static_cast<size_t>(b) * A.pps + slot];
      if (page < 0 || page >= A.num_pages)
        atomicOr(A.err, kDevBadPage);
      else
        row = page * A.Hkv * A.ps + (pos - slot * A.ps);
    }
    s_row[i] = row;
  }
  __syncthreads();
}

// Keys with a proxy copy, and the values beside them. The jobs (tile of TT
// tokens, KV head) are cut evenly over about as many blocks as are resident; a
// block keeps a tile's cosines in registers over its heads, and the stored
// (rounded) keys of one job in shared memory for the copy while the next job's
// rows are loaded.
template <typename T, int D, int E, int PROXY>
struct KeyTile {
  static constexpr int NP = D / (2 * E);
  static constexpr int TT = E > 1 ? kThreads / NP : 32;  // vectors: one chunk pair per thread
  // row pitch: odd in words for the transposed copy's column reads, 16-byte
  // rows for the projection's fragment loads
  static constexpr int LD = PROXY == VATTN_SPARQ ? D + 4 / sizeof(T) : D + 16 / sizeof(T);
  // shared memory: a head's split basis (bf16 projections), two tiles of keys
  static constexpr bool SPLIT = PROXY == VATTN_LOKI && sizeof(T) == 2;
  static constexpr size_t BASIS = SPLIT ? 6 * D * kRank : 0, BYTES = BASIS + 2 * TT * LD * sizeof(T);
};

__device__ __forceinline__ unsigned smem_addr(const void* p) { return static_cast<unsigned>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void ldsm4(unsigned addr, unsigned (&a)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(unsigned addr, unsigned (&a)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const unsigned*>(&v);
}

// Projected keys of a tile of bf16 keys: [TT tokens x D] . [D x 32] on the
// tensor cores, the fp32 basis as three bf16 terms, which hold its 24 bits whole:
// the products are exact and summed in fp32: 134 of 2.1 million bf16 results are
// not the 64-bit product rounded, 325 of an fp32 matrix product. (Two terms lose
// 2^-17 of a basis entry; that moved one result in 400.) The block splits
// a head's basis once per job into shared memory; every warp has 16 tokens and
// 4 TT / 16 components. 8190 tokens of 8 heads (71 MB): 26.2 us (two terms: 25.2), of which 6 us
// go without the projection and 3 without the cosines (each warp splitting its
// own operands: 27; fp32 FMAs from shared memory: 73). Loaded after the stores,
// where no other row is held, the basis costs no spill (before them: 27.6);
// copied a job ahead with cp.async it gains 0.5 us for 16 KB more.
template <int D, bool VEC>
struct Basis {
  static constexpr int N = D * kRank / 4 / kThreads;  // quads of components per thread
  float4 x[N];
  __device__ __forceinline__ void load(const float* basis) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const float* p = basis + 4 * (i * kThreads + threadIdx.x);
      if constexpr (VEC)
        x[i] = __ldg(reinterpret_cast<const float4*>(p));
      else
        x[i] = make_float4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
    }
  }
  // The first two terms: rows of 128 bytes, one per key dimension, whose 16-byte
  // chunk 2 c + term holds components 8 c to 8 c + 7, at place
  // (2 c + term) ^ (row % 8). The third behind them: rows of 64 bytes, chunk c at
  // place c ^ (row / 2 % 4). Eight rows of one chunk lie in different banks.
  __device__ __forceinline__ void split(unsigned char* s) const {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int at = i * kThreads + threadIdx.x, row = at / (kRank / 4), quad = at % (kRank / 4);
      const float4 v = x[i];
      const unsigned h0 = pack2(v.x, v.y), h1 = pack2(v.z, v.w);
      const float4 r = make_float4(v.x - low(h0), v.y - high(h0), v.z - low(h1), v.w - high(h1));
      const unsigned l0 = pack2(r.x, r.y), l1 = pack2(r.z, r.w);
      unsigned char* o = s + row * 128 + 8 * (quad & 1);
      *reinterpret_cast<uint2*>(o + (((quad & ~1) ^ (row & 7)) << 4)) = make_uint2(h0, h1);
      *reinterpret_cast<uint2*>(o + (((quad | 1) ^ (row & 7)) << 4)) = make_uint2(l0, l1);
      *reinterpret_cast<uint2*>(s + D * 128 + row * 64 + (((quad >> 1) ^ (row >> 1 & 3)) << 4) + 8 * (quad & 1)) =
          make_uint2(pack2(r.x - low(l0), r.y - high(l0)), pack2(r.z - low(l1), r.w - high(l1)));
    }
  }
  __device__ static __forceinline__ float low(unsigned h) { return __uint_as_float(h << 16); }
  __device__ static __forceinline__ float high(unsigned h) { return __uint_as_float(h & 0xFFFF0000u); }
};
template <int D, int LD, int TT>
__device__ __forceinline__ void project_tile(const __nv_bfloat16* s_key, const unsigned char* s_basis,
                                             const int* s_row, int n, int h, const AppendArgs& A) {
  constexpr int MT = TT / 16, NX = 4 * MT / 8;  // token tiles; 8-component tiles of a warp
  static_assert(kThreads / 32 * NX == 4 * MT && NX >= 1, "warps cover the tile");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int m0 = 16 * (warp % MT), n0 = 8 * NX * (warp / MT);
  if (m0 >= n) return;
  // The tensor core truncates what it adds, by the accumulator's magnitude: the
  // second and third terms have one of their own.
  float acc[NX][4], small[NX][4];
#pragma unroll
  for (int x = 0; x < NX; x++)
#pragma unroll
    for (int i = 0; i < 4; i++) acc[x][i] = small[x][i] = 0.0f;
  const unsigned rows = smem_addr(s_key + (m0 + (lane & 15)) * LD + (lane >> 4) * 8);
  // lanes 0-15 address the first term of 16 rows, lanes 16-31 the second
  const unsigned brow = smem_addr(s_basis + (lane & 15) * 128);
  // the third term of 32 rows, a row per lane
  const unsigned crow = smem_addr(s_basis + D * 128 + lane * 64);
#pragma unroll
  for (int k = 0; k < D; k += 32) {
    unsigned a[2][4];
    ldsm4(rows + k * 2, a[0]);
    ldsm4(rows + k * 2 + 32, a[1]);
#pragma unroll
    for (int x = 0; x < NX; x++) {
      unsigned c[4];
      ldsm4_t(crow + k * 64 + (((n0 / 8 + x) ^ (lane >> 1 & 3)) << 4), c);
#pragma unroll
      for (int i = 0; i < 2; i++) {
        unsigned b[4];
        ldsm4_t(brow + (k + 16 * i) * 128 + (((2 * (n0 / 8 + x) + (lane >> 4)) ^ (lane & 7)) << 4), b);
        mma16816(acc[x], a[i], b[0], b[1]);
        mma16816(small[x], a[i], b[2], b[3]);
        mma16816(small[x], a[i], c[2 * i], c[2 * i + 1]);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < NX; x++)
#pragma unroll
    for (int i = 0; i < 4; i++) acc[x][i] += small[x][i];
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(A.k_proj);
#pragma unroll
  for (int half = 0; half < 2; half++) {
    const int i = m0 + (lane >> 2) + 8 * half;
    if (i >= n || s_row[i] < 0) continue;
    unsigned* o =
        reinterpret_cast<unsigned*>(out + static_cast<size_t>(s_row[i] + h * A.ps) * kRank + n0 + 2 * (lane & 3));
#pragma unroll
    for (int x = 0; x < NX; x++) o[4 * x] = pack2(acc[x][2 * half], acc[x][2 * half + 1]);
  }
}
// The same of fp32 keys: fp32 FMAs, four tokens per thread.
template <int D, int LD, int TT>
__device__ __forceinline__ void project_tile(const float* s_key, const float* basis, const int* s_row, int n, int h,
                                             const AppendArgs& A) {
  static_assert(TT <= kThreads / kRank * 4, "threads cover the tile");
  const int r = threadIdx.x % kRank, i0 = threadIdx.x / kRank * 4;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (i0 >= n) return;
#pragma unroll 4
  for (int j = 0; j < D; j += 4) {
    float b[4];
#pragma unroll
    for (int e = 0; e < 4; e++) b[e] = __ldg(basis + (j + e) * kRank + r);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float4 k = *reinterpret_cast<const float4*>(s_key + (i0 + i) * LD + j);
      acc[i] = fmaf(k.x, b[0], acc[i]);
      acc[i] = fmaf(k.y, b[1], acc[i]);
      acc[i] = fmaf(k.z, b[2], acc[i]);
      acc[i] = fmaf(k.w, b[3], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (i0 + i < n && s_row[i0 + i] >= 0)
      static_cast<float*>(A.k_proj)[static_cast<size_t>(s_row[i0 + i] + h * A.ps) * kRank + r] =
          acc[i];
}

template <typename T, int D, int E, int PROXY>
__global__ void __launch_bounds__(kThreads) k_append(const __grid_constant__ AppendArgs A) {
  constexpr int NP = D / (2 * E);
  __shared__ int s_seq[kMaxTok], s_pos[kMaxTok];
  __shared__ int s_row[kMaxTok];
  using Tile = KeyTile<T, D, E, PROXY>;
  using Table = TurnTable<T, D, E>;
  // a block is one or the other: the table of cosines, or a tile's keys and the
  // split basis behind them
  constexpr size_t kTileBytes = PROXY == VATTN_EXACT ? 0 : Tile::BYTES;
  __shared__ __align__(128) unsigned char s_raw[kTileBytes > sizeof(Table) ? kTileBytes : sizeof(Table)];
  dependency_wait();
  int blk = blockIdx.x;
  if constexpr (PROXY != VATTN_EXACT) {
    if (blk < A.key_blocks) {
      constexpr int TT = Tile::TT, LD = Tile::LD, LANES = kThreads / NP;  // LANES: tokens at once
      constexpr bool kOnce = TT <= LANES;                           // every thread has one token
      constexpr bool kSplit = Tile::SPLIT;
      T* s_key = reinterpret_cast<T*>(s_raw + Tile::BASIS);
      const int jobs = (A.tokens + TT - 1) / TT * A.Hkv;
      const int j0 = static_cast<int>(static_cast<long long>(jobs) * blk / A.key_blocks);
      const int j1 = static_cast<int>(static_cast<long long>(jobs) * (blk + 1) / A.key_blocks);
      const int p = threadIdx.x % NP, lane0 = threadIdx.x / NP;
      Pair<T, D, E> P;
      P.place(A.rope, p);
      Chunk<T, E> next[4];  // the key's and the value's chunk pair of the next job
      auto load = [&](int t, int h, Chunk<T, E> (&c)[4]) {
        const T* x = static_cast<const T*>(A.k) + t * A.ks + h * D;
        const T* y = static_cast<const T*>(A.v) + t * A.vs + h * D;
        c[0].load(x + P.a);
        c[1].load(x + P.b);
        c[2].load(y + P.a);
        c[3].load(y + P.b);
      };
      auto load_next = [&](int j) {
        const long long t = static_cast<long long>(j / A.Hkv) * TT + lane0;
        if (kOnce && j < j1 && lane0 < TT && t < A.tokens) load(static_cast<int>(t), j % A.Hkv, next);
      };
      load_next(j0);  // in flight while positions and pages are found
      int tile = -1, n = 0;
      bool mine = false;
      for (int j = j0; j < j1; j++) {
        const int h = j % A.Hkv, t0 = j / A.Hkv * TT;
        if (j / A.Hkv != tile) {
          tile = j / A.Hkv;
          n = min(TT, A.tokens - t0);
          __syncthreads();  // the tile before is done with its rows
          resolve(A, t0, n, s_seq, s_pos, s_row);
          mine = lane0 < n && s_row[lane0] >= 0;
          if (kOnce && mine) P.turn(A.rope, p, s_pos[lane0], false);
        }
        T* key = s_key + ((j - j0) & 1) * (TT * LD);
        const float* basis = A.basis + static_cast<size_t>(h) * D * kRank;
        Basis<D, (E > 1)> split;
        auto put = [&](int i, Chunk<T, E> (&c)[4]) {
          if (P.turned) P.apply(c[0], c[1]);
          const size_t at = static_cast<size_t>(s_row[i] + h * A.ps) * D;
          T* o = static_cast<T*>(A.k_cache) + at;
          c[0].store(o + P.a);
          c[1].store(o + P.b);
          T* ov = static_cast<T*>(A.v_cache) + at;
          c[2].store(ov + P.a);
          c[3].store(ov + P.b);
          c[0].template put<(LD * sizeof(T)) % 16 == 0>(key + i * LD + P.a);
          c[1].template put<(LD * sizeof(T)) % 16 == 0>(key + i * LD + P.b);
        };
        if constexpr (kOnce) {
          Chunk<T, E> c[4] = {next[0], next[1], next[2], next[3]};
          load_next(j + 1);
          if (mine) put(lane0, c);
        } else {
          for (int i = lane0; i < n; i += LANES) {
            if (s_row[i] < 0) continue;
            P.turn(A.rope, p, s_pos[i], false);
            Chunk<T, E> c[4];
            load(t0 + i, h, c);
            put(i, c);
          }
        }
        if constexpr (kSplit) {
          split.load(basis);
          __syncthreads();  // the job before is done with its basis
          split.split(s_raw);
        }
        __syncthreads();  // (the other buffer's readers have passed the sync before)
        if constexpr (PROXY == VATTN_SPARQ) {
          // neighbouring lanes hold neighbouring tokens, whose slots are neighbours too
          const int i = threadIdx.x % TT;
          if (i < n && s_row[i] >= 0) {
            // row = page * Hkv * ps + slot: the head's dim-major block starts at (page * Hkv + h) * D * ps
            const int head = s_row[i] / A.ps + h, slot = s_row[i] % A.ps;
            T* o = static_cast<T*>(A.k_t) + static_cast<size_t>(head) * D * A.ps + slot;
#pragma unroll 8
            for (int j = threadIdx.x / TT; j < D; j += kThreads / TT) o[static_cast<size_t>(j) * A.ps] = key[i * LD + j];
          }
        } else if constexpr (kSplit) {
          project_tile<D, LD, TT>(key, s_raw, s_row, n, h, A);
        } else {
          project_tile<D, LD, TT>(key, basis, s_row, n, h, A);
        }
      }
      return;
    }
    blk -= A.key_blocks;
  }
  // rows of tok_block tokens: keys, queries and values, or the queries alone
  Table& table = *reinterpret_cast<Table*>(s_raw);
  const int hl = kThreads / NP / A.tok_block;
  const int t0 = blk / A.row_y * A.tok_block;
  const int n = min(A.tok_block, A.tokens - t0);
  const int p = threadIdx.x % NP, rest = threadIdx.x / NP, i = rest / hl;
  const int nk = PROXY == VATTN_EXACT ? A.Hkv : 0;  // the values are as many
  const int rows = 2 * nk + (A.q != nullptr ? A.Hq : 0), nq = rows - nk;
  const int r0 = i < n ? blk % A.row_y * hl + rest % hl : rows;
  const long long t = t0 + i;
  Pair<T, D, E> P;
  P.place(A.rope, p);
  auto src = [&](int r) -> const T* {
    if (r < nk) return static_cast<const T*>(A.k) + t * A.ks + r * D;
    if (r < nq) return static_cast<const T*>(A.q) + t * A.qs + (r - nk) * D;
    return static_cast<const T*>(A.v) + t * A.vs + (r - nq) * D;
  };
  Chunk<T, E> ca[kUnroll], cb[kUnroll];
  auto load = [&](int r) {
#pragma unroll
    for (int k = 0; k < kUnroll; k++) {
      const int h = r + k * A.lanes;
      if (h >= rows) break;
      const T* x = src(h);
      ca[k].load(x + P.a);
      cb[k].load(x + P.b);
    }
  };
  load(r0);  // in flight while positions, pages and cosines are found
  resolve(A, t0, n, s_seq, s_pos, s_row);
  if (A.rope.rot_dim > 0) {
    table.fill(A.rope, n, false, [&](int j) { return s_pos[j]; });
    __syncthreads();
  }
  if (i >= n || s_row[i] < 0 || r0 >= rows) return;
  table.read(P, i, p);
  const int row = s_row[i];
  auto dst = [&](int r) -> T* {
    if (r < nk) return static_cast<T*>(A.k_cache) + static_cast<size_t>(row + r * A.ps) * D;
    if (r < nq) return static_cast<T*>(A.q_out) + (t * A.Hq + (r - nk)) * D;
    return static_cast<T*>(A.v_cache) + static_cast<size_t>(row + (r - nq) * A.ps) * D;
  };
  for (int r = r0; r < rows;) {
#pragma unroll
    for (int k = 0; k < kUnroll; k++) {
      const int h = r + k * A.lanes;
      if (h >= rows) break;
      if (P.turned && h < nq) P.apply(ca[k], cb[k]);
      T* o = dst(h);
      ca[k].store(o + P.a);
      cb[k].store(o + P.b);
    }
    r += kUnroll * A.lanes;
    load(r);
  }
}

// ---------------------------------------------------------------- host side
// Threads that share a token's rows and tokens of a block. As many threads per
// token as it takes to put about `want` threads on the device, a power of two,
// at most one per row: a thread with more rows computes its cosines for more
// rows, and issues the loads of kUnroll of them together.
struct Split {
  int lanes, tok_block, row_y;
};
Split split_rows(long long tokens, int rows, int np, int sms) {
  const long long want = 1024LL * sms;
  int lanes = 1;
  while (lanes < rows && lanes < 4096 && tokens * np * lanes < want) lanes *= 2;
  Split s;
  const int per = kThreads / np;  // (token, lane) places of a block
  const int hl = std::min(lanes, per);
  s.tok_block = std::min(per / hl, kMaxTok);
  const int hl2 = per / s.tok_block;
  s.row_y = std::max(1, lanes / hl2);
  s.lanes = s.row_y * hl2;
  return s;
}

bool plan_ok(const vattn_rope* r) {
  return r && (r->head_dim == 64 || r->head_dim == 128) && r->rot_dim >= 2 && r->rot_dim <= r->head_dim &&
         r->rot_dim % 2 == 0 && (r->layout == VATTN_ROPE_HALF || r->layout == VATTN_ROPE_INTERLEAVED) &&
         r->amplitude > 0.0f && isfinite(r->amplitude);
}

template <typename A>
int launch_rows(void (*kern)(A), unsigned gx, unsigned gy, const A& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gx, gy);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess) return VATTN_OK;
  cudaGetLastError();  // reported here: the next call's check must not find it
  return VATTN_ECUDA;
}

template <typename T, int D>
int run_rotate(RotateArgs& a, bool vec, int sms, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  const int np = vec ? D / (2 * E) : D / 2;
  const Split s = split_rows(a.tokens, a.heads, np, sms);
  a.lanes = s.lanes;
  a.tok_block = s.tok_block;
  const unsigned gx = static_cast<unsigned>((a.tokens + s.tok_block - 1) / s.tok_block);
  return launch_rows(vec ? k_rotate<T, D, E> : k_rotate<T, D, 1>, gx, static_cast<unsigned>(s.row_y), a, st);
}

template <typename T, int D, int PROXY>
int run_append(AppendArgs& a, bool vec, int sms, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  const int np = vec ? D / (2 * E) : D / 2;
  const int rows = (PROXY == VATTN_EXACT ? 2 * a.Hkv : 0) + (a.q ? a.Hq : 0);
  const Split s = split_rows(a.tokens, std::max(rows, 1), np, sms);
  a.lanes = s.lanes;
  a.tok_block = s.tok_block;
  a.row_y = s.row_y;
  a.key_blocks = 0;
  if constexpr (PROXY != VATTN_EXACT) {
    const int TT = vec ? KeyTile<T, D, E, PROXY>::TT : KeyTile<T, D, 1, PROXY>::TT;
    const long long jobs = (static_cast<long long>(a.tokens) + TT - 1) / TT * a.Hkv;
    if (jobs > 0x3FFFFFFFLL) return VATTN_EINVAL;
    // three fit an SM. With queries behind them, which fill the SMs that they
    // leave, blocks stay within a tile, with as many of its heads as still give
    // every SM its three (8192 tokens, dim-major: 44 us; cut evenly 47.6)
    long long blocks = std::min(jobs, 3LL * sms);
    if (rows > 0) {
      int heads = a.Hkv;
      while (heads > 1 && (a.Hkv % heads || jobs / heads < 3LL * sms)) heads--;
      blocks = jobs / heads;
    }
    a.key_blocks = static_cast<int>(blocks);
  }
  const long long gx =
      a.key_blocks + (rows > 0 ? static_cast<long long>((a.tokens + s.tok_block - 1) / s.tok_block) * s.row_y : 0);
  if (gx > 0x7FFFFFFFLL) return VATTN_EINVAL;
  return launch_rows(vec ? k_append<T, D, E, PROXY> : k_append<T, D, 1, PROXY>, static_cast<unsigned>(gx), 1u, a, st);
}

template <typename T, int D>
int run_append(AppendArgs& a, int proxy, bool vec, int sms, cudaStream_t st) {
  if (proxy == VATTN_SPARQ) return run_append<T, D, VATTN_SPARQ>(a, vec, sms, st);
  if (proxy == VATTN_LOKI) return run_append<T, D, VATTN_LOKI>(a, vec, sms, st);
  return run_append<T, D, VATTN_EXACT>(a, vec, sms, st);
}

}  // namespace

extern "C" {

int vattn_rope_init(vattn_rope* rope, const vattn_rope_config* cfg) {
  if (!rope || !cfg) return VATTN_EINVAL;
  const vattn_rope_config& c = *cfg;
  if (!(c.head_dim == 64 || c.head_dim == 128)) return VATTN_EINVAL;
  if (c.rot_dim < 2 || c.rot_dim > c.head_dim || c.rot_dim % 2) return VATTN_EINVAL;
  if (c.layout != VATTN_ROPE_HALF && c.layout != VATTN_ROPE_INTERLEAVED) return VATTN_EINVAL;
  if (c.scaling < VATTN_ROPE_NONE || c.scaling > VATTN_ROPE_YARN) return VATTN_EINVAL;
  if (!(c.base > 1.0) || !isfinite(c.base)) return VATTN_EINVAL;
  if (!(c.amplitude >= 0.0) || !isfinite(c.amplitude)) return VATTN_EINVAL;
  if (c.scaling != VATTN_ROPE_NONE && (!(c.factor > 0.0) || !isfinite(c.factor))) return VATTN_EINVAL;
  const bool by_ctx = c.scaling == VATTN_ROPE_BANDS || c.scaling == VATTN_ROPE_YARN;
  if (by_ctx && (!(c.original_ctx > 0.0) || !isfinite(c.original_ctx))) return VATTN_EINVAL;
  if (c.scaling == VATTN_ROPE_BANDS && !(c.low > 0.0 && c.low < c.high && isfinite(c.high))) return VATTN_EINVAL;
  if (c.scaling == VATTN_ROPE_YARN && !(c.slow > 0.0 && c.slow < c.fast && isfinite(c.fast))) return VATTN_EINVAL;
  const long double two_pi = 6.283185307179586476925286766559L;
  const int r = c.rot_dim;
  long double base = c.base;
  if (c.scaling == VATTN_ROPE_BASE && r > 2)
    base *= powl(c.factor, static_cast<long double>(r) / (r - 2));
  if (!(base > 1.0L) || !isfinite(static_cast<double>(base))) return VATTN_EINVAL;
  auto corner = [&](double n) { return r * logl(c.original_ctx / (n * two_pi)) / (2.0L * logl(c.base)); };
  long double lo = 0.0L, span = 1.0L;
  if (c.scaling == VATTN_ROPE_YARN) {
    lo = fmaxl(floorl(corner(c.fast)), 0.0L);
    const long double hi = fminl(ceill(corner(c.slow)), static_cast<long double>(r - 1));
    span = hi > lo ? hi - lo : 0.001L;
  }
  vattn_rope out = {};
  out.head_dim = c.head_dim;
  out.rot_dim = r;
  out.layout = c.layout;
  double amp = c.amplitude;
  if (amp == 0.0) amp = c.scaling == VATTN_ROPE_YARN && c.factor > 1.0 ? 0.1 * log(c.factor) + 1.0 : 1.0;
  out.amplitude = static_cast<float>(amp);
  if (!(out.amplitude > 0.0f) || !isfinite(out.amplitude)) return VATTN_EINVAL;
  for (int i = 0; i < r / 2; i++) {
    long double f = powl(base, -2.0L * i / r);
    if (c.scaling == VATTN_ROPE_LINEAR) {
      f /= c.factor;
    } else if (c.scaling == VATTN_ROPE_BANDS) {
      const long double t = (c.original_ctx * f / two_pi - c.low) / (c.high - c.low);
      const long double keep = fminl(fmaxl(t, 0.0L), 1.0L);
      f = keep * f + (1.0L - keep) * f / c.factor;
    } else if (c.scaling == VATTN_ROPE_YARN) {
      const long double ramp = fminl(fmaxl((i - lo) / span, 0.0L), 1.0L);
      f = f * (1.0L - ramp) + f / c.factor * ramp;
    }
    const long double turns = fmodl(f / two_pi, 1.0L);
    // below 2^64: turns < 1; a value that rounds up to a whole turn is turn 0
    const long double scaled = rintl(turns * 18446744073709551616.0L);
    out.turns[i] = scaled >= 18446744073709551616.0L ? 0ull : static_cast<uint64_t>(scaled);
  }
  *rope = out;
  return VATTN_OK;
}

int vattn_rotate(const vattn_rope* rope, const void* x, void* out, const int32_t* positions, int tokens, int heads,
                 int dtype, long long xt, long long xh, long long ot, long long oh, int transpose, void* stream) {
  if (!plan_ok(rope) || tokens < 0 || tokens > kMaxTokens || heads < 0 || heads > kMaxHeads) return VATTN_EINVAL;
  if (dtype != VATTN_FP32 && dtype != VATTN_BF16) return VATTN_EINVAL;
  if (tokens == 0 || heads == 0) return VATTN_OK;
  if (!x || !out || !positions) return VATTN_EINVAL;
  if (!aligned_to(dtype == VATTN_BF16 ? 2 : 4, x, out) || !aligned_to(4, positions)) return VATTN_EINVAL;
  const int D = rope->head_dim;
  if (xt < 0 || xh < 0 || ot < 0 || oh < 0) return VATTN_EINVAL;
  // no two rows of out overlap: heads within a token's span, or tokens within a head's
  if ((heads > 1 && oh < D) || (tokens > 1 && ot < D)) return VATTN_EINVAL;
  if (heads > 1 && tokens > 1 && ot < (heads - 1) * oh + D && oh < (tokens - 1) * ot + D) return VATTN_EINVAL;
  if (x == out && ((tokens > 1 && xt != ot) || (heads > 1 && xh != oh))) return VATTN_EINVAL;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return VATTN_ECUDA;
  }
  RotateArgs a;
  a.rope = *rope;
  a.x = x;
  a.out = out;
  a.positions = positions;
  a.tokens = tokens;
  a.heads = heads;
  a.transpose = transpose;
  a.xt = tokens > 1 ? xt : 0;
  a.xh = heads > 1 ? xh : 0;
  a.ot = tokens > 1 ? ot : 0;
  a.oh = heads > 1 ? oh : 0;
  // 16-byte chunks where every chunk of every row is aligned and no chunk
  // crosses the end of the rotated part
  const int E = dtype == VATTN_BF16 ? 8 : 4;
  const bool vec = rope->rot_dim / 2 % E == 0 && aligned16(x) && aligned16(out) &&
                   (a.xt | a.xh | a.ot | a.oh) % E == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == VATTN_BF16)
    return D == 128 ? run_rotate<__nv_bfloat16, 128>(a, vec, sms, st) : run_rotate<__nv_bfloat16, 64>(a, vec, sms, st);
  return D == 128 ? run_rotate<float, 128>(a, vec, sms, st) : run_rotate<float, 64>(a, vec, sms, st);
}

int vattn_append(vattn_ctx* ctx, const vattn_append_params* prm, const int32_t* page_table, const int32_t* seq_lens,
                 int batch, void* stream) {
  if (!ctx) return VATTN_EINVAL;
  ctx->last_status = VATTN_EINVAL;
  const vattn_config& c = ctx->cfg;
  const int D = c.head_dim;
  if (!prm || batch < 0 || batch > c.max_batch || prm->tokens < 0 || prm->tokens > kMaxTokens || prm->num_pages < 1) return VATTN_EINVAL;
  if (prm->rope && (!plan_ok(prm->rope) || prm->rope->head_dim != D)) return VATTN_EINVAL;
  if (!prm->cu_tokens && prm->tokens != batch) return VATTN_EINVAL;
  if (static_cast<unsigned long long>(prm->num_pages) * c.num_kv_heads * static_cast<unsigned long long>(c.page_size) >
      0x7FFFFFFFull)
    return VATTN_EINVAL;
  if (batch == 0 || prm->tokens == 0) {
    ctx->last_launches = 0;
    return ctx->last_status = VATTN_OK;
  }
  if (!page_table || !seq_lens || !prm->k || !prm->v || !prm->k_cache || !prm->v_cache) return VATTN_EINVAL;
  if (prm->q && !prm->q_out) return VATTN_EINVAL;
  if (!aligned_to(c.dtype == VATTN_BF16 ? 2 : 4, prm->k, prm->v, prm->q, prm->q_out) ||
      !aligned_to(4, page_table, seq_lens, prm->cu_tokens, prm->proj_basis))
    return VATTN_EINVAL;
  const long long kvw = static_cast<long long>(c.num_kv_heads) * D, qw = static_cast<long long>(c.num_q_heads) * D;
  if (prm->k_stride < kvw || prm->v_stride < kvw) return VATTN_EINVAL;
  if (prm->q && (prm->q_stride < qw || (prm->q == prm->q_out && prm->q_stride != qw))) return VATTN_EINVAL;
  if (!aligned16(prm->k_cache) || !aligned16(prm->v_cache)) return VATTN_EINVAL;
  if (c.proxy == VATTN_SPARQ && (!prm->k_t_cache || !aligned16(prm->k_t_cache))) return VATTN_EINVAL;
  if (c.proxy == VATTN_LOKI && (!prm->k_proj_cache || !prm->proj_basis || !aligned16(prm->k_proj_cache)))
    return VATTN_EINVAL;
  AppendArgs a = {};
  const void *kc = prm->k_cache, *vc = prm->v_cache;
  if (const int rc = vattn::cache_ptrs(c, &kc, &vc)) return ctx->last_status = rc;
  if (prm->rope) a.rope = *prm->rope;
  a.k = prm->k;
  a.v = prm->v;
  a.q = prm->q;
  a.ks = prm->k_stride;
  a.vs = prm->v_stride;
  a.qs = prm->q_stride;
  a.q_out = prm->q_out;
  a.k_cache = const_cast<void*>(kc);
  a.v_cache = const_cast<void*>(vc);
  a.k_t = prm->k_t_cache;
  a.k_proj = prm->k_proj_cache;
  a.basis = prm->proj_basis;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.cu = prm->cu_tokens;
  a.err = ctx->err;
  a.tokens = prm->tokens;
  a.batch = batch;
  a.Hq = c.num_q_heads;
  a.Hkv = c.num_kv_heads;
  a.ps = c.page_size;
  a.pps = (c.max_ctx + c.page_size - 1) / c.page_size;
  a.max_ctx = c.max_ctx;
  a.num_pages = prm->num_pages;
  const int E = c.dtype == VATTN_BF16 ? 8 : 4;
  const bool vec = a.rope.rot_dim / 2 % E == 0 && aligned16(a.k) && aligned16(a.v) && (a.ks | a.vs) % E == 0 &&
                   (c.proxy != VATTN_LOKI || aligned16(a.basis)) &&
                   (!a.q || (aligned16(a.q) && aligned16(a.q_out) && a.qs % E == 0));
  vattn::DeviceScope scope(ctx->device);
  if (!scope.ok) return ctx->last_status = VATTN_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int rc;
  if (c.dtype == VATTN_BF16)
    rc = D == 128 ? run_append<__nv_bfloat16, 128>(a, c.proxy, vec, ctx->num_sms, st)
                  : run_append<__nv_bfloat16, 64>(a, c.proxy, vec, ctx->num_sms, st);
  else
    rc = D == 128 ? run_append<float, 128>(a, c.proxy, vec, ctx->num_sms, st)
                  : run_append<float, 64>(a, c.proxy, vec, ctx->num_sms, st);
  ctx->last_launches = rc == VATTN_OK ? 1 : 0;
  return ctx->last_status = rc;
}

}  // extern "C"
