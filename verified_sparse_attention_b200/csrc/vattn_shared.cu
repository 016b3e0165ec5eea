// Host side of vattn_shared_dense_decode.
#include <algorithm>
#include <type_traits>

#include "vattn_ctx.h"
#include "vattn_shared.cuh"
#include "vattn_prefix_tc.cuh"

using vattn::DevParams;
using vattn::SharedParams;

namespace {

struct SharedKernels {
  void (*prefix)(SharedParams);
  int RB, KT;
  bool tc;  // the tensor-core prefix kernel
  unsigned threads;
  size_t smem;
  void (*own)(SharedParams);  // the sequences' own positions; nullptr: by the gather
  int own_nw;                 // its warps per CTA (one CTA per SM)
  size_t own_smem;
  void (*gather)(DevParams);  // where there is no own kernel
  unsigned gather_threads;
  size_t gather_smem;
  void (*combine[4])(SharedParams);  // 1, 2, 4 or 8 warps per row
};

template <typename T, int D, int G>
SharedKernels kernels_for(bool host_kv) {
  using vattn::kModeSuffix;
  SharedKernels k = {};
  auto simt = [&](void (*prefix)(SharedParams), void (*gather)(DevParams)) {
    k.prefix = prefix;
    k.RB = vattn::PrefixShape<D>::RB;
    k.KT = vattn::PrefixShape<D>::KT;
    k.threads = 256;
    k.smem = vattn::PrefixShape<D>::SMEM;
    k.gather = gather;
    k.gather_smem = vattn::GatherShape<T, D, G>::SMEM;
    k.gather_threads = vattn::GatherShape<T, D, G>::NW * 32;
  };
  if (host_kv) {
    simt(vattn::k_shared_prefix<T, D, true>, vattn::k_gather<T, D, G, kModeSuffix, true>);
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    k.prefix = vattn::k_shared_prefix_tc<D>;
    k.RB = 2 * vattn::PrefixTcShape<D>::M;
    k.KT = vattn::PrefixTcShape<D>::KT;
    k.tc = true;
    k.threads = vattn::PrefixTcShape<D>::THREADS;
    k.smem = vattn::PrefixTcShape<D>::SMEM;
    k.own = vattn::k_shared_own<D, G>;
    k.own_nw = vattn::OwnShape<D>::NW;
    k.own_smem = vattn::OwnShape<D>::SMEM;
  } else {
    simt(vattn::k_shared_prefix<T, D, false>, vattn::k_gather<T, D, G, kModeSuffix>);
  }
  k.combine[0] = vattn::k_shared_combine<D, 1>;
  k.combine[1] = vattn::k_shared_combine<D, 2>;
  k.combine[2] = vattn::k_shared_combine<D, 4>;
  k.combine[3] = vattn::k_shared_combine<D, 8>;
  return k;
}

template <typename T, int D>
SharedKernels pick_g(int G, bool host_kv) {
  if (G == 1) return kernels_for<T, D, 1>(host_kv);
  if (G == 2) return kernels_for<T, D, 2>(host_kv);
  if (G == 4) return kernels_for<T, D, 4>(host_kv);
  return kernels_for<T, D, 8>(host_kv);
}

// The maps of the tensor-core prefix kernel.
int encode_tile_maps(const vattn_config& c, int G, const void* q, const void* k, const void* v, int batch,
                     int num_pages, SharedParams* P) {
  const vattn::EncodeTiledFn fn = vattn::encode_tiled();
  if (!fn) return VATTN_ECUDA;
  int box = P->KT;
  while (c.page_size % box) box /= 2;  // the page size is a multiple of 16
  P->box = box;
  const cuuint64_t d = static_cast<cuuint64_t>(c.head_dim);
  const cuuint64_t rows = static_cast<cuuint64_t>(num_pages) * c.num_kv_heads * static_cast<cuuint64_t>(c.page_size);
  const cuuint64_t dims[2] = {d, rows}, strides[1] = {2 * d};
  const cuuint32_t one[3] = {1u, 1u, 1u};
  auto cache_map = [&](CUtensorMap* map, const void* p, int r) {
    const cuuint32_t boxes[2] = {64u, static_cast<cuuint32_t>(r)};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, boxes, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!cache_map(&P->tmk_t, k, box) || !cache_map(&P->tmv_t, v, box) ||
      !cache_map(&P->tmk_16, k, vattn::kOwnChunk) || !cache_map(&P->tmv_16, v, vattn::kOwnChunk))
    return VATTN_ECUDA;
  const cuuint64_t Hq = static_cast<cuuint64_t>(c.num_q_heads);
  const cuuint64_t qd[3] = {d, Hq, static_cast<cuuint64_t>(batch)}, qs[2] = {2 * d, 2 * d * Hq};
  const cuuint32_t qb[3] = {64u, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(128 / G)};
  if (fn(&P->tmq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), qd, qs, qb, one,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return VATTN_ECUDA;
  return VATTN_OK;
}

SharedKernels pick(const vattn_ctx* ctx) {
  const vattn_config& c = ctx->cfg;
  const bool host_kv = c.kv_location == VATTN_KV_HOST;
  if (c.dtype == VATTN_BF16)
    return c.head_dim == 128 ? pick_g<__nv_bfloat16, 128>(ctx->G, host_kv) : pick_g<__nv_bfloat16, 64>(ctx->G, host_kv);
  return c.head_dim == 128 ? pick_g<float, 128>(ctx->G, host_kv) : pick_g<float, 64>(ctx->G, host_kv);
}

}  // namespace

namespace vattn {

size_t shared_workspace(vattn_ctx* ctx, char* p) {
  const vattn_config& c = ctx->cfg;
  const SharedKernels k = pick(ctx);
  const size_t B = static_cast<size_t>(c.max_batch);
  // every block's rows once, and per CTA the most that a block takes (a single
  // query tile of the tensor-core kernel twice: its second stage's scratch), for
  // segments that a CTA's end cuts. A single sequence shares nothing.
  const size_t most = B * ctx->G;  // query rows of a group
  const int stride = static_cast<int>(std::min<size_t>(k.RB, k.tc ? 2 * most : most));
  const size_t rows = B > 1 ? static_cast<size_t>(ctx->num_sms) * stride + B * c.num_q_heads : 0;
  const size_t sz_int = align256(B * sizeof(int)), sz_group = align256((B + 1) * sizeof(SharedGroup));
  const size_t sz_pre = align256((B + 1) * sizeof(int));
  const size_t sz_rec = align256(rows * c.head_dim * sizeof(float)), sz_ml = align256(rows * sizeof(float2));
  const int own_warps = k.own ? k.own_nw * ctx->num_sms : 0;
  // over the KV heads at most kOwnPieces pieces per warp, and one more per
  // sequence and head; of a sequence at most as many as its chunks make (of
  // max_ctx positions that begin inside a chunk). Every warp reads the entry of
  // its index before it knows how many there are.
  const size_t chunks = (static_cast<size_t>(c.max_ctx) + vattn::kOwnChunk - 1) / vattn::kOwnChunk + 1;
  const size_t pieces =
      k.own ? std::min(static_cast<size_t>(vattn::kOwnPieces) * own_warps / c.num_kv_heads + B + 1,
                       B * ((chunks + vattn::kOwnPiece - 1) / vattn::kOwnPiece))
            : 0;
  const size_t entries = k.own ? std::max(pieces, static_cast<size_t>(own_warps) / c.num_kv_heads + 1) : 0;
  const size_t own_rows = pieces * c.num_q_heads, sz_piece = align256(entries * sizeof(OwnPiece));
  const size_t sz_orec = align256(own_rows * c.head_dim * sizeof(float)), sz_oml = align256(own_rows * sizeof(float2));
  if (p) {
    SharedWork& w = ctx->shared;
    w.reach = reinterpret_cast<int*>(p); p += 2 * sz_int;
    w.pages_ok = reinterpret_cast<int*>(p); p += sz_int;
    w.group = reinterpret_cast<SharedGroup*>(p); p += sz_group;
    w.stride = stride;
    w.rec = reinterpret_cast<float*>(p); p += sz_rec;
    w.ml = reinterpret_cast<float2*>(p); p += sz_ml;
    w.own_pre = reinterpret_cast<int*>(p); p += sz_pre;
    w.own_next = reinterpret_cast<int*>(p); p += 256;
    w.own_piece = reinterpret_cast<OwnPiece*>(p); p += sz_piece;
    w.own_rec = reinterpret_cast<float*>(p); p += sz_orec;
    w.own_ml = reinterpret_cast<float2*>(p);
    w.own_warps = own_warps;
    w.grid = ctx->num_sms;
    cudaFuncSetAttribute(k.prefix, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(k.smem));
    if (k.own) cudaFuncSetAttribute(k.own, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(k.own_smem));
    if (k.gather)
      cudaFuncSetAttribute(k.gather, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(k.gather_smem));
  }
  return 3 * sz_int + sz_pre + 256 + sz_piece + sz_group + sz_rec + sz_ml + sz_orec + sz_oml;
}

}  // namespace vattn

extern "C" int vattn_shared_dense_decode(vattn_ctx* ctx, const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* page_table, const int32_t* seq_lens,
                                         const int32_t* group_start, const int32_t* prefix_lens, int groups, int batch,
                                         int num_pages, float* out, void* stream) {
  if (!ctx) return VATTN_EINVAL;
  ctx->last_status = VATTN_EINVAL;
  const vattn_config& c = ctx->cfg;
  if (batch < 0 || batch > c.max_batch || groups < 0 || groups > c.max_batch || num_pages < 1) return VATTN_EINVAL;
  if (batch > 0 && groups == 0) return VATTN_EINVAL;
  if (batch == 0) {
    ctx->last_launches = 0;
    return ctx->last_status = VATTN_OK;
  }
  if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !group_start || !prefix_lens || !out)
    return VATTN_EINVAL;
  if (!vattn::aligned16(q) || !vattn::aligned16(k_cache) || !vattn::aligned16(v_cache)) return VATTN_EINVAL;
  if (!vattn::aligned_to(4, page_table, seq_lens, group_start, prefix_lens, out)) return VATTN_EINVAL;
  vattn::DeviceScope scope(ctx->device);
  if (!scope.ok) return ctx->last_status = VATTN_ECUDA;
  SharedParams P;
  vattn::fill_common(ctx, &P.D, batch);
  P.D.num_pages = num_pages;
  P.D.dense = 1;
  P.D.proxy = VATTN_EXACT;
  if (const int rc = vattn::cache_ptrs(c, &k_cache, &v_cache)) return ctx->last_status = rc;
  if (static_cast<unsigned long long>(num_pages) * c.num_kv_heads * static_cast<unsigned long long>(c.page_size) >
      0x7FFFFFFFull)
    return VATTN_EINVAL;  // row coordinates are 32-bit
  P.D.q = q;
  P.D.k = k_cache;
  P.D.v = v_cache;
  P.D.page_table = page_table;
  P.D.seq_lens = seq_lens;
  P.D.out = out;
  const SharedKernels k = pick(ctx);
  P.W = ctx->shared;
  P.group_start = group_start;
  P.prefix_lens = prefix_lens;
  P.groups = groups;
  P.RB = k.RB;
  P.KT = k.KT;
  P.own_warps = ctx->shared.own_warps;
  // The tensor-core kernel reads a prefix at the gather's rate, and over the host
  // link every byte counts: two sequences are enough. The fp32 kernel takes as
  // long as the gather takes for 4.7, 3.7 and 2.2 sequences with 1, 4 and 8
  // query heads per KV head (16384 keys x 8 heads, d = 128: 91 to 94 us against
  // 19.5, 24.5 and 41 us a sequence; both grow with the keys).
  P.min_reach = k.tc || P.D.kv_host ? 2 : ctx->G < 4 ? 5 : ctx->G < 8 ? 4 : 3;
  if (!k.own && !P.D.kv_host)
    if (const int rc = vattn::encode_row_maps(c, k_cache, v_cache, num_pages, &P.D)) return ctx->last_status = rc;
  if (k.tc)
    if (const int rc = encode_tile_maps(c, ctx->G, q, k_cache, v_cache, batch, num_pages, &P))
      return ctx->last_status = rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int launches = 0;
  const int prep_warps = vattn::kSharedPrepThreads / 32;
  vattn::launch(vattn::k_shared_prep, dim3((batch + groups + prep_warps - 1) / prep_warps + 2),
                dim3(vattn::kSharedPrepThreads), 0, st, P, &launches);
  vattn::launch(k.prefix, dim3(ctx->num_sms), dim3(k.threads), k.smem, st, P, &launches);
  if (k.own)
    vattn::launch(k.own, dim3(ctx->num_sms), dim3(k.own_nw * 32), k.own_smem, st, P, &launches);
  else
    vattn::launch(k.gather, dim3(ctx->gather_grid), dim3(k.gather_threads), k.gather_smem, st, P.D, &launches);
  // as many warps per row as keep within 32 warps per SM (64: 3 to 4 us more)
  const int rows = batch * c.num_q_heads;
  int w = 3;
  while (w > 0 && (rows << w) > 32 * ctx->num_sms) w--;
  const int per = vattn::kSharedCombWarps >> w;
  vattn::launch(k.combine[w], dim3((rows + per - 1) / per), dim3(vattn::kSharedCombWarps * 32), 0, st, P, &launches);
  return vattn::finish(ctx, launches);
}
