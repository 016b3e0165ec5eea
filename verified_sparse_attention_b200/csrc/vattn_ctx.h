// The context behind the C ABI and the host helpers that its entry points share.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <vector>

#include "vattn.h"
#include "vattn_device.cuh"

namespace vattn {

// One group of a shared-prefix decode; record [groups] holds the totals.
struct alignas(16) SharedGroup {
  int b0, size;            // its sequences
  int prefix;
  int tiles;               // key tiles of the prefix (0: not shared)
  long long tile0, row0;   // key tiles (of every row block and head) and record rows before it
};

// A piece of a sequence's own positions [start, n): `chunks` chunks of 16 from
// position `pos` on. id: its index times Hkv, plus the KV head.
struct alignas(16) OwnPiece {
  int b, pos, chunks, start, n, id, pad[2];
};

// Workspace of the shared-prefix decode (see vattn_shared.cuh).
struct SharedWork {
  int* reach = nullptr;           // [2 max_batch] scratch of k_shared_prep's last two CTAs
  int* pages_ok = nullptr;        // [max_batch] per group: the prefix's pages are valid
  SharedGroup* group = nullptr;   // [max_batch + 1]
  int stride = 0;                 // record rows of a CTA of the prefix kernel
  float* rec = nullptr;           // [record rows][D]
  float2* ml = nullptr;           // [record rows] (maximum in log2 units, weight sum)
  int* own_pre = nullptr;         // [max_batch + 1] prefix sum of own pieces (of one KV head) over sequences
  int* own_next = nullptr;        // pieces (times Hkv) handed out
  OwnPiece* own_piece = nullptr;  // [pieces]
  float* own_rec = nullptr;       // [pieces][Hkv][G][D]
  float2* own_ml = nullptr;       // [pieces][Hkv][G]
  int own_warps = 0;              // warps of k_shared_own (0: not used)
  int grid = 0;                   // CTAs of the prefix kernel
};

}  // namespace vattn

struct vattn_ctx {
  vattn_config cfg;
  int device = 0;
  int num_sms = 0;
  int G = 1;
  int units_max = 0;
  int score_grid = 0;
  bool score_tma = false;   // contiguous cache: the bulk-copy score pass
  size_t score_smem = 0;
  int gather_grid = 0;     // CTAs of each gather launch
  int CD = 0, CS = 0;      // record producers (warps) of the det/dense and sample gathers
  size_t gather_smem = 0;   // gathers (all modes)
  int gather_threads = 0;
  int draw_splits = 1;
  size_t ws_bytes = 0;
  void* ws = nullptr;
  // carved workspace
  vattn::UnitInfo* info = nullptr;
  float* qbar = nullptr;
  float* qsel = nullptr;
  int* dims = nullptr;
  unsigned* ordk = nullptr;
  unsigned* hist = nullptr;
  float* pscore = nullptr;
  int* num_need = nullptr;
  long long* prefix = nullptr;
  unsigned* gcnt = nullptr;
  long long* pre_det = nullptr;
  long long* pre_samp = nullptr;
  float* rec_det = nullptr;
  float* rec_samp = nullptr;
  unsigned* err = nullptr;
  // shared-prefix decode
  vattn::SharedWork shared;
  // state
  int last_status = VATTN_OK;
  int last_launches = 0;
  double cached_delta = -1.0;
  double cached_z = 0.0;
  // timing of the score pass
  int timing = 0;            // period (0: off)
  long long timing_calls = 0;
  std::vector<cudaEvent_t> ev_start, ev_stop;
  size_t ev_used = 0;
};

namespace vattn {

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Every one of the arrays starts at an element of `size` bytes (a null pointer does).
template <typename... P>
bool aligned_to(size_t size, const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) % size == 0) && ...);
}

// The driver's tensor-map encoder, reached through the runtime (the library
// does not link the driver library itself).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// Row maps of the K and V caches for the gathers: a 2-D [rows][d] view with
// rows = num_pages * Hkv * page_size, one-row boxes of all d columns.
inline int encode_row_maps(const vattn_config& c, const void* k, const void* v, int num_pages, DevParams* P) {
  const unsigned long long rows =
      static_cast<unsigned long long>(num_pages) * c.num_kv_heads * static_cast<unsigned long long>(c.page_size);
  if (rows > 0x7FFFFFFFull) return VATTN_EINVAL;  // row coordinates are 32-bit
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return VATTN_ECUDA;
  const cuuint64_t esz = c.dtype == VATTN_BF16 ? 2 : 4;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.head_dim), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.head_dim) * esz};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(c.head_dim), 1u};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapDataType dt =
      c.dtype == VATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  for (int i = 0; i < 2; i++) {
    const CUresult r = fn(i ? &P->tmv : &P->tmk, dt, 2, const_cast<void*>(i ? v : k), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return VATTN_ECUDA;
  }
  if (c.dtype == VATTN_BF16) {  // the tensor-core gathers' swizzled half-row boxes
    const cuuint32_t hbox[2] = {64u, 1u};
    for (int i = 0; i < 2; i++) {
      const CUresult r = fn(i ? &P->tmv_sw : &P->tmk_sw, dt, 2, const_cast<void*>(i ? v : k), dims, strides, hbox,
                            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
      if (r != CUDA_SUCCESS) return VATTN_ECUDA;
    }
  }
  return VATTN_OK;
}

// Device address of a cache in page-locked host memory (nullptr if `p` is not
// such memory).
inline const void* host_cache_device_ptr(const void* p) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  if (a.type != cudaMemoryTypeHost || a.devicePointer == nullptr) return nullptr;
  return static_cast<const char*>(a.devicePointer) +
         (static_cast<const char*>(p) - static_cast<const char*>(a.hostPointer ? a.hostPointer : p));
}

// The caches as the kernels address them (host-resident caches mapped to
// their device addresses); VATTN_EINVAL if a host-resident cache is not
// page-locked.
inline int cache_ptrs(const vattn_config& c, const void** k, const void** v) {
  if (c.kv_location != VATTN_KV_HOST) return VATTN_OK;
  const void* dk = host_cache_device_ptr(*k);
  const void* dv = host_cache_device_ptr(*v);
  if (!dk || !dv) return VATTN_EINVAL;
  *k = dk;
  *v = dv;
  return VATTN_OK;
}

inline void fill_common(const vattn_ctx* ctx, DevParams* P, int batch) {
  memset(P, 0, sizeof(*P));
  const vattn_config& c = ctx->cfg;
  P->Hq = c.num_q_heads;
  P->Hkv = c.num_kv_heads;
  P->G = ctx->G;
  P->D = c.head_dim;
  P->pps = (c.max_ctx + c.page_size - 1) / c.page_size;
  P->ps = c.page_size;
  P->ps_magic = ~0ull / static_cast<unsigned long long>(c.page_size) + 1ull;
  P->max_ctx = c.max_ctx;
  P->batch = batch;
  P->units = batch * c.num_kv_heads;
  P->proxy = c.proxy;
  P->rank = c.proxy_rank;
  P->kv_host = c.kv_location == VATTN_KV_HOST;
  P->scale = static_cast<float>(1.0 / sqrt(static_cast<double>(c.head_dim)));
  P->info = ctx->info;
  P->qbar = ctx->qbar;
  P->qsel = ctx->qsel;
  P->dims = ctx->dims;
  P->ordk = ctx->ordk;
  P->hist = ctx->hist;
  P->pscore = ctx->pscore;
  P->num_need = ctx->num_need;
  P->prefix = ctx->prefix;
  P->gcnt = ctx->gcnt;
  P->pre_det = ctx->pre_det;
  P->pre_samp = ctx->pre_samp;
  P->rec_det = ctx->rec_det;
  P->rec_samp = ctx->rec_samp;
  P->CD = ctx->CD;
  P->CS = ctx->CS;
  P->err = ctx->err;
}

// Launch with programmatic dependent launch: the kernel may be scheduled while
// its predecessor on the stream drains; it waits (griddepcontrol.wait) before
// reading the predecessor's results.
template <typename Params>
void launch(void (*kern)(Params), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Params& P, int* count) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kern, P);
  (*count)++;
}

inline int finish(vattn_ctx* ctx, int launches) {
  ctx->last_launches = launches;
  const cudaError_t e = cudaGetLastError();
  ctx->last_status = e == cudaSuccess ? VATTN_OK : VATTN_ECUDA;
  return ctx->last_status;
}

// Bytes of the shared-prefix decode's scratch, set out from `p` when given
// (vattn_shared.cu). Nothing in it is kept from one call to the next.
size_t shared_workspace(vattn_ctx* ctx, char* p);

// The given device current for the lifetime of the object, whichever was before.
struct DeviceScope {
  int before = -1;
  bool ok = false;
  explicit DeviceScope(int device) {
    int now = -1;
    if (cudaGetDevice(&now) != cudaSuccess) return;
    if (now != device) {
      if (cudaSetDevice(device) != cudaSuccess) return;
      before = now;
    }
    ok = true;
  }
  ~DeviceScope() {
    if (before >= 0) cudaSetDevice(before);
  }
  DeviceScope(const DeviceScope&) = delete;
  DeviceScope& operator=(const DeviceScope&) = delete;
};

}  // namespace vattn
