// C ABI of the slots' 8-bit KV caches: argument checks, the handle's error word
// and the launches of kv8_rw.cu and kv8_attend.cu.
#include <cmath>
#include <memory>
#include <new>

#include "handle.h"
#include "kv8.cuh"
#include "strata_window.h"

using namespace strata;

struct strata_kv8 {
  strata_kv8_desc desc;
  int device = 0, nsm = 0;
  Kv8Dev C{};  // layer 0
  Kv8Maps maps{};
  void* ws = nullptr;
  long long ws_bytes = 0;
};

namespace {

void free_kv8(strata_kv8* h) {
  if (!h) return;
  if (h->ws) {
    DeviceScope on(h->device);
    cudaFree(h->ws);
  }
  delete h;
}

strata_status check_desc(const strata_kv8_desc* d) {
  if (!d) return STRATA_EINVAL;
  if (d->n_layers < 1 || d->n_slots < 1 || d->heads < 1 || d->kv_heads < 1 || d->max_ctx < 1) return STRATA_EINVAL;
  if (d->heads % d->kv_heads != 0) return STRATA_EINVAL;
  if (d->format != STRATA_KV8_E4M3 && d->format != STRATA_KV8_INT8) return STRATA_EINVAL;
  if (d->head_dim != 64 && d->head_dim != 128) return STRATA_EUNSUPPORTED;
  if (d->block != 16 && d->block != 32 && d->block != 64 && d->block != 128) return STRATA_EUNSUPPORTED;
  if (d->heads > 1024 || d->heads / d->kv_heads > 128 || d->max_ctx > (1 << 24)) return STRATA_EUNSUPPORTED;
  // rows of the code arrays are addressed by 31 bits in the attention's copies
  if ((long long)d->n_slots * d->kv_heads > 0x7FFFFFFFLL / d->max_ctx) return STRATA_EUNSUPPORTED;
  return STRATA_OK;
}

long long lines(const strata_kv8_desc& d) { return (long long)d.n_slots * d.kv_heads; }
long long n_blocks(const strata_kv8_desc& d) { return ((long long)d.max_ctx + d.block - 1) / d.block; }

// Codes as [layers][n_slots kv_heads max_ctx][head_dim] bytes in boxes of 64
// rows; a row is one swizzle span.  The encoder is the driver's, found at run
// time so that the library loads where there is no driver.
bool make_map(CUtensorMap* map, uint8_t* base, const strata_kv8_desc& d) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return false;
  const cuuint64_t rows = (cuuint64_t)lines(d) * d.max_ctx;
  const cuuint64_t dims[3] = {(cuuint64_t)d.head_dim, rows, (cuuint64_t)d.n_layers};
  const cuuint64_t strides[2] = {(cuuint64_t)d.head_dim, rows * d.head_dim};
  const cuuint32_t box[3] = {(cuuint32_t)d.head_dim, 64, 1}, step[3] = {1, 1, 1};
  return reinterpret_cast<Encode>(fn)(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, step,
                                      CU_TENSOR_MAP_INTERLEAVE_NONE,
                                      d.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                      CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// The part of a call's checks that the three calls share.  *skip: nothing to do.
strata_status check_call(const strata_kv8* h, int32_t layer, int32_t dtype, const strata_kv8_rows* r, bool* skip) {
  *skip = false;
  if (!h || !r || layer < 0 || layer >= h->desc.n_layers) return STRATA_EINVAL;
  if (dtype < STRATA_F32 || dtype > STRATA_BF16) return STRATA_EINVAL;
  if (r->n_seq < 0 || r->n_rows < 0 || r->max_rows < 0) return STRATA_EINVAL;
  if (r->n_seq > kKv8MaxSeq || r->n_rows > (1 << 28)) return STRATA_EUNSUPPORTED;
  if (r->n_seq == 0 || r->n_rows == 0 || r->max_rows == 0) {
    *skip = true;
    return STRATA_OK;
  }
  return r->row_start && r->slot && r->length ? STRATA_OK : STRATA_EINVAL;
}

strata_status check_values(const void* p, long long stride, int width, int dtype) {
  const int size = dtype == STRATA_F32 ? 4 : 2;
  if (!p || reinterpret_cast<uintptr_t>(p) % 16 != 0 || stride < width || stride > (1LL << 40) ||
      (stride * size) % 16 != 0)
    return STRATA_EINVAL;
  return STRATA_OK;
}

Kv8Dev layer_dev(const strata_kv8* h, int layer) {
  Kv8Dev C = h->C;
  const long long codes = lines(h->desc) * h->desc.max_ctx * h->desc.head_dim * layer;
  const long long exps = lines(h->desc) * C.n_blocks * layer;
  C.k += codes, C.v += codes, C.k_exp += exps, C.v_exp += exps;
  return C;
}

Kv8Rows rows_dev(const strata_kv8_rows* r) {
  return {r->n_seq, r->n_rows, r->max_rows < r->n_rows ? r->max_rows : r->n_rows, r->row_start, r->slot, r->length};
}

// The part of the workspace that starts at zero: the error word and the joins' counters.
bool clear(const strata_kv8* h) {
  return cudaMemset(h->ws, 0, (size_t)kv8_attend_zeroed(h->nsm)) == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess;
}

strata_status launched(cudaError_t e) {
  if (e == cudaSuccess) return STRATA_OK;
  cudaGetLastError();
  return e == cudaErrorNotSupported ? STRATA_EUNSUPPORTED : STRATA_ECUDA;
}

}  // namespace

extern "C" {

strata_status strata_kv8_create(const strata_kv8_desc* desc, const strata_kv8_cache* cache, strata_kv8** out) {
  if (!out) return STRATA_EINVAL;
  *out = nullptr;
  const strata_status st = check_desc(desc);
  if (st != STRATA_OK) return st;
  if (!cache || !cache->k || !cache->v || !cache->k_exp || !cache->v_exp) return STRATA_EINVAL;
  if (reinterpret_cast<uintptr_t>(cache->k) % 128 != 0 || reinterpret_cast<uintptr_t>(cache->v) % 128 != 0)
    return STRATA_EINVAL;
  if (fault_is("alloc")) return STRATA_ENOMEM;
  strata_kv8* h = new (std::nothrow) strata_kv8();
  if (!h) return STRATA_ENOMEM;
  h->desc = *desc;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->nsm, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) {
    cudaGetLastError();
    free_kv8(h);
    return STRATA_ECUDA;
  }
  if (setup_kv8_attend(desc->head_dim, desc->format) != cudaSuccess || !make_map(&h->maps.k, cache->k, *desc) ||
      !make_map(&h->maps.v, cache->v, *desc)) {
    cudaGetLastError();
    free_kv8(h);
    return STRATA_ECUDA;
  }
  h->ws_bytes = kv8_attend_workspace(h->nsm, desc->head_dim);
  if (cudaMalloc(&h->ws, (size_t)h->ws_bytes) != cudaSuccess) {
    cudaGetLastError();
    free_kv8(h);
    return STRATA_ENOMEM;
  }
  if (!clear(h)) {
    cudaGetLastError();
    free_kv8(h);
    return STRATA_ECUDA;
  }
  Kv8Dev& C = h->C;
  C.k = cache->k, C.v = cache->v, C.k_exp = cache->k_exp, C.v_exp = cache->v_exp;
  C.n_slots = desc->n_slots, C.heads = desc->heads, C.kv_heads = desc->kv_heads;
  C.head_dim = desc->head_dim, C.max_ctx = desc->max_ctx, C.format = desc->format;
  C.n_blocks = (int)n_blocks(*desc);
  C.block_log2 = desc->block == 16 ? 4 : desc->block == 32 ? 5 : desc->block == 64 ? 6 : 7;
  C.err = static_cast<unsigned*>(h->ws);
  *out = h;
  return STRATA_OK;
}

strata_status strata_kv8_append(strata_kv8* h, int32_t layer, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, int32_t dtype, const strata_kv8_rows* rows, void* cuda_stream) {
  bool skip;
  strata_status st = check_call(h, layer, dtype, rows, &skip);
  if (st != STRATA_OK || skip) return st;
  const int width = h->desc.kv_heads * h->desc.head_dim;
  if ((st = check_values(k, k_stride, width, dtype)) != STRATA_OK) return st;
  if ((st = check_values(v, v_stride, width, dtype)) != STRATA_OK) return st;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) return launched(cudaErrorInvalidDevice);
  return launched(launch_kv8_append(layer_dev(h, layer), rows_dev(rows), k, k_stride, v, v_stride, dtype,
                                    static_cast<cudaStream_t>(cuda_stream)));
}

strata_status strata_kv8_read(strata_kv8* h, int32_t layer, void* k, int64_t k_stride, void* v, int64_t v_stride,
                              int32_t dtype, const strata_kv8_rows* rows, void* cuda_stream) {
  bool skip;
  strata_status st = check_call(h, layer, dtype, rows, &skip);
  if (st != STRATA_OK || skip) return st;
  const int width = h->desc.kv_heads * h->desc.head_dim;
  if ((st = check_values(k, k_stride, width, dtype)) != STRATA_OK) return st;
  if ((st = check_values(v, v_stride, width, dtype)) != STRATA_OK) return st;
  if (k == v) return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) return launched(cudaErrorInvalidDevice);
  return launched(launch_kv8_read(layer_dev(h, layer), rows_dev(rows), k, k_stride, v, v_stride, dtype,
                                  static_cast<cudaStream_t>(cuda_stream)));
}

strata_status strata_kv8_attend(strata_kv8* h, int32_t layer, const void* q, int64_t q_stride, void* out,
                                int64_t out_stride, int32_t dtype, float scale, const strata_kv8_rows* rows,
                                void* cuda_stream) {
  bool skip;
  strata_status st = check_call(h, layer, dtype, rows, &skip);
  if (st != STRATA_OK || skip) return st;
  const int width = h->desc.heads * h->desc.head_dim;
  if ((st = check_values(q, q_stride, width, dtype)) != STRATA_OK) return st;
  if ((st = check_values(out, out_stride, width, dtype)) != STRATA_OK) return st;
  if (q == out || !std::isfinite(scale)) return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) return launched(cudaErrorInvalidDevice);
  st = launched(launch_kv8_attend(layer_dev(h, layer), rows_dev(rows), h->maps, layer, h->ws, h->nsm, q, q_stride, out,
                                  out_stride, dtype, scale, static_cast<cudaStream_t>(cuda_stream)));
  if (st == STRATA_OK && fault_is("overlap"))  // what two calls at once may leave: joins that are not through
    st = launched(cudaMemsetAsync(static_cast<char*>(h->ws) + 256, 1, (size_t)h->nsm * 4,
                                  static_cast<cudaStream_t>(cuda_stream)));
  return st;
}

strata_status strata_kv8_sync(strata_kv8* h) {
  if (!h) return STRATA_EINVAL;
  DeviceScope on(h->device);
  // The error word and the joins' counters.  On an idle device every counter is back at zero; one that is not (calls
  // that overlapped, a wait that gave up) would spoil the joins of every later call.
  const size_t bytes = (size_t)kv8_attend_zeroed(h->nsm);
  const std::unique_ptr<unsigned[]> state(new (std::nothrow) unsigned[bytes / 4]);
  if (!state) return STRATA_ENOMEM;
  if (!on.ok || cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(state.get(), h->ws, bytes, cudaMemcpyDeviceToHost) != cudaSuccess) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  unsigned err = 0;
  for (size_t i = 0; i < bytes / 4; ++i) err |= state[i];
  if (err == 0) return STRATA_OK;
  if (!clear(h)) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  return STRATA_EDEVICE;
}

strata_status strata_kv8_query(const strata_kv8* h, int64_t* cache_bytes, int64_t* workspace_bytes) {
  if (!h) return STRATA_EINVAL;
  const strata_kv8_desc& d = h->desc;
  if (cache_bytes)
    *cache_bytes = 2LL * d.n_layers * lines(d) * ((long long)d.max_ctx * d.head_dim + n_blocks(d));
  if (workspace_bytes) *workspace_bytes = h->ws_bytes;
  return STRATA_OK;
}

strata_status strata_kv8_destroy(strata_kv8* h) {
  free_kv8(h);
  return STRATA_OK;
}

}  // extern "C"
