// C ABI of the products with 4-bit matrices: argument checks, the handle's
// layout of the matrices, its workspace and error word.
#include <cmath>
#include <new>

#include "handle.h"
#include "linear.cuh"
#include "strata_window.h"

using namespace strata;

struct strata_linear {
  strata_linear_desc desc;
  int device = 0, nsm = 0, mats = 1, rounded = 0;
  int clusters[3] = {};  // of 2, 4 and 8 CTAs that run at once
  uint8_t* mem = nullptr;  // error word, then the matrices and their rows' powers of two
  unsigned* err = nullptr;
  LinMat w[2] = {};
  void* ws = nullptr;
  long long weight_bytes = 0, ws_bytes = 0;
};

namespace {

void free_linear(strata_linear* h) {
  if (!h) return;
  if (h->mem) {
    DeviceScope on(h->device);
    cudaFree(h->mem);
    cudaFree(h->ws);
  }
  delete h;
}

strata_status check_desc(const strata_linear_desc* d) {
  if (!d || d->n < 1 || d->in < 1 || d->out < 1 || d->max_rows < 1) return STRATA_EINVAL;
  if (d->bits != 4 || d->block != 32) return STRATA_EUNSUPPORTED;
  if (d->in % kLinStep != 0 || d->out % kLinTile != 0) return STRATA_EUNSUPPORTED;
  if (d->n > 1024 || d->in > 65536 || d->out > (1 << 22) || d->max_rows > (1 << 20)) return STRATA_EUNSUPPORTED;
  if ((long long)d->n * (d->out / kLinTile) > 0x7FFFFFFFLL) return STRATA_EUNSUPPORTED;
  return STRATA_OK;
}

bool mat_ok(const strata_qmat& q) {
  return q.codes && q.scale && q.min && reinterpret_cast<uintptr_t>(q.scale) % 2 == 0 &&
         reinterpret_cast<uintptr_t>(q.min) % 2 == 0;
}

bool rows_ok(const void* p, long long stride, int width, int size) {
  return p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride >= width && stride <= (1LL << 40) &&
         (stride * size) % 16 == 0;
}

}  // namespace

extern "C" {

strata_status strata_linear_create(const strata_linear_desc* desc, const strata_qmat* weight, const strata_qmat* up,
                                   void* cuda_stream, strata_linear** out) {
  if (!out) return STRATA_EINVAL;
  *out = nullptr;
  const strata_status st = check_desc(desc);
  if (st != STRATA_OK) return st;
  if (!weight || !mat_ok(*weight) || (up && !mat_ok(*up))) return STRATA_EINVAL;
  if (fault_is("alloc")) return STRATA_ENOMEM;
  strata_linear* h = new (std::nothrow) strata_linear();
  if (!h) return STRATA_ENOMEM;
  h->desc = *desc;
  h->mats = up ? 2 : 1;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->nsm, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) {
    cudaGetLastError();
    free_linear(h);
    return STRATA_ECUDA;
  }
  const long long packed = linear_packed_bytes(desc->n, desc->in, desc->out);
  const long long rows = ((long long)desc->n * desc->out * 4 + 255) / 256 * 256;
  h->weight_bytes = h->mats * packed;
  // (2 KB behind: the few-row kernel reads up to three tiles' steps past the last tile)
  if (cudaMalloc(&h->mem, (size_t)(256 + h->mats * (packed + rows) + 2048)) != cudaSuccess) {
    cudaGetLastError();
    free_linear(h);
    return STRATA_ENOMEM;
  }
  h->err = reinterpret_cast<unsigned*>(h->mem);
  if (desc->n > 1 || desc->max_rows > kLinFewRows) {
    h->ws_bytes = linear_many_workspace(desc->in, desc->max_rows);
    if (cudaMalloc(&h->ws, (size_t)h->ws_bytes) != cudaSuccess) {
      cudaGetLastError();
      free_linear(h);
      return STRATA_ENOMEM;
    }
    if (setup_linear_many(h->clusters) != cudaSuccess) {
      cudaGetLastError();
      free_linear(h);
      return STRATA_ECUDA;
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaMemsetAsync(h->mem, 0, 256, s);
  for (int m = 0; m < h->mats && e == cudaSuccess; ++m) {
    const strata_qmat& q = m ? *up : *weight;
    uint8_t* to = h->mem + 256 + m * (packed + rows);
    float* undo = reinterpret_cast<float*>(to + packed);
    h->w[m] = {to, undo};
    e = launch_linear_pack(q.codes, q.scale, q.min, desc->n, desc->in, desc->out, to, undo, s);
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    free_linear(h);
    return STRATA_ECUDA;
  }
  *out = h;
  return STRATA_OK;
}

strata_status strata_linear_forward(strata_linear* h, const void* x, int64_t x_stride, void* y, int64_t y_stride,
                                    int32_t dtype, int32_t T, const int32_t* offsets, void* cuda_stream) {
  if (!h || T < 0 || dtype < STRATA_F32 || dtype > STRATA_BF16) return STRATA_EINVAL;
  const strata_linear_desc& d = h->desc;
  if (T > d.max_rows || (d.n > 1 && !offsets) || reinterpret_cast<uintptr_t>(offsets) % 4 != 0) return STRATA_EINVAL;
  if (T == 0) return STRATA_OK;
  const int size = dtype == STRATA_F32 ? 4 : 2;
  if (!rows_ok(x, x_stride, d.in, size) || !rows_ok(y, y_stride, d.out, size) || x == y) return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  LinArgs A{};
  A.w[0] = h->w[0], A.w[1] = h->w[1];
  A.n = d.n, A.in = d.in, A.out = d.out, A.glu = h->mats == 2, A.rounded = h->rounded;
  A.x = x, A.y = y, A.xs = x_stride, A.ys = y_stride, A.dtype = dtype, A.T = T, A.offsets = offsets, A.err = h->err;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool few = linear_few_rows(A, h->nsm);
  if ((few ? launch_linear_few(A, h->nsm, s) : launch_linear_many(A, h->ws, d.max_rows, h->nsm, h->clusters, s)) != cudaSuccess) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  return STRATA_OK;
}

strata_status strata_linear_round_weights(strata_linear* h, int32_t on) {
  if (!h || (on != 0 && on != 1)) return STRATA_EINVAL;
  h->rounded = on;
  return STRATA_OK;
}

strata_status strata_linear_sync(strata_linear* h) {
  if (!h) return STRATA_EINVAL;
  DeviceScope on(h->device);
  unsigned err = 0;
  if (!on.ok || cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(&err, h->err, sizeof(err), cudaMemcpyDeviceToHost) != cudaSuccess) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  if (err == 0) return STRATA_OK;
  if (cudaMemset(h->err, 0, sizeof(err)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  return STRATA_EDEVICE;
}

strata_status strata_linear_query(const strata_linear* h, int64_t* weight_bytes, int64_t* workspace_bytes) {
  if (!h) return STRATA_EINVAL;
  if (weight_bytes) *weight_bytes = h->weight_bytes;
  if (workspace_bytes) *workspace_bytes = h->ws_bytes;
  return STRATA_OK;
}

strata_status strata_linear_destroy(strata_linear* h) {
  free_linear(h);
  return STRATA_OK;
}

}  // extern "C"
