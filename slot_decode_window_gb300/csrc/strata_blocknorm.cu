// C ABI and kernel of the norms after and before a block, fused with its gate
// and the residual.
#include <cmath>
#include <new>

#include "handle.h"
#include "kv8.cuh"
#include "strata_window.h"

using namespace strata;

struct strata_blocknorm {
  strata_blocknorm_desc desc;
  int device = 0;
  float* mem = nullptr;  // [2][hidden]: after gain times channel gate, before gain (ones where there is none)
};

namespace {

struct BnArgs {
  const void *x, *y, *gate;
  void *h, *n;
  long long xs, ys, gs, hs, ns;
  const float* par;  // [2][hidden]
  int hidden, after, before, gate_kind, sigmoid;
  float eps, rscale, bscale, inv;
};

// Sum over the CTA, in a fixed order; every thread has it.  `part` is written once per call: two calls take two of them.
__device__ __forceinline__ float cta_sum(float v, float* part, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = (int)(threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// A CTA of at most kMax threads owns a row: kVec 16-byte pieces of it in each thread's registers from the first load to the last store, so that
// x, y and an element gate are read once and h and n written once, with two sums over the CTA between.
// HBM bound in a prompt: 8191 bf16 rows of 4096 with the before norm alone 44 us (90% of the measured rate), with the after norm and a
// channel gate 51 us: the gains, twice a row's bytes, come from L1, and there is a second sum.  The bounds ask for 2048 threads an SM
// (32 registers; at 40, three CTAs of 512, 57.5 us).  Two rows to a CTA 58.8 us, two or four pieces a thread of smaller CTAs no
// better; CTAs that keep the gains in registers and take rows in turn from copies in shared memory 58 us (half the warps).
template <typename T, int kVec, int kMax>
__global__ void __launch_bounds__(kMax, kVec == 1 ? 2048 / kMax : 1) blocknorm_kernel(BnArgs A) {
  constexpr int E = Val<T>::kPer;
  __shared__ float part[2][32];
  const long long row = blockIdx.x;
  const int pieces = A.hidden / E, threads = blockDim.x, warps = threads / 32;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(A.x) + row * A.xs);
  const uint4* y = A.y ? reinterpret_cast<const uint4*>(static_cast<const T*>(A.y) + row * A.ys) : nullptr;
  const uint4* ge = A.gate_kind == STRATA_GATE_ELEMENT
                        ? reinterpret_cast<const uint4*>(static_cast<const T*>(A.gate) + row * A.gs)
                        : nullptr;
  uint4 xr[kVec], yr[kVec], gr[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int p = i * threads + threadIdx.x;
    xr[i] = yr[i] = gr[i] = make_uint4(0, 0, 0, 0);
    if (p < pieces) {
      xr[i] = x[p];
      if (y) yr[i] = y[p];
      if (ge) gr[i] = ge[p];
    }
  }
  float g0 = A.bscale;
  if (A.gate_kind == STRATA_GATE_ROW) {
    const float g = static_cast<const float*>(A.gate)[row];
    g0 *= A.sigmoid ? 1.f / (1.f + expf(-g)) : g;
  }
  float h[kVec][E];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    Val<T>::unpack(yr[i], h[i]);
#pragma unroll
    for (int j = 0; j < E; ++j) sum = fmaf(h[i][j], h[i][j], sum);
  }
  const float* after = A.par;
  const float* before = A.par + A.hidden;
  float r = 1.f;
  if (A.after) r = rsqrtf(cta_sum(sum, part[0], warps) * A.inv + A.eps);
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int p = i * threads + threadIdx.x;
    if (p >= pieces) {  // (its registers are zeros)
#pragma unroll
      for (int j = 0; j < E; ++j) h[i][j] = 0.f;
      continue;
    }
    if (A.after || A.gate_kind == STRATA_GATE_CHANNEL) {  // (one vector: its reads are L1's, for every row)
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        const float4 w = reinterpret_cast<const float4*>(after + p * E)[j / 4];
        h[i][j] *= r * w.x, h[i][j + 1] *= r * w.y, h[i][j + 2] *= r * w.z, h[i][j + 3] *= r * w.w;
      }
    }
    if (ge) {
      float f[E];
      Val<T>::unpack(gr[i], f);
#pragma unroll
      for (int j = 0; j < E; ++j) h[i][j] *= A.sigmoid ? 1.f / (1.f + expf(-f[j])) : f[j];
    }
    float f[E];
    Val<T>::unpack(xr[i], f);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      h[i][j] = y ? fmaf(A.rscale, f[j], g0 * h[i][j]) : A.rscale * f[j];
      sum = fmaf(h[i][j], h[i][j], sum);
    }
    if (A.h) reinterpret_cast<uint4*>(static_cast<T*>(A.h) + row * A.hs)[p] = Val<T>::pack(h[i]);
  }
  if (!A.before) return;
  r = rsqrtf(cta_sum(sum, part[1], warps) * A.inv + A.eps);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int p = i * threads + threadIdx.x;
    if (p >= pieces) break;
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const float4 w = reinterpret_cast<const float4*>(before + p * E)[j / 4];
      h[i][j] *= r * w.x, h[i][j + 1] *= r * w.y, h[i][j + 2] *= r * w.z, h[i][j + 3] *= r * w.w;
    }
    reinterpret_cast<uint4*>(static_cast<T*>(A.n) + row * A.ns)[p] = Val<T>::pack(h[i]);
  }
}

// gain *= gate (through the sigmoid)
__global__ void fold_kernel(float* gain, const float* gate, int sigmoid, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) gain[i] *= sigmoid ? 1.f / (1.f + expf(-gate[i])) : gate[i];
}

template <typename T, int kVec, int kMax>
void launch_vec(const BnArgs& A, unsigned rows, cudaStream_t s) {
  const int pieces = A.hidden / Val<T>::kPer, threads = (pieces + kVec - 1) / kVec;
  blocknorm_kernel<T, kVec, kMax><<<rows, (threads + 31) / 32 * 32, 0, s>>>(A);
}

// One piece a thread where a row has at most 512 of them (a row's loads are all in flight at once either way), and no more warps
// than the pieces fill: their places are other rows' (8191 bf16 rows of 2304 28.3 us, with 512 threads to a row 38.2 us; of 5120
// 62.5 and 82 us; 16384 rows of 512 12.3 us, with 128 threads 16.3 us).  Larger rows take two or four pieces: one piece of up to 1024
// threads is no better (rows of 8192 103 us against 100 us).
template <typename T>
void launch_t(const BnArgs& A, unsigned rows, cudaStream_t s) {
  const int pieces = A.hidden / Val<T>::kPer;
  if (pieces <= 512)
    launch_vec<T, 1, 512>(A, rows, s);
  else if (pieces <= 1024)
    launch_vec<T, 2, 512>(A, rows, s);
  else if (pieces <= 2048)
    launch_vec<T, 4, 512>(A, rows, s);
  else if constexpr (Val<T>::kPer == 4)  // (only f32 rows have more)
    launch_vec<T, 4, 1024>(A, rows, s);
}

void free_blocknorm(strata_blocknorm* h) {
  if (!h) return;
  if (h->mem) {
    DeviceScope on(h->device);
    cudaFree(h->mem);
  }
  delete h;
}

bool rows_ok(const void* p, long long stride, int width, int size) {
  return p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride >= width && stride <= (1LL << 40) &&
         (stride * size) % 16 == 0;
}

}  // namespace

extern "C" {

strata_status strata_blocknorm_create(const strata_blocknorm_desc* d, const float* after_gain, const float* before_gain,
                                      const float* channel_gate, void* cuda_stream, strata_blocknorm** out) {
  if (!out) return STRATA_EINVAL;
  *out = nullptr;
  if (!d || d->hidden < 1 || (d->after != 0 && d->after != 1) || (d->before != 0 && d->before != 1) ||
      (d->sigmoid != 0 && d->sigmoid != 1) || d->gate < STRATA_GATE_NONE || d->gate > STRATA_GATE_ELEMENT)
    return STRATA_EINVAL;
  if (!(d->eps >= 0.f) || std::isinf(d->eps) || !std::isfinite(d->residual_scale) || !std::isfinite(d->block_scale))
    return STRATA_EINVAL;
  if (d->gate == STRATA_GATE_CHANNEL && !channel_gate) return STRATA_EINVAL;
  if (d->hidden % 8 != 0 || d->hidden > 16384) return STRATA_EUNSUPPORTED;
  if (fault_is("alloc")) return STRATA_ENOMEM;
  strata_blocknorm* h = new (std::nothrow) strata_blocknorm();
  float* ones = new (std::nothrow) float[d->hidden];
  if (!h || !ones) {
    delete h;
    delete[] ones;
    return STRATA_ENOMEM;
  }
  h->desc = *d;
  strata_status st = STRATA_OK;
  const size_t row = (size_t)d->hidden * 4;
  if (cudaGetDevice(&h->device) != cudaSuccess)
    st = STRATA_ECUDA;
  else if (cudaMalloc(&h->mem, 2 * row) != cudaSuccess)
    st = STRATA_ENOMEM;
  if (st == STRATA_OK) {
    for (int i = 0; i < d->hidden; ++i) ones[i] = 1.f;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const float* from[2] = {d->after ? after_gain : nullptr, d->before ? before_gain : nullptr};
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 2 && e == cudaSuccess; ++i)
      e = cudaMemcpyAsync(h->mem + (size_t)i * d->hidden, from[i] ? from[i] : ones, row,
                          from[i] ? cudaMemcpyDeviceToDevice : cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess && d->gate == STRATA_GATE_CHANNEL) {
      fold_kernel<<<(d->hidden + 255) / 256, 256, 0, s>>>(h->mem, channel_gate, d->sigmoid, d->hidden);
      e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) st = STRATA_ECUDA;
  }
  delete[] ones;
  if (st != STRATA_OK) {
    cudaGetLastError();
    free_blocknorm(h);
    return st;
  }
  *out = h;
  return STRATA_OK;
}

strata_status strata_blocknorm_forward(strata_blocknorm* h, const void* x, int64_t x_stride, const void* y,
                                       int64_t y_stride, const void* gate, int64_t gate_stride, void* h_out,
                                       int64_t h_stride, void* n_out, int64_t n_stride, int32_t dtype, int32_t T,
                                       void* cuda_stream) {
  if (!h || T < 0 || dtype < STRATA_F32 || dtype > STRATA_BF16) return STRATA_EINVAL;
  if (T == 0) return STRATA_OK;
  const strata_blocknorm_desc& d = h->desc;
  const int size = dtype == STRATA_F32 ? 4 : 2, w = d.hidden;
  if (!rows_ok(x, x_stride, w, size)) return STRATA_EINVAL;
  if (y ? !rows_ok(y, y_stride, w, size) : (d.after || d.gate != STRATA_GATE_NONE)) return STRATA_EINVAL;
  if (h_out ? !rows_ok(h_out, h_stride, w, size) : !d.before) return STRATA_EINVAL;
  if (d.before ? !rows_ok(n_out, n_stride, w, size) : n_out != nullptr) return STRATA_EINVAL;
  if (d.gate == STRATA_GATE_ROW && (!gate || reinterpret_cast<uintptr_t>(gate) % 4 != 0)) return STRATA_EINVAL;
  if (d.gate == STRATA_GATE_ELEMENT && !rows_ok(gate, gate_stride, w, size)) return STRATA_EINVAL;
  if (d.gate <= STRATA_GATE_CHANNEL && gate) return STRATA_EINVAL;
  // an output over x or y row for row, or elsewhere
  const void* o[2] = {h_out, n_out};
  const int64_t os[2] = {h_stride, n_stride};
  if (h_out && h_out == n_out) return STRATA_EINVAL;
  for (int i = 0; i < 2; ++i)
    if (o[i] && ((T > 1 && o[i] == x && os[i] != x_stride) || (T > 1 && o[i] == y && os[i] != y_stride) || o[i] == gate))
      return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  BnArgs A;
  A.x = x, A.y = y, A.gate = gate, A.h = h_out, A.n = n_out;
  A.xs = x_stride, A.ys = y_stride, A.gs = gate_stride, A.hs = h_stride, A.ns = n_stride;
  A.par = h->mem, A.hidden = d.hidden, A.after = d.after, A.before = d.before, A.gate_kind = d.gate;
  A.sigmoid = d.sigmoid, A.eps = d.eps, A.rscale = d.residual_scale, A.bscale = d.block_scale;
  A.inv = 1.f / (float)d.hidden;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (dtype == STRATA_F32)
    launch_t<float>(A, (unsigned)T, s);
  else if (dtype == STRATA_F16)
    launch_t<__half>(A, (unsigned)T, s);
  else
    launch_t<__nv_bfloat16>(A, (unsigned)T, s);
  return cudaGetLastError() == cudaSuccess ? STRATA_OK : STRATA_ECUDA;
}

strata_status strata_blocknorm_destroy(strata_blocknorm* h) {
  free_blocknorm(h);
  return STRATA_OK;
}

}  // extern "C"
