// C ABI and kernel of the per-head norms of queries and keys with the rotation
// by position.
#include <cmath>
#include <new>

#include "handle.h"
#include "kv8.cuh"
#include "strata_window.h"

using namespace strata;

struct strata_qknorm {
  strata_qknorm_desc desc;
  int device = 0, nsm = 0;
  void* mem = nullptr;
  float* gain = nullptr;               // [2][head_dim]: q, k (ones where the caller gave none)
  unsigned long long* turn = nullptr;  // [rotary_dim / 2] freq / 2 pi as a fraction of 2^64
};

namespace {

struct QkArgs {
  const void *q, *k;
  void *q_out, *k_out;
  long long qs, ks, qos, kos;
  const float* gain;
  const unsigned long long* turn;
  const int* position;
  int T, heads, total, rotary, norm, per_cta, groups;
  float eps;
};

constexpr int kQkThreads = 128;
constexpr int kQkBatch = 1;  // 16-byte accesses a thread has in flight

// A CTA owns `per_cta` heads of a row (of q's and then k's).  Its threads form the row's angles once, an angle a
// thread, in shared memory; then a warp takes kGroup heads at a time: E neighbouring dims of a head in a lane,
// 32 / kGroup lanes to a head, 16 bytes a lane wherever the rotation's halves allow it, kQkBatch accesses in flight.
// The head's mean is a sum over its lanes; the half-apart partner of a dim is in another lane at the same place, one
// shuffle away (half a rotary_dim is a multiple of E).
// The angle in turns is position * turn mod 2^64: the product wraps to the exact fraction, its top 32 bits go to
// sincospi.
// HBM bound in a prompt.  8191 rows of 32 + 8 bf16 heads: with the angles and gains in every warp's registers (91 of
// them, six times the angles) 74 us; in shared memory 64 us with four accesses a thread in flight (79 registers), 45 us
// with one and twelve CTAs an SM (40 registers, of which half-apart pairs spill 4 to 28 bytes in seven variants), which is
// what is here (39.4 us called in turn, 63% of the measured HBM rate).
template <typename T, int kHd, int E, bool kInter>
__global__ void __launch_bounds__(kQkThreads, 12) qknorm_kernel(QkArgs A) {
  constexpr int kLanes = kHd / E, kGroup = 32 / kLanes, kWarps = kQkThreads / 32;
  __shared__ float2 turn[kHd / 2];        // cosine and sine of each pair's angle
  __shared__ alignas(16) float gain[2][kHd];
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const long long row = blockIdx.x / A.groups;
  const int h_end = min(A.total, (int)(blockIdx.x % A.groups + 1) * A.per_cta);
  const int first = (int)(blockIdx.x % A.groups) * A.per_cta + (threadIdx.x >> 5) * kGroup;
  const int d0 = sub * E, half = A.rotary >> 1;

  struct alignas(sizeof(T) * E < 16 ? sizeof(T) * E : 16) Vec { T v[E]; };  // rows are 16-byte aligned
  Vec x[kQkBatch];
  auto fetch = [&](int h) {
#pragma unroll
    for (int b = 0; b < kQkBatch; ++b) {
      const int hh = h + b * kWarps * kGroup + lane / kLanes;
      if (hh < h_end) {
        const T* src = hh < A.heads ? static_cast<const T*>(A.q) + row * A.qs + (long long)hh * kHd
                                    : static_cast<const T*>(A.k) + row * A.ks + (long long)(hh - A.heads) * kHd;
        x[b] = reinterpret_cast<const Vec*>(src)[sub];
      } else {
        x[b] = Vec{};
      }
    }
  };
  fetch(first);  // on its way while the angles are formed
  const unsigned long long pos = (unsigned long long)(long long)A.position[row];
  for (int i = threadIdx.x; i < half; i += kQkThreads) {
    float2 t;
    sincospif((float)(int)((pos * A.turn[i]) >> 32) * 0x1p-31f, &t.y, &t.x);
    turn[i] = t;
  }
  if (A.norm)
    for (int i = threadIdx.x; i < 2 * kHd; i += kQkThreads) (&gain[0][0])[i] = A.gain[i];
  __syncthreads();

  float cs[E], sn[E];
  int partner = lane;
#pragma unroll
  for (int i = 0; i < E; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (d0 < A.rotary) {  // (rotary_dim is a multiple of E or of 2)
    if constexpr (kInter) {
#pragma unroll
      for (int i = 0; i < E; i += 2)
        if (d0 + i < A.rotary) cs[i] = turn[(d0 + i) >> 1].x, sn[i] = turn[(d0 + i) >> 1].y;
    } else {
      const bool upper = d0 >= half;
      partner = upper ? lane - half / E : lane + half / E;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float2 t = turn[d0 + i - (upper ? half : 0)];
        cs[i] = t.x, sn[i] = upper ? t.y : -t.y;  // first of the pair: a cos - b sin; second: b cos + a sin
      }
    }
  }

  constexpr int kStep = kQkBatch * kWarps * kGroup;
  for (int h = first; h < h_end; h += kStep) {
    if (h > first) fetch(h);
#pragma unroll
    for (int b = 0; b < kQkBatch; ++b) {
      if (h + b * kWarps * kGroup >= h_end) break;
      const int hh = h + b * kWarps * kGroup + lane / kLanes;
      const bool is_q = hh < A.heads;
      float f[E];
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = Val<T>::up(x[b].v[i]);
      if (A.norm) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(f[i], f[i], s);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        const float r = rsqrtf(s * (1.f / kHd) + A.eps);  // (2 ulp)
        const float* g = gain[is_q ? 0 : 1] + d0;
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = f[i] * r * g[i];
      }
      if (A.rotary > 0) {
        if constexpr (kInter) {
#pragma unroll
          for (int i = 0; i < E; i += 2) {
            const float a = f[i], c = f[i + 1];
            if (d0 + i < A.rotary) {
              f[i] = a * cs[i] - c * sn[i];
              f[i + 1] = a * sn[i] + c * cs[i];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const float o = __shfl_sync(0xFFFFFFFFu, f[i], partner);
            if (d0 < A.rotary) f[i] = f[i] * cs[i] + o * sn[i];
          }
        }
      }
      if (hh < h_end) {
        Vec y;
#pragma unroll
        for (int i = 0; i < E; ++i) y.v[i] = Val<T>::down(f[i]);
        T* dst = is_q ? static_cast<T*>(A.q_out) + row * A.qos + (long long)hh * kHd
                      : static_cast<T*>(A.k_out) + row * A.kos + (long long)(hh - A.heads) * kHd;
        reinterpret_cast<Vec*>(dst)[sub] = y;
      }
    }
  }
}

template <typename T, int kHd, int E>
void launch_e(const QkArgs& A, int interleaved, unsigned grid, cudaStream_t s) {
  if (interleaved)
    qknorm_kernel<T, kHd, E, true><<<grid, kQkThreads, 0, s>>>(A);
  else
    qknorm_kernel<T, kHd, E, false><<<grid, kQkThreads, 0, s>>>(A);
}

// E: 16 bytes of a lane where the rotation's halves are a multiple of them, else the head over all 32 lanes.
template <typename T, int kHd>
void launch_h(const QkArgs& A, int interleaved, unsigned grid, cudaStream_t s) {
  constexpr int kWide = kHd == 256 ? 8 : 16 / sizeof(T);
  if (interleaved || A.rotary % (2 * kWide) == 0)
    launch_e<T, kHd, kWide>(A, interleaved, grid, s);
  else
    launch_e<T, kHd, kHd / 32>(A, interleaved, grid, s);
}

template <typename T>
void launch_t(const QkArgs& A, int head_dim, int interleaved, unsigned grid, cudaStream_t s) {
  if (head_dim == 64)
    launch_h<T, 64>(A, interleaved, grid, s);
  else if (head_dim == 128)
    launch_h<T, 128>(A, interleaved, grid, s);
  else
    launch_h<T, 256>(A, interleaved, grid, s);
}

void free_qknorm(strata_qknorm* h) {
  if (!h) return;
  if (h->mem) {
    DeviceScope on(h->device);
    cudaFree(h->mem);
  }
  delete h;
}

bool rows_ok(const void* p, long long stride, int width, int size) {
  return p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride >= width && (stride * size) % 16 == 0;
}

}  // namespace

extern "C" {

strata_status strata_qknorm_create(const strata_qknorm_desc* d, const float* q_gain, const float* k_gain,
                                   const double* freqs, void* cuda_stream, strata_qknorm** out) {
  if (!out) return STRATA_EINVAL;
  *out = nullptr;
  if (!d || d->heads < 1 || d->kv_heads < 0 || d->head_dim < 1 || d->rotary_dim < 0 || d->rotary_dim > d->head_dim)
    return STRATA_EINVAL;
  if ((d->interleaved != 0 && d->interleaved != 1) || (d->norm != 0 && d->norm != 1)) return STRATA_EINVAL;
  if (!(d->eps >= 0.f) || std::isinf(d->eps)) return STRATA_EINVAL;
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return STRATA_EUNSUPPORTED;
  if (d->heads > 1024 || d->kv_heads > 1024 || d->rotary_dim % (d->head_dim / 16) != 0) return STRATA_EUNSUPPORTED;
  const int half = d->rotary_dim / 2, hd = d->head_dim;
  if (half > 0 && !freqs) return STRATA_EINVAL;
  for (int i = 0; i < half; ++i)
    if (!std::isfinite(freqs[i])) return STRATA_EINVAL;
  if (fault_is("alloc")) return STRATA_ENOMEM;
  strata_qknorm* h = new (std::nothrow) strata_qknorm();
  if (!h) return STRATA_ENOMEM;
  h->desc = *d;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->nsm, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) {
    cudaGetLastError();
    free_qknorm(h);
    return STRATA_ECUDA;
  }
  const size_t tb = 128 * 8;  // at most head_dim / 2 turns
  if (cudaMalloc(&h->mem, tb + 2 * 256 * 4) != cudaSuccess) {
    cudaGetLastError();
    free_qknorm(h);
    return STRATA_ENOMEM;
  }
  h->turn = static_cast<unsigned long long*>(h->mem);
  h->gain = reinterpret_cast<float*>(static_cast<char*>(h->mem) + tb);
  unsigned long long turn[128] = {};
  for (int i = 0; i < half; ++i) {
    const long double t = (long double)freqs[i] / 6.283185307179586476925286766559005768L;
    turn[i] = (unsigned long long)ldexpl(t - floorl(t), 64);
    if (t - floorl(t) >= 1.0L) turn[i] = 0;  // a tiny negative frequency rounded up to a whole turn
  }
  float ones[256];
  for (float& g : ones) g = 1.f;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaMemcpyAsync(h->turn, turn, sizeof(turn), cudaMemcpyHostToDevice, s);
  for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
    const float* g = i ? k_gain : q_gain;
    e = cudaMemcpyAsync(h->gain + i * hd, g ? g : ones, hd * 4, g ? cudaMemcpyDeviceToDevice : cudaMemcpyHostToDevice,
                        s);
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    free_qknorm(h);
    return STRATA_ECUDA;
  }
  *out = h;
  return STRATA_OK;
}

strata_status strata_qknorm_forward(strata_qknorm* h, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                    void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, int32_t dtype,
                                    const int32_t* position, int32_t T, void* cuda_stream) {
  if (!h || T < 0 || dtype < STRATA_F32 || dtype > STRATA_BF16) return STRATA_EINVAL;
  if (T == 0) return STRATA_OK;
  const strata_qknorm_desc& d = h->desc;
  const int size = dtype == STRATA_F32 ? 4 : 2, qw = d.heads * d.head_dim, kw = d.kv_heads * d.head_dim;
  if (!rows_ok(q, q_stride, qw, size) || !rows_ok(q_out, q_out_stride, qw, size) || !position) return STRATA_EINVAL;
  if (kw > 0 && (!rows_ok(k, k_stride, kw, size) || !rows_ok(k_out, k_out_stride, kw, size))) return STRATA_EINVAL;
  // an output over its own input row for row, or elsewhere
  if (T > 1 && q == q_out && q_stride != q_out_stride) return STRATA_EINVAL;
  if (kw > 0 && (q_out == k_out || q_out == k || k_out == q)) return STRATA_EINVAL;
  if (kw > 0 && T > 1 && k == k_out && k_stride != k_out_stride) return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  QkArgs A;
  A.q = q, A.k = k, A.q_out = q_out, A.k_out = k_out;
  A.qs = q_stride, A.ks = k_stride, A.qos = q_out_stride, A.kos = k_out_stride;
  A.gain = h->gain, A.turn = h->turn, A.position = position;
  A.T = T, A.heads = d.heads, A.total = d.heads + d.kv_heads;
  A.rotary = d.rotary_dim, A.norm = d.norm, A.eps = d.eps;
  // heads per CTA: a row's, so that its angles are formed once, unless there are too few rows to give every SM 8 CTAs;
  // then as few as a CTA's warps take at once
  const long long want = 8LL * h->nsm;
  long long parts = (want + T - 1) / T;
  const int least = kQkThreads / 32;
  const long long most = (A.total + least - 1) / least;
  if (parts > most) parts = most;
  A.per_cta = (int)((A.total + parts - 1) / parts);
  A.groups = (A.total + A.per_cta - 1) / A.per_cta;
  const unsigned grid = (unsigned)T * A.groups;  // T, or fewer than `want` + T where T is below it
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (dtype == STRATA_F32)
    launch_t<float>(A, d.head_dim, d.interleaved, grid, s);
  else if (dtype == STRATA_F16)
    launch_t<__half>(A, d.head_dim, d.interleaved, grid, s);
  else
    launch_t<__nv_bfloat16>(A, d.head_dim, d.interleaved, grid, s);
  if (cudaGetLastError() != cudaSuccess) return STRATA_ECUDA;
  return STRATA_OK;
}

strata_status strata_qknorm_destroy(strata_qknorm* h) {
  free_qknorm(h);
  return STRATA_OK;
}

}  // extern "C"
