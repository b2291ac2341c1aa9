// The 8-bit KV caches' format, the rows of a call, and value types, shared by
// the append, read and attention kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace strata {

constexpr int kKv8EMin = -48, kKv8EMax = 47, kKv8Bias = 127;
constexpr int kKv8MaxSeq = 1024;

// One layer's caches as a launch sees them.
struct Kv8Dev {
  uint8_t* k;          // [n_slots][kv_heads][max_ctx][head_dim]
  uint8_t* v;
  uint8_t* k_exp;      // [n_slots][kv_heads][n_blocks]
  uint8_t* v_exp;
  int n_slots, heads, kv_heads, head_dim, max_ctx, block_log2, n_blocks, format;
  unsigned* err;
};

struct Kv8Rows {
  int n_seq, n_rows, max_rows;
  const int* row_start;
  const int* slot;
  const int* length;
};

// One sequence of a call.  rows_ok: its rows may be touched; held_ok: its slot
// and length are in range too.
struct Kv8Seq {
  int row0, n, slot, length;
  bool rows_ok, held_ok;
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8Rows& R, const Kv8Dev& C, int i) {
  Kv8Seq s;
  s.row0 = R.row_start[i];
  const int end = R.row_start[i + 1];
  s.slot = R.slot[i];
  s.length = R.length[i];
  s.rows_ok = s.row0 >= 0 && s.row0 <= end && end <= R.n_rows;
  s.n = s.rows_ok ? end - s.row0 : 0;
  s.rows_ok = s.rows_ok && s.n <= R.max_rows;
  s.held_ok = s.rows_ok && s.slot >= 0 && s.slot < C.n_slots && s.length >= 0 && s.length <= C.max_ctx;
  return s;
}

// Work that is cut into pieces of a sequence: pieces(n) of n rows, at least one (so that some CTA looks at every
// sequence).  A launch either has as many places for each sequence as the longest may need, or one list of all
// sequences' pieces.  kv8_find, for a whole block of kThreads: the sequence and the piece at place u of the list (seq < 0
// past its end), and the list's length.
struct Kv8Piece { int seq, at; long long all; };
template <int kThreads, class Pieces>
__device__ __forceinline__ Kv8Piece kv8_find(const Kv8Rows& R, long long u, Pieces pieces) {
  static_assert(4 * kThreads >= kKv8MaxSeq, "sequences per thread");
  __shared__ long long warp_sums[kThreads / 32];
  __shared__ Kv8Piece found;
  const int share = (R.n_seq + kThreads - 1) / kThreads, first = threadIdx.x * share, lane = threadIdx.x & 31;
  long long count[4], sum = 0;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const int i = first + y;
    count[y] = 0;
    if (y < share && i < R.n_seq) {
      const int a = R.row_start[i], b = R.row_start[i + 1];
      count[y] = a >= 0 && a <= b && b <= R.n_rows && b - a <= R.max_rows ? max(1LL, pieces(b - a)) : 1;
    }
    sum += count[y];
  }
  long long upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += t;
  }
  if (threadIdx.x == kThreads - 1) found.seq = -1;
  if (lane == 31) warp_sums[threadIdx.x >> 5] = upto;
  __syncthreads();
  long long before = upto - sum;
  for (int w = 0; w < (int)threadIdx.x >> 5; ++w) before += warp_sums[w];
  if (threadIdx.x == kThreads - 1) found.all = before + sum;
  if (u >= before && u < before + sum) {
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if (u >= before && u < before + count[y]) found.seq = first + y, found.at = (int)(u - before);
      before += count[y];
    }
  }
  __syncthreads();
  const Kv8Piece p = found;
  __syncthreads();  // the next call writes again
  return p;
}

__device__ __forceinline__ int kv8_exp(uint8_t byte) { return min(max((int)byte - kKv8Bias, kKv8EMin), kKv8EMax); }

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// The least e with a <= qmax 2^e, clamped.  448 = 1.75 * 2^8, 127 = 1.984375 * 2^6.
__device__ __forceinline__ int kv8_least_exp(float a, int format) {
  const unsigned bits = __float_as_uint(a);
  const int shift = format == 0 ? 8 : 6;
  const unsigned top = format == 0 ? 0x600000u : 0x7E0000u;
  int e = (int)(bits >> 23) - 127 - shift + ((bits & 0x7FFFFFu) > top ? 1 : 0);
  if (bits == 0) e = kKv8EMin;
  return min(max(e, kKv8EMin), kKv8EMax);
}

// What the products of a row of q (brought to [1, 2) by 1 / power) with a block's codes are multiplied by, besides the
// block's 2^ek, to be scores in base 2.  Products are below 2^17 and 2^ek at most 2^47, so with a factor of at most 2^63
// every score of a row without infinities or NaN is finite, and so is zero times the factors.  Rows beyond it (scale |q|
// of some 1e18 and more) keep the order of their scores and differences that are far larger than the softmax tells apart.
__device__ __forceinline__ float kv8_row_factor(float scale2, float power) {
  return fminf(fmaxf(scale2 * power, -0x1p63f), 0x1p63f);
}

// Two e4m3 codes to f16x2 and back (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n.reg .b16 t;\ncvt.u16.u32 t, %1;\ncvt.rn.f16x2.e4m3x2 %0, t;\n}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n.reg .b16 t;\ncvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\ncvt.u32.u16 %0, t;\n}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four values (already scaled by 2^-e, no NaN) to a word of four codes.
__device__ __forceinline__ uint32_t kv8_encode4(const float* v, int format) {
  if (format == 0) return f32_to_e4m3x2(v[0], v[1]) | (f32_to_e4m3x2(v[2], v[3]) << 16);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= (uint32_t)(__float2int_rn(fminf(fmaxf(v[i], -127.f), 127.f)) & 0xFF) << (8 * i);
  return w;
}

// A word of four codes to four numbers.
__device__ __forceinline__ void kv8_decode4(uint32_t w, int format, float* v) {
  if (format == 0) {
    const uint32_t a = e4m3x2_to_f16x2(w & 0xFFFFu), b = e4m3x2_to_f16x2(w >> 16);
    const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
    v[0] = fa.x, v[1] = fa.y, v[2] = fb.x, v[3] = fb.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i));
  }
}

// Value types: kPer values in one 16-byte access.
template <typename T> struct Val;
template <> struct Val<float> {
  static constexpr int kPer = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};
template <> struct Val<__half> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(h[i]);
      f[2 * i] = t.x, f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint4 u;
    __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    return u;
  }
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};
template <> struct Val<__nv_bfloat16> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return u;
  }
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};

// Makes a device current while it lives.
struct DeviceScope {
  int before = -1;
  bool ok = true;
  explicit DeviceScope(int device) {
    int now = -1;
    ok = cudaGetDevice(&now) == cudaSuccess;
    if (ok && now != device) {
      ok = cudaSetDevice(device) == cudaSuccess;
      if (ok) before = now;
    }
  }
  ~DeviceScope() {
    if (before >= 0) cudaSetDevice(before);
  }
};

cudaError_t launch_kv8_append(const Kv8Dev& C, const Kv8Rows& R, const void* k, long long k_stride, const void* v,
                              long long v_stride, int dtype, cudaStream_t s);
cudaError_t launch_kv8_read(const Kv8Dev& C, const Kv8Rows& R, void* k, long long k_stride, void* v,
                            long long v_stride, int dtype, cudaStream_t s);
// The attention's copy descriptors: codes as [layers][rows][head_dim], boxes of 64 rows, swizzled.
struct Kv8Maps {
  CUtensorMap k, v;
};
// Shared-memory limits of the attention kernels for a shape, on the current device (once per handle).
cudaError_t setup_kv8_attend(int head_dim, int format);
// Workspace: 256 bytes that begin with the error word, a counter per SM (both start at zero), then the joins' parts.
long long kv8_attend_zeroed(int nsm);
long long kv8_attend_workspace(int nsm, int head_dim);
cudaError_t launch_kv8_attend(const Kv8Dev& C, const Kv8Rows& R, const Kv8Maps& M, int layer, void* workspace, int nsm,
                              const void* q, long long q_stride, void* out, long long out_stride, int dtype,
                              float scale, cudaStream_t s);

// The many-row path of the same call (kv8_prompt.cu).
int kv8_prompt_part_floats(int head_dim);
cudaError_t setup_kv8_prompt(int head_dim, int format);
cudaError_t launch_kv8_prompt(const Kv8Dev& C, const Kv8Rows& R, const Kv8Maps& M, int layer, unsigned* count,
                              float* parts, int nsm, const void* q, long long q_stride, void* out,
                              long long out_stride, int dtype, float scale, cudaStream_t s);

}  // namespace strata
