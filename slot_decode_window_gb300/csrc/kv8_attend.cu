// Attention of a call's rows over the slots' 8-bit caches.
#include "kv8.cuh"

namespace strata {
namespace {

// A warp per (row, query head): lane l holds head_dim / 32 neighbouring dims,
// and one pass over the positions keeps the running maximum and sum of the
// softmax.
template <typename T, int E>
__global__ void __launch_bounds__(128) attend_simple_kernel(Kv8Dev C, Kv8Rows R, const T* __restrict__ q,
                                                            long long q_stride, T* __restrict__ out,
                                                            long long out_stride, float scale) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int row = (int)(w / C.heads), head = (int)(w % C.heads);
  if (row >= R.n_rows) return;
  for (int i = 0; i < R.n_seq; ++i) {
    const Kv8Seq s = kv8_seq(R, C, i);
    if (!s.held_ok && w == 0 && lane == 0) atomicOr(C.err, kErrIndex);
    if (!s.rows_ok || row < s.row0 || row >= s.row0 + s.n) continue;
    const int seen = s.held_ok ? s.length - (s.row0 + s.n - row) + 1 : 0;
    const int kvh = head / (C.heads / C.kv_heads);
    const long long line = s.held_ok ? (long long)s.slot * C.kv_heads + kvh : 0;
    const uint8_t* kc = C.k + line * C.max_ctx * C.head_dim + lane * E;
    const uint8_t* vc = C.v + line * C.max_ctx * C.head_dim + lane * E;
    const uint8_t* ke = C.k_exp + line * C.n_blocks;
    const uint8_t* ve = C.v_exp + line * C.n_blocks;
    float x[E], o[E], m = -INFINITY, l = 0.f;
    const T* src = q + (long long)row * q_stride + head * C.head_dim + lane * E;
#pragma unroll
    for (int d = 0; d < E; ++d) x[d] = Val<T>::up(src[d]) * scale, o[d] = 0.f;
    for (int j = 0; j < seen; ++j) {
      uint32_t kw = 0, vw = 0;
#pragma unroll
      for (int d = 0; d < E; ++d) {
        kw |= (uint32_t)kc[(long long)j * C.head_dim + d] << (8 * d);
        vw |= (uint32_t)vc[(long long)j * C.head_dim + d] << (8 * d);
      }
      float k4[4], v4[4], dot = 0.f;
      kv8_decode4(kw, C.format, k4);
      kv8_decode4(vw, C.format, v4);
#pragma unroll
      for (int d = 0; d < E; ++d) dot = fmaf(x[d], k4[d], dot);
#pragma unroll
      for (int b = 16; b > 0; b >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, b);
      dot *= pow2i(kv8_exp(ke[j >> C.block_log2]));
      const float mn = fmaxf(m, dot), a = expf(m - mn), p = expf(dot - mn), pv = p * pow2i(kv8_exp(ve[j >> C.block_log2]));
      l = l * a + p;
#pragma unroll
      for (int d = 0; d < E; ++d) o[d] = fmaf(pv, v4[d], o[d] * a);
      m = mn;
    }
    T* dst = out + (long long)row * out_stride + head * C.head_dim + lane * E;
#pragma unroll
    for (int d = 0; d < E; ++d) dst[d] = Val<T>::down(seen > 0 ? o[d] / l : 0.f);
  }
}

template <typename T>
cudaError_t attend_typed(const Kv8Dev& C, const Kv8Rows& R, const void* q, long long q_stride, void* out,
                         long long out_stride, float scale, cudaStream_t s) {
  const long long warps = (long long)R.n_rows * C.heads;
  const unsigned grid = (unsigned)((warps + 3) / 4);
  if (C.head_dim == 64)
    attend_simple_kernel<T, 2><<<grid, 128, 0, s>>>(C, R, static_cast<const T*>(q), q_stride, static_cast<T*>(out),
                                                    out_stride, scale);
  else
    attend_simple_kernel<T, 4><<<grid, 128, 0, s>>>(C, R, static_cast<const T*>(q), q_stride, static_cast<T*>(out),
                                                    out_stride, scale);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_attend(const Kv8Dev& C, const Kv8Rows& R, const void* q, long long q_stride, void* out,
                              long long out_stride, int dtype, float scale, cudaStream_t s) {
  if (dtype == 0) return attend_typed<float>(C, R, q, q_stride, out, out_stride, scale, s);
  if (dtype == 1) return attend_typed<__half>(C, R, q, q_stride, out, out_stride, scale, s);
  return attend_typed<__nv_bfloat16>(C, R, q, q_stride, out, out_stride, scale, s);
}

}  // namespace strata
