// Products of few rows with 4-bit matrices.
//
// y = W x with W = s q + m per block of 32 columns.  A tile of 16 weight rows is
// the A operand of mma.sync.m16n8k16, up to 8 rows of x the B operand; the order
// of the columns within a block is the codes' (the same for both operands).  A
// code becomes the exact number 16 + q with a shift and one logic operation per
// pair, and a block's products t = sum (16 + q) x start from zero, so
//   y += s t + (m - 16 s) sum x
// in f32 keeps the weights exact; sum x comes out of the same instruction with
// ones for A, in the lanes that need it.  x is exact too: bf16 as it is, f16 on
// the f16 instruction, f32 as three bf16 parts by truncation (24 bits).
#include "linear.cuh"

namespace strata {
namespace {

constexpr int kFewWarps = 16, kFewThreads = kFewWarps * 32;

template <int DT> struct FewType;
template <> struct FewType<kF32> {
  static constexpr int kParts = 3;
};
template <> struct FewType<kF16> {
  static constexpr int kParts = 1;
};
template <> struct FewType<kBF16> {
  static constexpr int kParts = 1;
};

template <int DT>
__device__ __forceinline__ void few_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (DT == kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Pair i of a word of codes as two numbers 16 + q: the code in the top mantissa bits of 16.
template <int DT, int I>
__device__ __forceinline__ uint32_t few_pair(uint32_t w) {
  if constexpr (DT == kF16) {
    const uint32_t v = I == 0 ? w << 6 : I == 1 ? w << 2 : I == 2 ? w >> 2 : w >> 6;
    return (v & 0x03C003C0u) | 0x4C004C00u;
  } else {
    const uint32_t v = I == 0 ? w << 3 : I == 1 ? w >> 1 : I == 2 ? w >> 5 : w >> 9;
    return (v & 0x00780078u) | 0x41804180u;
  }
}

__device__ __forceinline__ float half_of(uint32_t two, int upper) {
  const __half2 h = *reinterpret_cast<const __half2*>(&two);
  return __half2float(upper ? h.y : h.x);
}

// Eight neighbouring values of a row, as kParts times four pairs.
template <int DT>
__device__ __forceinline__ void few_x(const void* row, int i, bool live, uint32_t (&b)[FewType<DT>::kParts][4]) {
  if constexpr (DT == kF32) {
    uint4 u[2] = {};
    if (live) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + i);
      u[0] = p[0], u[1] = p[1];
    }
    const uint32_t v[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float r0 = __uint_as_float(v[2 * p]), r1 = __uint_as_float(v[2 * p + 1]);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        b[k][p] = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
        r0 -= __uint_as_float(__float_as_uint(r0) & 0xFFFF0000u);
        r1 -= __uint_as_float(__float_as_uint(r1) & 0xFFFF0000u);
      }
    }
  } else {
    uint4 u = {};
    if (live) u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
    b[0][0] = u.x, b[0][1] = u.y, b[0][2] = u.z, b[0][3] = u.w;
  }
}

// A CTA takes kTiles tiles of each stack; its warps take the steps in turn.
template <int DT, int kTiles, bool kGlu>
__global__ void __launch_bounds__(kFewThreads) few_kernel(LinArgs A) {
  constexpr int kMats = kGlu ? 2 : 1, kParts = FewType<DT>::kParts;
  constexpr uint32_t kOnes = DT == kF16 ? 0x3C003C00u : 0x3F803F80u;
  __shared__ float red[kFewWarps][kMats][kTiles * 128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int tiles = A.out / kLinTile, nks = A.in / kLinStep;
  const int tile0 = blockIdx.x * kTiles, mat = blockIdx.y;
  int begin, end;
  if (!lin_rows(A, mat, begin, end) && threadIdx.x == 0 && blockIdx.x == 0) atomicOr(A.err, kErrIndex);
  const uint8_t* src[kMats][kTiles];
  int stride[kTiles];
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int t = 0; t < kTiles; ++t)  // (a CTA past the last tile reads it again and writes nothing)
      src[m][t] = lin_tile(A.w[m].packed, mat, min(tile0 + t, tiles - 1), tiles, nks, stride[t]);
  for (int r0 = begin; r0 < end; r0 += kLinFewRows) {
    const bool live = r0 + g < end;
    const char* row = static_cast<const char*>(A.x) + (long long)(r0 + g) * A.xs * (DT == kF32 ? 4 : 2);
    float acc[kMats][kTiles][4] = {};
    for (int ks = warp; ks < nks; ks += kFewWarps) {
      uint4 code[kMats][kTiles], rec[kMats][kTiles];
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          const uint8_t* p = src[m][t] + (long long)ks * stride[t];
          code[m][t] = __ldg(reinterpret_cast<const uint4*>(p + lane * 16));
          rec[m][t] = __ldg(reinterpret_cast<const uint4*>(p + 512 + g * 16));
        }
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        uint32_t b[kParts][4];
        few_x<DT>(row, ks * kLinStep + blk * 32 + c * 8, live, b);
        float xsum[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t ones[4] = {kOnes, kOnes, kOnes, kOnes};
#pragma unroll
        for (int k = kParts - 1; k >= 0; --k) {
          few_mma<DT>(xsum, ones, b[k][0], b[k][1]);
          few_mma<DT>(xsum, ones, b[k][2], b[k][3]);
        }
#pragma unroll
        for (int m = 0; m < kMats; ++m)
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            const uint32_t w0 = blk ? code[m][t].z : code[m][t].x, w1 = blk ? code[m][t].w : code[m][t].y;
            const uint32_t a0[4] = {few_pair<DT, 0>(w0), few_pair<DT, 0>(w1), few_pair<DT, 1>(w0), few_pair<DT, 1>(w1)};
            const uint32_t a1[4] = {few_pair<DT, 2>(w0), few_pair<DT, 2>(w1), few_pair<DT, 3>(w0), few_pair<DT, 3>(w1)};
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = kParts - 1; k >= 0; --k) {
              few_mma<DT>(d, a0, b[k][0], b[k][1]);
              few_mma<DT>(d, a1, b[k][2], b[k][3]);
            }
            const uint32_t* h = &rec[m][t].x;  // scales of rows g, g + 8 (both blocks), then mins
            const float s0 = 0x1p-24f * half_of(h[0], blk), s1 = 0x1p-24f * half_of(h[1], blk);
            const float o0 = fmaf(-16.f, s0, half_of(h[2], blk)), o1 = fmaf(-16.f, s1, half_of(h[3], blk));
            float(&z)[4] = acc[m][t];
            z[0] = fmaf(s0, d[0], fmaf(o0, xsum[0], z[0]));
            z[1] = fmaf(s0, d[1], fmaf(o0, xsum[1], z[1]));
            z[2] = fmaf(s1, d[2], fmaf(o1, xsum[0], z[2]));
            z[3] = fmaf(s1, d[3], fmaf(o1, xsum[1], z[3]));
          }
      }
    }
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        *reinterpret_cast<float4*>(&red[warp][m][t * 128 + lane * 4]) =
            make_float4(acc[m][t][0], acc[m][t][1], acc[m][t][2], acc[m][t][3]);
    __syncthreads();
    if (threadIdx.x < kTiles * 128) {
      // consecutive threads take consecutive weight rows of one row of x
      const int t = threadIdx.x >> 7, col = (threadIdx.x >> 4) & 7, r = threadIdx.x & 15;
      const int from = t * 128 + ((r & 7) * 4 + (col >> 1)) * 4 + (r >> 3) * 2 + (col & 1);
      const int o = (tile0 + t) * kLinTile + r;
      if (tile0 + t < tiles && r0 + col < end) {
        float v[kMats];
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
          float s = 0.f;
#pragma unroll
          for (int w = 0; w < kFewWarps; ++w) s += red[w][m][from];
          v[m] = s * A.w[m].undo[(long long)mat * A.out + o];
        }
        const float y = kGlu ? silu_f32(v[0]) * v[kMats - 1] : v[0];
        const long long at = (long long)(r0 + col) * A.ys + o;
        if constexpr (DT == kF32)
          static_cast<float*>(A.y)[at] = y;
        else if constexpr (DT == kF16)
          static_cast<__half*>(A.y)[at] = __float2half_rn(y);
        else
          static_cast<__nv_bfloat16*>(A.y)[at] = __float2bfloat16_rn(y);
      }
    }
    __syncthreads();
  }
}

template <int DT, int kTiles>
void launch_t(const LinArgs& A, cudaStream_t s) {
  const dim3 grid((A.out / kLinTile + kTiles - 1) / kTiles, A.n);
  if (A.glu)
    few_kernel<DT, kTiles, true><<<grid, kFewThreads, 0, s>>>(A);
  else
    few_kernel<DT, kTiles, false><<<grid, kFewThreads, 0, s>>>(A);
}

}  // namespace

cudaError_t launch_linear_few(const LinArgs& A, int nsm, cudaStream_t s) {
  (void)nsm;
  if (A.dtype == kF32)
    launch_t<kF32, 1>(A, s);
  else if (A.dtype == kF16)
    launch_t<kF16, 1>(A, s);
  else
    launch_t<kBF16, 1>(A, s);
  return cudaGetLastError();
}

}  // namespace strata
