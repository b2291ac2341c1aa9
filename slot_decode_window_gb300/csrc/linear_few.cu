// Products of few rows with 4-bit matrices (8 to a CTA).
//
// y = W x with W = s q + m per block of 32 columns.  A tile of 16 weight rows is
// the A operand of mma.sync.m16n8k16, up to 8 rows of x the B operand; the order
// of the columns within a block is the codes' (the same for both operands).  A
// code becomes the exact number 16 + q with a shift and one logic operation per
// pair, and a block's products t = sum (16 + q) x start from zero, so
//   y += s t + (m - 16 s) sum x
// in f32 keeps the weights exact; sum x comes out of the same instruction with
// ones for A (2^-18: the records' mins are 2^18 m), in the lanes that need it.  x is exact too: bf16 as it is, f16 on
// the f16 instruction, f32 as three bf16 parts by truncation (24 bits).  Rows are not
// scaled: nothing here passes f32's range, and no bit falls out of it, while they are
// between 2^-100 and 2^100 (a row's largest, found by a first read, and its power of
// two would cost 20 to 45% of 9 to 64 rows' time: 16 bf16 rows of 4096 -> 4096 12.8 us
// against 9.1 us).
//
// Measured: one bf16 row of 2048 -> 4096 6.1 us (3.5 us in a graph), eight f32 rows of 4096 -> 2048 8.2 us (5.2; latency: launch,
// one or two rounds of loads a warp, the join); 16 bf16 rows of 4096 -> 4096 9.1 us; one bf16 row of 2048 -> 151936 53 us (3.7 TB/s, 54% of the measured HBM rate: 60% of the issue slots,
// some 110 instructions for a tile's 640 bytes), eight f32 rows 76 us.
#include "linear.cuh"

namespace strata {
namespace {

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

// D = A B + C; C is D, or zeros (kStart).
template <int DT, bool kStart>
__device__ __forceinline__ void few_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  const float c[4] = {kStart ? 0.f : d[0], kStart ? 0.f : d[1], kStart ? 0.f : d[2], kStart ? 0.f : d[3]};
  if constexpr (DT == kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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
__device__ __forceinline__ void few_x(const uint4 (&u)[DT == kF32 ? 2 : 1], uint32_t (&b)[FewType<DT>::kParts][4]) {
  if constexpr (DT == kF32) {
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
    b[0][0] = u[0].x, b[0][1] = u[0].y, b[0][2] = u[0].z, b[0][3] = u[0].w;
  }
}

// A CTA takes kTiles neighbouring tiles of each stack, whose step is one piece of memory; its kWarps warps take the steps in
// turn, and their sums meet in shared memory in the warps' order.  A step's columns of x are split into parts once for
// all of its tiles.
template <int DT, int kTiles, int kWarps, bool kGlu>
__global__ void __launch_bounds__(kWarps * 32, kWarps < 16 ? 16 / kWarps : 1) few_kernel(LinArgs A) {
  constexpr int kMats = kGlu ? 2 : 1, kParts = FewType<DT>::kParts, kAll = kMats * kTiles;
  constexpr uint32_t kOnes = DT == kF16 ? 0x00400040u : 0x36803680u;  // 1 / kLinMin, which the mins carry
  __shared__ float red[kWarps][kAll * 128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int tiles = A.out / kLinTile, nks = A.in / kLinStep;
  const int tile0 = blockIdx.x * kTiles;
  int begin, end;
  if (!lin_rows(A, 0, begin, end) && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(A.err, kErrIndex);
  begin += blockIdx.y * kLinFewRows;  // 8 rows to a CTA
  if (begin >= end) return;
  int stride;  // (the tiles of a CTA are of one group of 8; one past the last reads what is behind it and writes nothing)
  const uint8_t* src[kMats];
#pragma unroll
  for (int m = 0; m < kMats; ++m)
    src[m] = lin_tile(A.w[m].packed, 0, tile0, tiles, nks, stride) + (long long)warp * stride + lane * 16;
  const int to_rec = 512 + g * 16 - lane * 16;
  const long long ahead = (long long)kWarps * stride;
  const bool live = begin + g < end;
  const char* row = static_cast<const char*>(A.x) + (long long)(begin + g) * A.xs * (DT == kF32 ? 4 : 2);
  float acc[kAll][4] = {};
  uint4 code[kAll], rec[kAll];
  auto load = [&](int y) {  // from the step that src is at
    const uint8_t* p = src[y / kTiles] + y % kTiles * kLinStepBytes;
    code[y] = __ldg(reinterpret_cast<const uint4*>(p));
    rec[y] = __ldg(reinterpret_cast<const uint4*>(p + to_rec));
  };
  uint4 xr[2][DT == kF32 ? 2 : 1];  // this lane's eight columns of the step's two blocks
  auto load_x = [&](int ks) {
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int w = 0; w < (DT == kF32 ? 2 : 1); ++w)
        xr[blk][w] = live ? reinterpret_cast<const uint4*>(row + (ks * kLinStep + blk * 32 + c * 8) * (DT == kF32 ? 4 : 2))[w]
                          : make_uint4(0, 0, 0, 0);
  };
  if (warp < nks) {
    load_x(warp);
#pragma unroll
    for (int y = 0; y < kAll; ++y) load(y);
  }
  for (int ks = warp; ks < nks; ks += kWarps) {
    const int next = ks + kWarps;
    uint32_t b[2][kParts][4];
    float xsum[2][4];
    const uint32_t ones[4] = {kOnes, kOnes, kOnes, kOnes};
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      few_x<DT>(xr[blk], b[blk]);
#pragma unroll
      for (int k = kParts - 1; k >= 0; --k) {
        if (k == kParts - 1)
          few_mma<DT, true>(xsum[blk], ones, b[blk][k][0], b[blk][k][1]);
        else
          few_mma<DT, false>(xsum[blk], ones, b[blk][k][0], b[blk][k][1]);
        few_mma<DT, false>(xsum[blk], ones, b[blk][k][2], b[blk][k][3]);
      }
    }
    if (next < nks) load_x(next);
#pragma unroll
    for (int m = 0; m < kMats; ++m) src[m] += ahead;
#pragma unroll
    for (int y = 0; y < kAll; ++y) {
      // a tile's next step is on its way from here on
      const uint4 now = code[y], scales = rec[y];
      if (next < nks) load(y);
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint32_t w0 = blk ? now.z : now.x, w1 = blk ? now.w : now.y;
        const uint32_t a0[4] = {few_pair<DT, 0>(w0), few_pair<DT, 0>(w1), few_pair<DT, 1>(w0), few_pair<DT, 1>(w1)};
        const uint32_t a1[4] = {few_pair<DT, 2>(w0), few_pair<DT, 2>(w1), few_pair<DT, 3>(w0), few_pair<DT, 3>(w1)};
        float d[4];
#pragma unroll
        for (int k = kParts - 1; k >= 0; --k) {
          if (k == kParts - 1)
            few_mma<DT, true>(d, a0, b[blk][k][0], b[blk][k][1]);
          else
            few_mma<DT, false>(d, a0, b[blk][k][0], b[blk][k][1]);
          few_mma<DT, false>(d, a1, b[blk][k][2], b[blk][k][3]);
        }
        const float s0 = 1.f / kLinScale * half_of(scales.x, blk), s1 = 1.f / kLinScale * half_of(scales.y, blk);
        const float o0 = fmaf(-16.f * kLinMin, s0, half_of(scales.z, blk)), o1 = fmaf(-16.f * kLinMin, s1, half_of(scales.w, blk));
        float(&z)[4] = acc[y];
        z[0] = fmaf(s0, d[0], fmaf(o0, xsum[blk][0], z[0]));
        z[1] = fmaf(s0, d[1], fmaf(o0, xsum[blk][1], z[1]));
        z[2] = fmaf(s1, d[2], fmaf(o1, xsum[blk][0], z[2]));
        z[3] = fmaf(s1, d[3], fmaf(o1, xsum[blk][1], z[3]));
      }
    }
  }
#pragma unroll
  for (int y = 0; y < kAll; ++y)
    *reinterpret_cast<float4*>(&red[warp][y * 128 + lane * 4]) = make_float4(acc[y][0], acc[y][1], acc[y][2], acc[y][3]);
  __syncthreads();
  for (int i = threadIdx.x; i < kTiles * 128; i += kWarps * 32) {
    // consecutive threads take consecutive weight rows of one row of x
    const int col = i / (kTiles * 16), t = i / 16 % kTiles, r = i & 15;
    const int from = t * 128 + ((r & 7) * 4 + (col >> 1)) * 4 + (r >> 3) * 2 + (col & 1);
    const int o = (tile0 + t) * kLinTile + r;
    if (tile0 + t >= tiles || begin + col >= end) continue;
    float v[kMats];
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += red[w][m * kTiles * 128 + from];
      v[m] = s * A.w[m].undo[o];
    }
    const float y = kGlu ? lin_silu<false>(v[0]) * v[kMats - 1] : v[0];
    const long long at = (long long)(begin + col) * A.ys + o;
    if constexpr (DT == kF32)
      static_cast<float*>(A.y)[at] = y;
    else if constexpr (DT == kF16)
      static_cast<__half*>(A.y)[at] = __float2half_rn(y);
    else
      static_cast<__nv_bfloat16*>(A.y)[at] = __float2bfloat16_rn(y);
  }
}

template <int DT, int kTiles, int kWarps, bool kGlu>
void launch_k(const LinArgs& A, cudaStream_t s) {
  const dim3 grid((A.out / kLinTile + kTiles - 1) / kTiles, (A.T + kLinFewRows - 1) / kLinFewRows);
  few_kernel<DT, kTiles, kWarps, kGlu><<<grid, kWarps * 32, 0, s>>>(A);
}

// One tile a CTA while all tiles' CTAs run at once (two an SM), so that a small matrix is spread over the SMs: 16 warps for f32 rows,
// whose parts cost most (eight rows of 4096 -> 2048 in a graph 5.2 us, with 8 warps 5.5 us), else 8 (one bf16 row of 2048 -> 4096
// 3.5 us, with 16 warps 3.9 us; with gate 5.2 and 6.4 us: two of the larger CTAs do not fit an SM).  4 tiles (of a pair, 2 of each)
// for larger matrices, which are bound by memory and by x's parts, with 8 warps and, where an SM gets CTAs enough, 4: the fewer warps
// share the steps, the less of a CTA's time is its start and its join.  One row of 4096 columns: 8192 weight rows 10.5 us with
// 8 warps, 12.8 us with 4; 2048 columns, 151936 weight rows 60.5 and 55.6 us (51.7 us since).
template <int DT, bool kGlu>
void launch_t(const LinArgs& A, int nsm, cudaStream_t s) {
  const int tiles = A.out / kLinTile;
  if (tiles <= 2 * nsm)
    launch_k<DT, 1, DT == kF32 && !kGlu ? 16 : 8, kGlu>(A, s);
  else if (tiles <= 16 * nsm)
    launch_k<DT, kGlu ? 2 : 4, 8, kGlu>(A, s);
  else
    launch_k<DT, kGlu ? 2 : 4, 4, kGlu>(A, s);
}

}  // namespace

// At most 8 rows; and more, 8 to a CTA, where the steps of all tiles and groups of 8 rows are few: then one launch without a
// workspace is faster than two with (in a graph, 16-bit rows against exact weights: 16 rows of 4096 -> 4096 9.2 us against 19.1 us, 32 rows
// 14.5 and 19.2 us, 48 rows 21.5 and 20.1 us; 64 rows of 2048 -> 4096 16.0 and 14.8 us, of 4096 -> 2048 14.7 and 15.9 us, of 2048 -> 512 3.9 and
// 12.8 us.  Against rounded weights: 24 rows of 4096 -> 4096 12.6 and 12.6 us, 32 rows 14.5 and 12.6 us.  f32 rows of 4096 -> 2048: 16 9.8
// and 14.0 us, 24 14.2 and 14.1 us).
bool linear_few_rows(const LinArgs& A, int nsm) {
  if (A.n != 1) return false;
  if (A.T <= kLinFewRows) return true;
  const long long tiles = A.out / kLinTile, groups = (A.T + kLinFewRows - 1) / kLinFewRows;
  const long long most = A.dtype == kF32 ? 130 : A.dtype == kBF16 && A.rounded ? 320 : 440;
  return A.T <= 64 && tiles <= 2 * nsm && (A.glu ? 2 : 1) * tiles * groups * (A.in / kLinStep) <= most * nsm;
}

cudaError_t launch_linear_few(const LinArgs& A, int nsm, cudaStream_t s) {
  if (A.dtype == kF32)
    A.glu ? launch_t<kF32, true>(A, nsm, s) : launch_t<kF32, false>(A, nsm, s);
  else if (A.dtype == kF16)
    A.glu ? launch_t<kF16, true>(A, nsm, s) : launch_t<kF16, false>(A, nsm, s);
  else
    A.glu ? launch_t<kBF16, true>(A, nsm, s) : launch_t<kBF16, false>(A, nsm, s);
  return cudaGetLastError();
}

}  // namespace strata
