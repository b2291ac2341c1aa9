// One-time repack of a product's matrices into the layout of linear.cuh.
#include "linear.cuh"

namespace strata {
namespace {

__device__ __forceinline__ float half_bits(uint16_t b) { return __half2float(__ushort_as_half(b)); }

// A CTA takes a tile: the rows' powers of two first, then its steps.
__global__ void __launch_bounds__(128) linear_pack_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scale,
                                                          const uint16_t* __restrict__ mn, int in, int out, uint8_t* packed,
                                                          float* undo) {
  __shared__ float most_s[16][8], most_m[16][8], mul[16];
  const int tiles = out / kLinTile, nks = in / kLinStep, nblk = in / 32;
  const long long at = blockIdx.x;  // matrix * tiles + tile
  const long long row0 = at * kLinTile;
  {
    const int r = threadIdx.x >> 3, part = threadIdx.x & 7;
    const uint16_t* s = scale + (row0 + r) * nblk;
    const uint16_t* m = mn + (row0 + r) * nblk;
    float bs = 0.f, bm = 0.f;
    for (int i = part; i < nblk; i += 8) {
      const float a = fabsf(half_bits(s[i])), c = fabsf(half_bits(m[i]));
      bs = a < INFINITY ? fmaxf(bs, a) : INFINITY;
      bm = c < INFINITY ? fmaxf(bm, c) : INFINITY;
    }
    most_s[r][part] = bs, most_m[r][part] = bm;
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    float bs = 0.f, bm = 0.f;
    for (int i = 0; i < 8; ++i) bs = fmaxf(bs, most_s[threadIdx.x][i]), bm = fmaxf(bm, most_m[threadIdx.x][i]);
    int k = 0;
    if (bs < INFINITY && bm < INFINITY && (bs > 0.f || bm > 0.f)) {  // rows of zeros or with an infinity: as they are
      int es, em;  // the largest is in [2^(e-1), 2^e)
      frexpf(bs, &es), frexpf(bm, &em);
      k = bs == 0.f ? -3 - em : bm == 0.f ? -9 - es : min(-9 - es, -3 - em);
    }
    mul[threadIdx.x] = pow2i(k);
    undo[row0 + threadIdx.x] = pow2i(-k);
  }
  __syncthreads();
  const int mat = (int)(at / tiles);
  int stride;
  uint8_t* dst = const_cast<uint8_t*>(lin_tile(packed, mat, (int)(at - (long long)mat * tiles), tiles, nks, stride));
  for (int item = threadIdx.x; item < nks * 32; item += 128) {
    const int ks = item >> 5, lane = item & 31, g = lane >> 2, c = lane & 3;
    uint32_t words[4];
    for (int wi = 0; wi < 4; ++wi) {
      const long long row = row0 + g + (wi & 1) * 8;
      const uint8_t* src = codes + row * (in / 2) + (2 * ks + (wi >> 1)) * 16 + 4 * c;
      const uint32_t cw = (uint32_t)src[0] | (uint32_t)src[1] << 8 | (uint32_t)src[2] << 16 | (uint32_t)src[3] << 24;
      uint32_t w = 0;
      for (int u = 0; u < 8; ++u) w |= ((cw >> (4 * u)) & 15u) << ((u & 1 ? 16 : 0) + 4 * (u >> 1));
      words[wi] = w;
    }
    uint8_t* step = dst + (long long)ks * stride;
    *reinterpret_cast<uint4*>(step + lane * 16) = make_uint4(words[0], words[1], words[2], words[3]);
    if (c < 2) {  // c = 0: the scales, 1: the mins
      const uint16_t* src = c ? mn : scale;
      __half h[4];
      for (int i = 0; i < 4; ++i) {
        const int r = g + (i >> 1) * 8;
        h[i] = __float2half_rn(half_bits(src[(row0 + r) * nblk + 2 * ks + (i & 1)]) * (mul[r] * (c ? kLinMin : kLinScale)));
      }
      *reinterpret_cast<uint2*>(step + 512 + g * 16 + c * 8) = *reinterpret_cast<uint2*>(h);
    }
  }
}

}  // namespace

long long linear_packed_bytes(int n, int in, int out) {
  return (long long)n * (out / kLinTile) * (in / kLinStep) * kLinStepBytes;
}

cudaError_t launch_linear_pack(const void* codes, const uint16_t* scale, const uint16_t* mn, int n, int in, int out,
                               uint8_t* packed, float* undo, cudaStream_t s) {
  linear_pack_kernel<<<(unsigned)((long long)n * (out / kLinTile)), 128, 0, s>>>(static_cast<const uint8_t*>(codes), scale, mn,
                                                                                 in, out, packed, undo);
  return cudaGetLastError();
}

}  // namespace strata
