// The products' matrices in the handle's own layout, and the launches of their
// kernels (linear_pack.cu, linear_few.cu, linear_many.cu).
//
// A matrix [out][in] is out/16 tiles by in/64 steps.  A tile's step is 640 bytes
// (0.625 a weight, as in the block format); the tiles of 128 rows (8, or what is
// left) are together, step by step, so that one copy brings a step of all of them.
// The 640 bytes are 512 of codes and 8 records:
//   codes: lane (g = lane/4, c = lane%4) has 16 bytes, a word for row g and one
//     for row g + 8 of the step's first block of 32 columns, then the same of its
//     second; a word holds columns 8c..8c+7 of the block, column 8c+2i in bits
//     4i..4i+3 and column 8c+2i+1 in bits 16+4i..16+4i+3
//   record g (16 bytes, f16): scales of row g (first block, second), of row
//     g + 8, then the mins in the same order
// Both carry a power of two of their row, scales 2^24 more (a masked code read as
// f16 is the subnormal q 2^-24) and mins 2^18 more: the row's largest scale is in
// [2^14, 2^15), or its largest min where that is less.  A row's results are multiplied
// by `undo`, the inverse.  (f16's least step, 2^-24, is 2^-38 of the row's largest
// scale for scales and 2^-32 of it for mins, or 2^-44 and 2^-38 of its largest min.)
#pragma once
#include "kv8.cuh"

namespace strata {

constexpr int kLinStep = 64, kLinStepBytes = 640, kLinTile = 16;
constexpr int kLinFewRows = 8;
constexpr float kLinScale = 0x1p24f, kLinMin = 0x1p18f;  // what the records' scales and mins carry
constexpr int kF32 = 0, kF16 = 1, kBF16 = 2;  // strata_dtype

struct LinMat {
  const uint8_t* packed;  // [n][out/16][in/64][640]
  const float* undo;      // [n][out]
};

struct LinArgs {
  LinMat w[2];        // the stack, and the one behind the gate (glu)
  int n, in, out, glu;
  int rounded;        // many bf16 rows take weights rounded to f16
  const void* x;
  void* y;
  long long xs, ys;
  int dtype, T;
  const int* offsets;  // [n + 1], or null (n = 1)
  unsigned* err;
};

// Where tile `tile` of matrix `mat` has step 0, and the bytes from a step of it to the next.
__device__ __forceinline__ const uint8_t* lin_tile(const uint8_t* packed, int mat, int tile, int tiles, int nks, int& stride) {
  const int group = tile & ~7, here = min(8, tiles - group);
  stride = here * kLinStepBytes;
  return packed + (((long long)mat * tiles + group) * nks + (tile - group)) * kLinStepBytes;
}

// The rows of matrix i: begin, end.  A range that is out of order or outside 0..T is empty and noted.
__device__ __forceinline__ bool lin_rows(const LinArgs& A, int i, int& begin, int& end) {
  begin = 0, end = A.T;
  if (!A.offsets) return true;
  begin = A.offsets[i], end = A.offsets[i + 1];
  if (begin >= 0 && begin <= end && end <= A.T) return true;
  end = begin = 0;
  return false;
}

// silu(z) = z / (1 + e^-z) from e^-|z|, which is never above 1: z far below zero keeps its z e^z, where e^-z leaves f32's range
// from -88.7 on.  kFast: the fast exponential and quotient (a few 2^-22, and 2^-17 of the exponent's rounding far out, against the 2^-12
// of 16-bit results).
template <bool kFast>
__device__ __forceinline__ float lin_silu(float z) {
  const float t = kFast ? __expf(-fabsf(z)) : expf(-fabsf(z));
  const float top = z < 0.f ? z * t : z;
  return kFast ? __fdividef(top, 1.f + t) : top / (1.f + t);
}

long long linear_packed_bytes(int n, int in, int out);
cudaError_t launch_linear_pack(const void* codes, const uint16_t* scale, const uint16_t* mn, int n, int in, int out,
                               uint8_t* packed, float* undo, cudaStream_t s);
// Whether a call is the few-row path's.
bool linear_few_rows(const LinArgs& A, int nsm);
cudaError_t launch_linear_few(const LinArgs& A, int nsm, cudaStream_t s);

// The many-row path: its workspace's bytes; its shared memory limit and how many clusters of 2, 4 and 8 CTAs run at once
// (once per handle, on the current device).
long long linear_many_workspace(int in, int max_rows);
cudaError_t setup_linear_many(int (&clusters)[3]);
cudaError_t launch_linear_many(const LinArgs& A, void* workspace, int max_rows, int nsm, const int (&clusters)[3], cudaStream_t s);

}  // namespace strata
