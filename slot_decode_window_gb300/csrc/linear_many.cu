// Products of many rows with 4-bit matrices on the 5th-generation tensor cores.
//
// D = W X^T for 256 weight rows (two halves of 128: the second half, or the
// stack behind the gate) and up to 192 rows of x (64 of f32 rows): weights are the
// A operand, in tensor memory, where the conversion warps write them as f16 from
// the 4-bit codes, 64 columns at a time; x is the B operand, f16 in the order of
// the codes, swizzled, brought by bulk copies from the workspace that
// linear_rows_kernel fills.  Weight rows on the M side leave the rows of x free
// to be few: an expert with 20 rows costs 32 columns, not 128.
//
// f16 and bf16 rows: one product, W rounded to f16.  f32 rows: x and W in two
// f16 parts each (22 bits), hi hi + hi lo + lo hi; the accumulators' adds
// truncate, so after every 512 columns they are added to f32 registers, with
// two sets of accumulators in turn.
//
// Roles (18 warps): 8 of conversion (each its quarter of the lanes of one half,
// its codes through a ring of its own with cp.async), 8 of results (each a
// quarter of the lanes and half of the rows of x), one of copies of x, one that
// issues the products.  CTAs (one per SM) take the tiles of all matrices in
// turn, weight rows fastest, so that concurrent CTAs share rows of x in L2.
#include "linear.cuh"
#include "tcgen05.cuh"

namespace strata {
namespace {

constexpr int kManyThreads = 18 * 32, kLoadWarp = 16, kMmaWarp = 17;
constexpr int kFifo = 8;                      // steps of codes a conversion warp has under way
constexpr int kFifoStep = 2 * kLinStepBytes;  // its two tiles' step
constexpr int kChunk = 8;                     // steps between sums of f32 rows
constexpr int kMaxMats = 1024;

template <bool TWO> struct ManyPlan {
  static constexpr int kParts = TWO ? 2 : 1;
  static constexpr int kCols = TWO ? 64 : 192;   // most rows of x in a tile
  static constexpr int kSets = TWO ? 2 : 1;      // of accumulators
  static constexpr int kA = 2 * kSets * kCols;   // first column of the weights in tensor memory
  static constexpr int kStages = TWO ? 7 : 5;    // of x
  static constexpr int kPart = kCols * 128;      // bytes of a part of a stage of x
  static constexpr int kStage = kPart * kParts;
  static constexpr int kFifoOff = kStages * kStage;
  static constexpr int kBars = kFifoOff + 8 * kFifo * kFifoStep;
  static constexpr int kMisc = kBars + 256;
  static constexpr int kPre = kMisc + 64;        // [n + 1] tiles before each matrix
  static_assert(kA + 4 * 32 * kParts <= 512, "tensor memory");
  static_assert(kPre + (kMaxMats + 1) * 4 <= 232448, "shared memory");
};

struct ManyArgs {
  LinArgs L;
  const uint8_t* xt;     // [parts][in / 64][pad][128 bytes], swizzled
  const float* undo_x;   // [pad]
  long long pad;         // rows of the workspace
};

// --- rows of x into the workspace --------------------------------------------------

// A warp takes a row: its largest magnitude, then the values times a power of two that brings it to [2^14, 2^15), as f16
// (f32: two of them).  A lane writes 16 bytes: pairs j of the four groups of eight columns of a block, the order in which
// the conversion warps' stores put the codes; the 16-byte pieces of a row's 128 are swizzled by the row.
template <int DT>
__global__ void __launch_bounds__(256) linear_rows_kernel(const void* x, long long xs, int T, int in, uint8_t* xt, long long pad,
                                                          float* undo) {
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= T) return;
  constexpr int kPer = DT == kF32 ? 4 : 8;
  const char* src = static_cast<const char*>(x) + (long long)row * xs * (DT == kF32 ? 4 : 2);
  float most = 0.f;
  for (int i = lane; i < in / kPer; i += 32) {
    const uint4 u = reinterpret_cast<const uint4*>(src)[i];
    float f[kPer];
    if constexpr (DT == kF32)
      Val<float>::unpack(u, f);
    else if constexpr (DT == kF16)
      Val<__half>::unpack(u, f);
    else
      Val<__nv_bfloat16>::unpack(u, f);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float a = fabsf(f[j]);
      most = fmaxf(most, a < INFINITY ? a : 0.f);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  int e = 15;
  if (most > 0.f) frexpf(most, &e);
  const int up = max(-126, min(126, 15 - e));
  const float mul = pow2i(up);
  if (lane == 0) undo[row] = pow2i(-up);
  const long long part = (long long)(in / 64) * pad * 128;
  for (int i = lane; i < in / 8; i += 32) {
    const int first = (i >> 2) * 32 + (i & 3) * 2, ks = i >> 3, at = (i & 7) ^ (row & 7);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float a, b;
      if constexpr (DT == kF32) {
        const float2 t = *reinterpret_cast<const float2*>(src + (first + 8 * c) * 4);
        a = t.x, b = t.y;
      } else {
        const uint32_t t = *reinterpret_cast<const uint32_t*>(src + (first + 8 * c) * 2);
        if constexpr (DT == kF16) {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&t));
          a = h.x, b = h.y;
        } else {
          a = __uint_as_float(t << 16), b = __uint_as_float(t & 0xFFFF0000u);
        }
      }
      a *= mul, b *= mul;
      const __half2 h = __floats2half2_rn(a, b);
      hi[c] = *reinterpret_cast<const uint32_t*>(&h);
      if constexpr (DT == kF32) {
        const float2 back = __half22float2(h);
        lo[c] = pack_half2(a - back.x, b - back.y);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(xt + ((long long)ks * pad + row) * 128 + at * 16);
    *dst = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if constexpr (DT == kF32)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(dst) + part) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// --- tiles --------------------------------------------------------------------------

// A tile: 256 weight rows (128 of each stack where there are two) of one matrix and `cols` rows of x from row0, of which
// those from begin to end are the matrix's.  Tiles of x begin at a multiple of 8 rows, where the swizzle does.
struct Tile {
  int mat, mt, row0, cols, begin, end;
};

template <int COLS>
__device__ __forceinline__ int x_tiles(int begin, int end) {
  return end > begin ? (end - (begin & ~7) + COLS - 1) / COLS : 0;
}

template <int COLS>
__device__ __forceinline__ Tile tile_at(const LinArgs& L, const int* pre, int m_tiles, int item) {
  int a = 0, b = L.n;
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (pre[m] <= item)
      a = m;
    else
      b = m;
  }
  Tile t;
  t.mat = a;
  int begin, end;
  lin_rows(L, a, begin, end);
  const int base = begin & ~7, tiles = x_tiles<COLS>(begin, end);
  const int local = item - pre[a], nt = local / m_tiles;
  t.mt = local - nt * m_tiles;
  const int per = ((end - base + tiles - 1) / tiles + 31) & ~31;  // (at most COLS)
  t.row0 = base + nt * per;
  t.begin = max(begin, t.row0), t.end = min(end, t.row0 + per);
  t.cols = (t.end - t.row0 + 31) & ~31;
  return t;
}

// --- conversion ---------------------------------------------------------------------

__device__ __forceinline__ void tc_st_16x128_x8(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// A step of a tile, row g and row g + 8 of this lane, into the registers of a 16x128b store: the word's pair i goes to
// column 4 i + c of its block's 16, register 2 i (row g) or 2 i + 1 (row g + 8).  A masked code is the subnormal q 2^-24
// (or q 2^-20); times 2^15 (2^11) it is q 2^-9 exactly, and one fma with 512 s and m rounds once.
__device__ __forceinline__ void convert(const uint4& code, const uint4& rec, uint32_t (&r)[16]) {
  const __half2 up15 = __float2half2_rn(32768.f), up11 = __float2half2_rn(2048.f), k512 = __float2half2_rn(512.f);
  const uint32_t words[4] = {code.x, code.y, code.z, code.w};
  const __half2 s[2] = {__hmul2(as_half2(rec.x), k512), __hmul2(as_half2(rec.y), k512)};
  const __half2 m[2] = {as_half2(rec.z), as_half2(rec.w)};
#pragma unroll
  for (int wi = 0; wi < 4; ++wi) {
    const int row = wi & 1, blk = wi >> 1;
    const __half2 sv = blk ? __high2half2(s[row]) : __low2half2(s[row]);
    const __half2 mv = blk ? __high2half2(m[row]) : __low2half2(m[row]);
    const uint32_t w = words[wi], v = w >> 8;
    r[blk * 8 + 0 + row] = as_u32(__hfma2(__hmul2(as_half2(w & 0x000F000Fu), up15), sv, mv));
    r[blk * 8 + 2 + row] = as_u32(__hfma2(__hmul2(as_half2(w & 0x00F000F0u), up11), sv, mv));
    r[blk * 8 + 4 + row] = as_u32(__hfma2(__hmul2(as_half2(v & 0x000F000Fu), up15), sv, mv));
    r[blk * 8 + 6 + row] = as_u32(__hfma2(__hmul2(as_half2(v & 0x00F000F0u), up11), sv, mv));
  }
}

// The same in two parts: (16 + q) s + (m - 16 s) in f32, its f16 and what is left.
__device__ __forceinline__ void convert_two(const uint4& code, const uint4& rec, uint32_t (&hi)[16], uint32_t (&lo)[16]) {
  const uint32_t words[4] = {code.x, code.y, code.z, code.w};
  const uint32_t sr[2] = {rec.x, rec.y}, mr[2] = {rec.z, rec.w};
#pragma unroll
  for (int wi = 0; wi < 4; ++wi) {
    const int row = wi & 1, blk = wi >> 1;
    const float2 sp = __half22float2(as_half2(sr[row])), mp = __half22float2(as_half2(mr[row]));
    const float s = blk ? sp.y : sp.x, m = fmaf(-16.f, s, blk ? mp.y : mp.x);
    const uint32_t w = words[wi];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = w << (19 - 4 * i), b = i == 0 ? w << 3 : w >> (4 * i - 3);
      const float v0 = fmaf(__uint_as_float((a & 0x00780000u) | 0x41800000u), s, m);
      const float v1 = fmaf(__uint_as_float((b & 0x00780000u) | 0x41800000u), s, m);
      const __half2 h = __floats2half2_rn(v0, v1);
      const float2 back = __half22float2(h);
      hi[blk * 8 + 2 * i + row] = as_u32(h);
      lo[blk * 8 + 2 * i + row] = pack_half2(v0 - back.x, v1 - back.y);
    }
  }
}

// --- results ------------------------------------------------------------------------

__device__ __forceinline__ uint32_t pack16(int dtype, float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  const __half2 y = __floats2half2_rn(a, b);
  return dtype == kBF16 ? *reinterpret_cast<const uint32_t*>(&x) : as_u32(y);
}

// A lane's 16 results of one weight row f for rows r0.. of x.  16-bit types: neighbouring lanes trade, so that each
// stores two weight rows of one row of x.
template <bool TWO>
__device__ __forceinline__ void store16(const LinArgs& L, const float (&v)[16], int r0, int begin, int end, int f, int lane) {
  if constexpr (TWO) {
    float* y = static_cast<float*>(L.y) + f;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (r0 + j >= begin && r0 + j < end && f < L.out) y[(long long)(r0 + j) * L.ys] = v[j];
  } else {
    const int odd = lane & 1;
    uint16_t* y = static_cast<uint16_t*>(L.y) + (f - odd);
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const float give = odd ? v[j] : v[j + 1], keep = odd ? v[j + 1] : v[j];
      const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
      const uint32_t two = odd ? pack16(L.dtype, got, keep) : pack16(L.dtype, keep, got);
      const int r = r0 + j + odd;
      if (r >= begin && r < end && f < L.out) *reinterpret_cast<uint32_t*>(y + (long long)r * L.ys) = two;
    }
  }
}

// --- the kernel ---------------------------------------------------------------------

template <bool TWO, bool GLU>
__global__ void __launch_bounds__(kManyThreads, 1) linear_many_kernel(const __grid_constant__ ManyArgs A) {
  using P = ManyPlan<TWO>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const LinArgs& L = A.L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::kBars);
  uint64_t *x_full = bars, *x_empty = bars + 8, *a_full = bars + 16, *a_empty = bars + 18, *d_full = bars + 20,
           *d_empty = bars + 22, *last = bars + 24;
  uint32_t* tmem_word = reinterpret_cast<uint32_t*>(smem + P::kMisc);
  volatile int* dead = reinterpret_cast<volatile int*>(smem + P::kMisc + 8);
  int* pre = reinterpret_cast<int*>(smem + P::kPre);
  unsigned* err = L.err;
  if (smem_u32(smem) & 1023) {  // the swizzle counts on it
    if (tid == 0) atomicOr(err, kErrConfig);
    return;
  }
  const int nks = L.in / kLinStep, w_tiles = L.out / kLinTile;
  const int m_tiles = (L.out + (GLU ? 127 : 255)) / (GLU ? 128 : 256);
  if (tid == 0) {
    for (int i = 0; i < P::kStages; ++i) mbar_init(&x_full[i], 1), mbar_init(&x_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&a_full[i], 8), mbar_init(&a_empty[i], 1);
    for (int i = 0; i < P::kSets; ++i) mbar_init(&d_full[i], 1), mbar_init(&d_empty[i], 8);
    mbar_init(last, 1);
    *dead = 0;
    fence_mbar_init();
  }
  if (warp == 0) {  // tiles before each matrix
    const int share = (L.n + 31) / 32, i0 = min(L.n, lane * share), i1 = min(L.n, i0 + share);
    int sum = 0;
    for (int i = i0; i < i1; ++i) {
      int begin, end;
      if (!lin_rows(L, i, begin, end) && blockIdx.x == 0) atomicOr(err, kErrIndex);
      sum += x_tiles<P::kCols>(begin, end) * m_tiles;
      pre[i + 1] = sum;
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += t;
    }
    for (int i = i0; i < i1; ++i) pre[i + 1] += upto - sum;
    if (lane == 0) pre[0] = 0;
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_word)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  const int total = pre[L.n];

  if (warp < 8) {
    // ---- conversion: codes of two tiles of 16 weight rows, a step at a time ----
    const int quarter = warp & 3, half = warp >> 2;
    uint8_t* fifo = smem + P::kFifoOff + warp * (kFifo * kFifoStep);
    const uint32_t lanes = tmem + ((uint32_t)quarter << 21) + P::kA + half * 32 * P::kParts;
    // what is fetched next: a step of an item's two tiles
    int f_item = blockIdx.x, f_ks = 0, f_slot = 0;
    const uint8_t *src0 = nullptr, *src1 = nullptr;
    auto find = [&]() {
      src0 = src1 = nullptr;
      if (f_item >= total) return;
      const Tile t = tile_at<P::kCols>(L, pre, m_tiles, f_item);
      const LinMat& w = L.w[GLU ? half : 0];
      const int wt = (GLU ? t.mt * 8 : t.mt * 16 + half * 8) + quarter * 2;
      const uint8_t* base = w.packed + ((long long)t.mat * w_tiles + wt) * nks * kLinStepBytes;
      if (wt < w_tiles) src0 = base;
      if (wt + 1 < w_tiles) src1 = base + (long long)nks * kLinStepBytes;
    };
    auto fetch = [&]() {
      uint8_t* slot = fifo + f_slot * kFifoStep;
      if (src0) {
        cp_async16(slot + lane * 16, src0 + lane * 16);
        if (lane < 8) cp_async16(slot + 512 + lane * 16, src0 + 512 + lane * 16);
        src0 += kLinStepBytes;
      }
      if (src1) {
        cp_async16(slot + kLinStepBytes + lane * 16, src1 + lane * 16);
        if (lane < 8) cp_async16(slot + kLinStepBytes + 512 + lane * 16, src1 + 512 + lane * 16);
        src1 += kLinStepBytes;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (++f_slot == kFifo) f_slot = 0;
      if (f_item < total && ++f_ks == nks) {
        f_ks = 0, f_item += gridDim.x;
        find();
      }
    };
    find();
    for (int i = 0; i < kFifo - 1; ++i) fetch();
    int at = 0, slot_at = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
      const Tile t = tile_at<P::kCols>(L, pre, m_tiles, item);
      const int wt = (GLU ? t.mt * 8 : t.mt * 16 + half * 8) + quarter * 2;
      for (int ks = 0; ks < nks; ++ks, ++at) {
        __syncwarp();  // the slot of the step before has been read
        fetch();
        asm volatile("cp.async.wait_group %0;" ::"n"(kFifo - 1) : "memory");
        __syncwarp();
        const uint8_t* slot = fifo + slot_at * kFifoStep;
        if (++slot_at == kFifo) slot_at = 0;
        const int st = at & 1;
        const uint32_t to = lanes + st * 64 * P::kParts;
        bool waited = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (wt + h >= w_tiles) break;  // its lanes' results are not used
          const uint4 code = *reinterpret_cast<const uint4*>(slot + h * kLinStepBytes + lane * 16);
          const uint4 rec = *reinterpret_cast<const uint4*>(slot + h * kLinStepBytes + 512 + (lane >> 2) * 16);
          uint32_t r[16], r_lo[TWO ? 16 : 1];
          if constexpr (TWO)
            convert_two(code, rec, r, r_lo);
          else
            convert(code, rec, r);
          if (!waited) {
            waited = true;
            if (at >= 2 && !(ok = wait_warp(&a_empty[st], ((at >> 1) - 1) & 1, dead, err))) break;
            tc_fence_after();
          }
          tc_st_16x128_x8(to + ((uint32_t)(16 * h) << 16), r);
          if constexpr (TWO) tc_st_16x128_x8(to + 32 + ((uint32_t)(16 * h) << 16), r_lo);
        }
        if (!ok) break;
        if (!waited && at >= 2 && !(ok = wait_warp(&a_empty[st], ((at >> 1) - 1) & 1, dead, err))) break;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&a_full[st]);
      }
    }
    cp_async_wait_all();
  } else if (warp < 16) {
    // ---- results: 32 weight rows of each half, half of the tile's rows of x ----
    const int quarter = warp & 3, side = (warp - 8) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)quarter << 21);
    int chunk = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
      const Tile t = tile_at<P::kCols>(L, pre, m_tiles, item);
      const int f0 = (GLU ? t.mt * 128 : t.mt * 256) + quarter * 32 + lane;
      const int halves = GLU || t.mt * 256 + 128 < L.out ? 2 : 1;
      const int r0 = t.row0 + side * (t.cols >> 1), mine = t.cols >> 1;
      float undo[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f = GLU ? f0 : f0 + h * 128;
        undo[h] = f < L.out ? __ldg(L.w[GLU ? h : 0].undo + (long long)t.mat * L.out + f) : 0.f;
      }
      if constexpr (!TWO) {
        if (!(ok = wait_warp(&d_full[0], chunk & 1, dead, err))) break;
        tc_fence_after();
        for (int c = 0; c < mine; c += 16) {
          const float ux = __ldg(A.undo_x + r0 + c + (lane & 15));
          float v[2][16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h >= halves) break;
            uint32_t r[16];
            tc_ld16(lanes + h * P::kCols + side * mine + c, r);
            tc_wait_ld(r);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[h][j] = __uint_as_float(r[j]) * undo[h] * __shfl_sync(0xFFFFFFFFu, ux, j);
            if constexpr (!GLU) store16<TWO>(L, v[h], r0 + c, t.begin, t.end, f0 + h * 128, lane);
          }
          if constexpr (GLU) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[0][j] = silu_f32(v[0][j]) * v[1][j];
            store16<TWO>(L, v[0], r0 + c, t.begin, t.end, f0, lane);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[0]);
        ++chunk;
      } else {
        float acc[2][2][16];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[h][c][j] = 0.f;
        for (int ks = 0; ks < nks; ks += kChunk, ++chunk) {
          const int set = chunk & 1;
          if (!(ok = wait_warp(&d_full[set], (chunk >> 1) & 1, dead, err))) break;
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (h < halves && c * 16 < mine) {
                uint32_t r[16];
                tc_ld16(lanes + (set * 2 + h) * P::kCols + side * mine + c * 16, r);
                tc_wait_ld(r);
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[h][c][j] += __uint_as_float(r[j]);
              }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_empty[set]);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c * 16 >= mine) break;
          const float ux = __ldg(A.undo_x + r0 + c * 16 + (lane & 15));
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[h][c][j] *= undo[h] * __shfl_sync(0xFFFFFFFFu, ux, j);
          if constexpr (GLU) {
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[0][c][j] = silu_f32(acc[0][c][j]) * acc[1][c][j];
          }
#pragma unroll
          for (int h = 0; h < (GLU ? 1 : 2); ++h)
            if (h < halves) store16<TWO>(L, acc[h][c], r0 + c * 16, t.begin, t.end, f0 + h * 128, lane);
        }
      }
    }
  } else if (warp == kLoadWarp) {
    // ---- copies of x ----
    if (lane == 0) {
      int copies = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
        const Tile t = tile_at<P::kCols>(L, pre, m_tiles, item);
        const uint32_t bytes = (uint32_t)t.cols * 128;
        for (int ks = 0; ks < nks; ++ks, ++copies) {
          const int st = copies % P::kStages, round = copies / P::kStages;
          if (round > 0 && !(ok = wait_for(&x_empty[st], (round - 1) & 1, dead, err))) break;
          mbar_arrive_expect_tx(&x_full[st], bytes * P::kParts);
#pragma unroll
          for (int p = 0; p < P::kParts; ++p)
            bulk_g2s(smem + st * P::kStage + p * P::kPart, A.xt + (((long long)p * nks + ks) * A.pad + t.row0) * 128, bytes,
                     &x_full[st]);
        }
      }
      for (int i = max(0, copies - P::kStages); i < copies; ++i)  // the copies have landed before the CTA ends
        mbar_wait(&x_full[i % P::kStages], (i / P::kStages) & 1, err);
    }
    __syncwarp();
  } else {
    // ---- products ----
    int at = 0, chunk = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
      const Tile t = tile_at<P::kCols>(L, pre, m_tiles, item);
      const int halves = GLU || t.mt * 256 + 128 < L.out ? 2 : 1;
      const uint32_t id = 1u << 4 | (uint32_t)(t.cols >> 3) << 17 | (uint32_t)(128 >> 4) << 24;  // f16, f32, M = 128
      int set = 0;
      for (int ks = 0; ks < nks; ++ks, ++at) {
        const bool first = TWO ? ks % kChunk == 0 : ks == 0;
        if (first) {
          set = chunk % P::kSets;
          const int round = chunk / P::kSets;
          if (round > 0 && !(ok = wait_warp(&d_empty[set], (round - 1) & 1, dead, err))) break;
          ++chunk;
        }
        const int st = at & 1, xst = at % P::kStages;
        if (!(ok = wait_warp(&x_full[xst], (at / P::kStages) & 1, dead, err))) break;
        if (!(ok = wait_warp(&a_full[st], (at >> 1) & 1, dead, err))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b = tc_desc(smem + xst * P::kStage, 1024, 0);
          const uint64_t b_lo = tc_desc(smem + xst * P::kStage + (P::kParts - 1) * P::kPart, 1024, 0);
          for (int h = 0; h < halves; ++h) {
            const uint32_t d = tmem + (set * 2 + h) * P::kCols;
            const uint32_t a = tmem + P::kA + (st * 2 + h) * 32 * P::kParts;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              tc_mma_ts(d, a + y * 8, b + y * 2, id, !first || y > 0);
              if constexpr (TWO) {
                tc_mma_ts(d, a + y * 8, b_lo + y * 2, id, 1);
                tc_mma_ts(d, a + 32 + y * 8, b + y * 2, id, 1);
              }
            }
          }
          tc_commit(&a_empty[st]);
          tc_commit(&x_empty[xst]);
          if (ks == nks - 1 || (TWO && ks % kChunk == kChunk - 1)) tc_commit(&d_full[set]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) tc_commit(last);
    __syncwarp();
    mbar_wait(last, 0, err);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <bool TWO>
int smem_bytes(int n) { return ManyPlan<TWO>::kPre + (n + 1) * 4; }

template <bool TWO, bool GLU>
cudaError_t launch(const ManyArgs& A, int nsm, cudaStream_t s) {
  linear_many_kernel<TWO, GLU><<<nsm, kManyThreads, smem_bytes<TWO>(A.L.n), s>>>(A);
  return cudaGetLastError();
}

template <bool TWO, bool GLU>
cudaError_t setup() {
  return cudaFuncSetAttribute(linear_many_kernel<TWO, GLU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              smem_bytes<TWO>(kMaxMats));
}

// Rows of the workspace: a tile's copies may pass a matrix's last row by less than a tile.
long long pad_rows(int max_rows) { return (((long long)max_rows + 7) & ~7LL) + 192; }

}  // namespace

long long linear_many_workspace(int in, int max_rows) { return pad_rows(max_rows) * (4LL * in + 4); }

cudaError_t setup_linear_many() {
  const cudaError_t e[4] = {setup<false, false>(), setup<false, true>(), setup<true, false>(), setup<true, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t launch_linear_many(const LinArgs& L, void* workspace, int max_rows, int nsm, cudaStream_t s) {
  ManyArgs A;
  A.L = L;
  A.pad = pad_rows(max_rows);
  uint8_t* xt = static_cast<uint8_t*>(workspace);
  float* undo = reinterpret_cast<float*>(xt + A.pad * 4 * L.in);
  A.xt = xt, A.undo_x = undo;
  const unsigned grid = (unsigned)((L.T + 7) / 8);
  if (L.dtype == kF32)
    linear_rows_kernel<kF32><<<grid, 256, 0, s>>>(L.x, L.xs, L.T, L.in, xt, A.pad, undo);
  else if (L.dtype == kF16)
    linear_rows_kernel<kF16><<<grid, 256, 0, s>>>(L.x, L.xs, L.T, L.in, xt, A.pad, undo);
  else
    linear_rows_kernel<kBF16><<<grid, 256, 0, s>>>(L.x, L.xs, L.T, L.in, xt, A.pad, undo);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (L.dtype == kF32) return L.glu ? launch<true, true>(A, nsm, s) : launch<true, false>(A, nsm, s);
  return L.glu ? launch<false, true>(A, nsm, s) : launch<false, false>(A, nsm, s);
}

}  // namespace strata
