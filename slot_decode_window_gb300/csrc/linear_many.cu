// Products of many rows with 4-bit matrices on the 5th-generation tensor cores.
//
// D = W X^T for 256 weight rows (two halves of 128: the second half, or the
// stack behind the gate) and up to 128 rows of x (64 of f32 rows, 192 with rounded
// weights): weights are the A operand, in tensor memory, where the conversion warps write them as f16 from
// the 4-bit codes, 64 columns at a time; x is the B operand, f16 in the order of
// the codes, swizzled, brought by bulk copies from the workspace that
// linear_rows_kernel fills.  Weight rows on the M side leave the rows of x free
// to be few: an expert with 20 rows costs 32 columns, not 128.
//
// bf16 rows: one product, W rounded to f16 (2^-11 of a weight against the 2^-8 of
// the results' own rounding).  f16 and f32 rows: exact weights,
//   W x = s (q - 8) x + (8 s + m) sum x   over a block of 32 columns:
// s (q - 8) has 15 bits, two f16 parts (hi and what is left, both exact); after the
// last columns come steps whose "weights" are m and 8 s of 16 blocks each and
// whose "x" are the blocks' sums, in two f16 parts.  16-bit rows: hi x + lo x.  f32 rows: x
// in two f16 parts (22 bits), lo hi + hi lo + hi hi; the accumulators' adds
// truncate, so every two steps they are added to f32 registers, with two sets of
// accumulators in turn; so are f16 rows of more than 29120 columns.
// Rounded weights (bf16 rows, where the caller asks for them): one product, W
// rounded to f16, 2^-11 of a weight.
//
// Roles (28 warps): 16 of conversion, in two groups that take a block of 32 columns
// each of every step (rounded weights: the steps in turn), with stages of
// weights of their own (a warp has two tiles of 16 weight rows, a quarter of the
// lanes of one half); 8 of results (each a quarter of the lanes
// and half of the rows of x); one of copies, codes and x of a step into one stage;
// one for each half that issues its products (and one that fills the warpgroup).  A step has to pass in 768 clocks (1024 of
// 16-bit rows with exact weights) for the tensor cores never to wait, and a warp's waits and hand-overs alone take about
// as many: hence the two groups, and two warps that issue.  CTAs (one per SM) take
// the tiles of all matrices in turn, weight rows fastest, so that concurrent CTAs
// share rows of x in L2.  Where there are fewer tiles than SMs, a cluster of 2, 4 or
// 8 CTAs takes a tile, each a part of its columns; a CTA sends its part of the
// results to those that add them up (each a share of the rows of x, in the cluster's
// order) through distributed shared memory.
// Measured: 8191 bf16 or f16 rows of 2048 -> 5120 234 to 239 us (1.45 PFLOP/s of the two products, 76% of the measured cuBLAS rate;
// rounded weights 130 us), of which 14 us prepare the rows; 2041 f32 rows of 4096 -> 2048 108 us (three products: 0.95 PFLOP/s with the
// preparation, 1.7 waves of tiles); 128 experts' gate and up of 2048 -> 768 for 32104 bf16 rows 386 us (rounded 213 us), 46 us of it the
// rows (HBM), down 227 us (rounded 142 us); 512 rows over those experts, gate and up, 143 us, 152 us of f32; 203 f16 rows with gate
// 2048 -> 4096 27 us; 64 bf16 rows of 4096 -> 4096 20 us in a graph.  Tiles of fewer than some 170 rows of x are bound by the roles'
// instructions and hand-overs, some 650 clocks a step with rounded weights.
#include "linear.cuh"
#include "tcgen05.cuh"

namespace strata {
namespace {

constexpr int kConvert = 16, kResults = 8;    // warps
constexpr int kLoadWarp = kConvert + kResults, kMmaWarp = kLoadWarp + 1;
constexpr int kManyThreads = (kConvert + kResults + 4) * 32;
constexpr int kRegs = 72;  // registers a thread at launch; the roles' shares below are drawn from them
constexpr int kHalfCodes = 8 * kLinStepBytes; // a step of 128 weight rows
constexpr int kChunk = 2;                     // steps between sums of f32 rows
constexpr int kGroup = 8;                     // steps whose blocks' sums are one step
constexpr int kMaxMats = 1024;
// Kinds of rows besides strata_dtype's: bf16 rows with exact weights (kBF16: with weights rounded to f16), f16 rows of many columns.
constexpr int kBF16X = 3, kF16Long = 4;
constexpr int value_type(int kind) { return kind == kBF16X ? kBF16 : kind == kF16Long ? kF16 : kind; }

template <int DT> struct ManyPlan {
  static constexpr bool kSums = DT != kBF16;     // exact weights
  static constexpr int kXParts = DT == kF32 ? 2 : 1, kWParts = kSums ? 2 : 1;
  static constexpr int kCols = DT == kF32 ? 64 : DT == kBF16 ? 192 : 128;  // most rows of x in a tile
  static constexpr int kSets = DT == kF32 ? 2 : 1;  // of accumulators
  static constexpr int kA = 2 * kSets * kCols;   // first column of the weights in tensor memory
  static constexpr int kStages = DT == kBF16 ? 6 : 8;  // of copies (even: a group's steps keep to its stages)
  static constexpr int kPart = kCols * 128;      // bytes of a part of a step of x
  static constexpr int kCodes = kPart * kXParts; // where a stage has its codes
  static constexpr int kStage = kCodes + 2 * kHalfCodes;
  static constexpr int kBars = kStages * kStage;
  static constexpr int kMisc = kBars + 256;
  static constexpr int kPre = kMisc + 64;        // [n + 1] tiles before each matrix
  static constexpr int kUnits = kSums ? 4 : 2;   // stages of weights: 32 columns each, or 64
  static constexpr int kRegConvert = 56, kRegResults = 120, kRegIssue = 40;
  static_assert(kConvert * kRegConvert + kResults * kRegResults + 4 * kRegIssue <= (kConvert + kResults + 4) * kRegs, "register split");
  static_assert(kStage % 1024 == 0 && kStages % 2 == 0, "stages");
  static_assert(kA + 4 * 32 * kWParts <= 512, "tensor memory");
  static_assert(kPre + (kMaxMats + 1) * 4 <= 232448, "shared memory");
};

// As f32 rows, with one part of x (the place of the other is not used).
template <> struct ManyPlan<kF16Long> : ManyPlan<kF32> {
  static constexpr int kXParts = 1;
};

__host__ __device__ inline int sum_steps(int nks) { return (nks + kGroup - 1) / kGroup; }

struct ManyArgs {
  LinArgs L;
  const uint8_t* xt;     // [parts][in / 64][pad][128 bytes], swizzled, then [groups][pad][128 bytes] of sums (f16, f32)
  const float* undo_x;   // [pad]
  long long pad;         // rows of the workspace
  int split;             // CTAs of a cluster that share a tile's columns
};

__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// --- rows of x into the workspace --------------------------------------------------

// `warps` warps of a CTA take a row: its largest magnitude, then the values times a power of two that brings it to
// [2^14, 2^15) ([2^9, 2^10) where sums are formed), as f16 (f32: two of them).  A lane has eight columns of a block of 32 at
// a time, kOct of them in registers between the two passes (longer rows are read again).  The four lanes of a block trade
// pairs, so that lane j stores pairs j of all four: 16 bytes, in the order in which the conversion warps' stores put the
// codes; the 16-byte pieces of a row's 128 are swizzled by the row.  The blocks' sums go to steps of their own, in the order of
// `convert_sums`; blocks past the last are zeros.
template <int DT> struct RowsPlan {
  static constexpr int kOct = DT == kF32 ? 4 : 8;
};
template <int DT>
__global__ void __launch_bounds__(256) linear_rows_kernel(const void* x, long long xs, int T, int in, int warps, uint8_t* xt,
                                                          long long pad, float* undo) {
  constexpr int kOct = RowsPlan<DT>::kOct, kWords = DT == kF32 ? 2 : 1;  // 16-byte words of eight columns
  constexpr bool kSums = ManyPlan<DT>::kSums;
  __shared__ float part[8];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * (8 / warps) + warp / warps, mine = (warp % warps) * 32 + lane, step = warps * 32;
  const bool live = row < T;  // (the CTA meets at a barrier)
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + (long long)(live ? row : 0) * xs * (DT == kF32 ? 4 : 2));
  const int octets = in / 8, all = kSums ? sum_steps(in / 64) * kGroup * 8 : octets;
  auto values = [](const uint4 (&u)[kWords], float (&f)[8]) {
    if constexpr (DT == kF32) {
      Val<float>::unpack(u[0], f);
      Val<float>::unpack(u[1], f + 4);
    } else if constexpr (DT == kF16) {
      Val<__half>::unpack(u[0], f);
    } else {
      Val<__nv_bfloat16>::unpack(u[0], f);
    }
  };
  uint4 held[kOct][kWords];
  float most = 0.f;
  auto look = [&](const uint4 (&u)[kWords]) {
    float f[8];
    values(u, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(f[j]);
      most = fmaxf(most, a < INFINITY ? a : 0.f);
    }
  };
#pragma unroll
  for (int k = 0; k < kOct; ++k) {
    const int i = mine + k * step;
#pragma unroll
    for (int w = 0; w < kWords; ++w) held[k][w] = live && i < octets ? src[i * kWords + w] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < kOct; ++k) look(held[k]);
  for (int i = mine + kOct * step; live && i < octets; i += step) {
    uint4 u[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w) u[w] = src[i * kWords + w];
    look(u);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  if (warps > 1) {
    if (lane == 0) part[warp] = most;
    __syncthreads();
    for (int w = 0; w < warps; ++w) most = fmaxf(most, part[warp / warps * warps + w]);
  }
  if (!live) return;
  constexpr int kTop = kSums ? 10 : 15;  // (a block's sum has to be an f16 too)
  int e = kTop;
  if (most > 0.f) frexpf(most, &e);
  const int up = max(-126, min(126, kTop - e));
  const float mul = pow2i(up);
  if (mine == 0) undo[row] = pow2i(-up);
  const long long next = (long long)(in / 64) * pad * 128;  // from a part to the other
  uint8_t* sums = xt + next * ManyPlan<DT>::kXParts;
  auto put = [&](int i, const uint4 (&u)[kWords]) {
    const int ks = i >> 3, j = i & 3, odd = lane & 1, two = lane & 2;
    float f[8], sum = 0.f;
    values(u, f);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float a = f[2 * c] * mul, b = f[2 * c + 1] * mul;
      sum += a + b;
      const __half2 h = __floats2half2_rn(a, b);
      hi[c] = as_u32(h);
      if constexpr (DT == kF32) {
        const float2 back = __half22float2(h);
        lo[c] = pack_half2(a - back.x, b - back.y);
      }
    }
    auto trade = [&](uint32_t (&r)[4]) {  // r[c] of lane l becomes r[l] of lane c, within the four lanes
      const uint32_t s0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? r[0] : r[1], 1), s1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? r[2] : r[3], 1);
      if (odd) r[0] = s0, r[2] = s1;
      else r[1] = s0, r[3] = s1;
      const uint32_t t0 = __shfl_xor_sync(0xFFFFFFFFu, two ? r[0] : r[2], 2), t1 = __shfl_xor_sync(0xFFFFFFFFu, two ? r[1] : r[3], 2);
      if (two) r[0] = t0, r[1] = t1;
      else r[2] = t0, r[3] = t1;
    };
    trade(hi);
    if constexpr (DT == kF32) trade(lo);
    if (i < octets) {
      uint8_t* dst = xt + ((long long)ks * pad + row) * 128 + ((i & 7) ^ (row & 7)) * 16;
      *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if constexpr (DT == kF32) *reinterpret_cast<uint4*>(dst + next) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    if constexpr (kSums) {
      // the block's sum (at most 2^15) in two parts, to the columns of its min (lane 0 of the four) and its 8 s (lane 1)
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      const int blk = (i >> 2) & 1, at = ks % kGroup, piece = (at >> 2) * 4 + blk * 2 + j;
      const __half h = __float2half_rn(sum);
      if (j < 2 && i < all)
        *reinterpret_cast<uint32_t*>(sums + ((long long)(ks / kGroup) * pad + row) * 128 + (piece ^ (row & 7)) * 16 + (at & 3) * 4) =
            pack_half2(__half2float(h), sum - __half2float(h));
    }
  };
#pragma unroll
  for (int k = 0; k < kOct; ++k)
    if (k * step < all) put(mine + k * step, held[k]);
  for (int i = kOct * step; i < all; i += step) {  // (whole warps: lanes past the end trade zeros)
    uint4 u[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w) u[w] = i + mine < octets ? src[(i + mine) * kWords + w] : make_uint4(0, 0, 0, 0);
    put(i + mine, u);
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

__device__ __forceinline__ void tc_st_16x128_x4(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Products and commits of the lane whose `lead` is not 0, without a branch.
__device__ __forceinline__ void tc_mma_ts_if(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
// Two products, 16 columns on, and a look at a barrier: whether its phase is complete.  The look is issued first and its answer
// read last, so that the products do not wait for it.
__device__ __forceinline__ uint32_t tc_mma_pair_look(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                                     uint64_t* bar, uint32_t parity) {
  uint32_t seen;
  asm volatile(
      "{\n.reg .pred p, q, t, s;\n.reg .b32 a1;\n.reg .b64 b1;\n"
      "mbarrier.test_wait.parity.shared::cta.b64 s, [%7], %8;\n"
      "setp.ne.u32 p, %5, 0;\nsetp.ne.u32 q, %6, 0;\nsetp.eq.u32 t, 0, 0;\nadd.u32 a1, %2, 8;\nadd.u64 b1, %3, 2;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [a1], b1, %4, t;\n"
      "selp.u32 %0, 1, 0, s;\n}"
      : "=r"(seen)
      : "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead), "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return seen;
}
__device__ __forceinline__ void tc_commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.u32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)), "r"(lead)
      : "memory");
}

// A step of a tile, row g and row g + 8 of this lane, into the registers of a 16x128b store: the word's pair i goes to
// column 4 i + c of its block's 16, register 2 i (row g) or 2 i + 1 (row g + 8).  A masked code is the subnormal q 2^-24 (or
// q 2^-20), the records' scales carry the 2^24, so a pair is one mask and one fma, which rounds once (a min that is then below
// f16's least normal number is rounded before).
__device__ __forceinline__ void convert(const uint4& code, const uint4& rec, uint32_t (&r)[16]) {
  const __half2 k16 = __float2half2_rn(0.0625f);
  const uint32_t words[4] = {code.x, code.y, code.z, code.w};
  const __half2 s[2] = {as_half2(rec.x), as_half2(rec.y)}, down = __float2half2_rn(1.f / kLinMin);
  const __half2 m[2] = {__hmul2(as_half2(rec.z), down), __hmul2(as_half2(rec.w), down)};
  const __half2 s16[2] = {__hmul2(s[0], k16), __hmul2(s[1], k16)};
#pragma unroll
  for (int wi = 0; wi < 4; ++wi) {
    const int row = wi & 1, blk = wi >> 1;
    const __half2 sv = blk ? __high2half2(s[row]) : __low2half2(s[row]);
    const __half2 tv = blk ? __high2half2(s16[row]) : __low2half2(s16[row]);
    const __half2 mv = blk ? __high2half2(m[row]) : __low2half2(m[row]);
    const uint32_t w = words[wi], v = w >> 8;
    r[blk * 8 + 0 + row] = as_u32(__hfma2(as_half2(w & 0x000F000Fu), sv, mv));
    r[blk * 8 + 2 + row] = as_u32(__hfma2(as_half2(w & 0x00F000F0u), tv, mv));
    r[blk * 8 + 4 + row] = as_u32(__hfma2(as_half2(v & 0x000F000Fu), sv, mv));
    r[blk * 8 + 6 + row] = as_u32(__hfma2(as_half2(v & 0x00F000F0u), tv, mv));
  }
}

// 2^18 s (q - 8) in two parts, both exact: the code in the mantissa of 1024 (or of 64) less 1032 (72) is q - 8, and the
// product's f16 leaves at most 5 bits.  2^18 is the mins' factor, which results lose again.  s is the records' scale times 2^-6,
// [2^8, 2^9) for the row's largest: down to 2^-22 of that it keeps all of its bits.
constexpr float kTwoUndo = 1.f / kLinMin;
__device__ __forceinline__ void convert_two(const uint2& code, const uint2& scale, int blk, uint32_t (&hi)[8], uint32_t (&lo)[8]) {
  const __half2 low = __float2half2_rn(-1032.f), high = __float2half2_rn(-72.f), down = __float2half2_rn(kLinMin / kLinScale);
#pragma unroll
  for (int row = 0; row < 2; ++row) {
    const uint32_t word = row ? code.y : code.x;
    const __half2 s = __hmul2(as_half2(row ? scale.y : scale.x), down), sv = blk ? __high2half2(s) : __low2half2(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? word : word >> 8;
      const __half2 q = i & 1 ? __hadd2(as_half2((w & 0x00F000F0u) | 0x54005400u), high)
                              : __hadd2(as_half2((w & 0x000F000Fu) | 0x64006400u), low);
      const __half2 h = __hmul2(q, sv);
      hi[2 * i + row] = as_u32(h);
      lo[2 * i + row] = as_u32(__hfma2(q, sv, __hneg2(h)));
    }
  }
}

// The weights of half a step of sums (16 columns) from the record of step c (first half) or 4 + c of the group: 2^18 m in column
// 4 i + c for even i, 2^18 8 s for odd i, i / 2 the block; a column's two f16 meet the sum's two parts.
__device__ __forceinline__ void convert_sums(const uint4& rec, uint32_t (&r)[8]) {
  const __half2 down = __float2half2_rn(8.f * kLinMin / kLinScale);
  const __half2 s[2] = {__hmul2(as_half2(rec.x), down), __hmul2(as_half2(rec.y), down)};
  const __half2 m[2] = {as_half2(rec.z), as_half2(rec.w)};
#pragma unroll
  for (int row = 0; row < 2; ++row) {
    r[0 + row] = as_u32(__low2half2(m[row]));
    r[2 + row] = as_u32(__low2half2(s[row]));
    r[4 + row] = as_u32(__high2half2(m[row]));
    r[6 + row] = as_u32(__high2half2(s[row]));
  }
}

// --- results ------------------------------------------------------------------------

template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (value_type(DT) == kF16) return pack_half2(a, b);
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// Two products in one instruction.
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y) {
  asm("{\n.reg .b64 p, q;\nmov.b64 p, {%0, %1};\nmov.b64 q, {%2, %3};\nmul.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  asm("{\n.reg .b64 p, q;\nmov.b64 p, {%0, %1};\nmov.b64 q, {%2, %3};\nadd.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

// A lane's 16 results of one weight row f for rows r0.. of x; those from begin to end are stored.  16-bit types:
// neighbouring lanes trade, so that each stores two weight rows of every other row of x.
template <int DT>
__device__ __forceinline__ void store16(const LinArgs& L, const float (&v)[16], int r0, int begin, int end, int f, int lane) {
  if (f - lane >= L.out) return;  // the warp's 32 weight rows are all past the last
  const bool all = r0 >= begin && r0 + 16 <= end, mine = f < L.out;
  if constexpr (DT == kF32) {
    float* y = static_cast<float*>(L.y) + (long long)r0 * L.ys + f;
#pragma unroll
    for (int j = 0; j < 16; ++j, y += L.ys)
      if (mine && (all || (r0 + j >= begin && r0 + j < end))) *y = v[j];
  } else {
    const int odd = lane & 1;
    const uint32_t pick = odd ? 0x3276u : 0x5410u;  // own and got: even lanes take the lower halves, odd ones the upper
    uint16_t* y = static_cast<uint16_t*>(L.y) + (long long)(r0 + odd) * L.ys + (f - odd);
#pragma unroll
    for (int j = 0; j < 16; j += 2, y += 2 * L.ys) {
      const uint32_t own = pack16<DT>(v[j], v[j + 1]);
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
      const uint32_t two = __byte_perm(own, got, pick);
      const int r = r0 + j + odd;
      if (mine && (all || (r >= begin && r < end))) *reinterpret_cast<uint32_t*>(y) = two;
    }
  }
}

// Powers of two of rows of x.  Ordinary loads: the kernel that writes them runs beside this one's start, and the read-only path
// is for what does not change while a kernel lives.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = load4(p + 4 * i);
    v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
  }
}

// The same for two rows of x (all lanes of a warp call it).
template <int DT>
__device__ __forceinline__ void store2(const LinArgs& L, const float* v, int r0, int begin, int end, int f, int lane) {
  if (f - lane >= L.out) return;
  const bool mine = f < L.out;
  if constexpr (DT == kF32) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (mine && r0 + j >= begin && r0 + j < end) static_cast<float*>(L.y)[(long long)(r0 + j) * L.ys + f] = v[j];
  } else {
    const int odd = lane & 1, r = r0 + odd;
    const uint32_t own = pack16<DT>(v[0], v[1]);
    const uint32_t two = __byte_perm(own, __shfl_xor_sync(0xFFFFFFFFu, own, 1), odd ? 0x3276u : 0x5410u);
    if (mine && r >= begin && r < end)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(L.y) + (long long)r * L.ys + (f - odd)) = two;
  }
}

// A cluster's parts of a tile, in the shared memory of the CTA that adds them up (where the stages of copies were):
// [part][half][row of x of its share][128 weight rows] f32.
__device__ __forceinline__ uint32_t part_at(uint32_t smem, int part, int h, int share, int c, int row) {
  return smem + (((part * 2 + h) * share + c) * 128 + row) * 4;
}
// 16 rows of x from row c of the tile on.
__device__ __forceinline__ void give_part(uint32_t smem, int part, int h, int share, int c, int row, const float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 16; j += 4) {  // (a share is a multiple of 4 rows)
    const int to = (c + j) / share;
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(part_at(smem, part, h, share, c + j - to * share, row)), "r"(to));
#pragma unroll
    for (int y = 0; y < 4; ++y) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + y * 512), "f"(v[j + y]) : "memory");
  }
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// --- the kernel ---------------------------------------------------------------------

template <int DT, bool GLU>
__global__ void __launch_bounds__(kManyThreads, 1) linear_many_kernel(const __grid_constant__ ManyArgs A) {
  using P = ManyPlan<DT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const LinArgs& L = A.L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::kBars);
  uint64_t *full = bars, *empty = bars + 8, *a_full = bars + 16, *a_empty = bars + 20, *d_full = bars + 24,
           *d_empty = bars + 26, *last = bars + 28;
  uint32_t* tmem_word = reinterpret_cast<uint32_t*>(smem + P::kMisc);
  volatile int* dead = reinterpret_cast<volatile int*>(smem + P::kMisc + 8);
  int* pre = reinterpret_cast<int*>(smem + P::kPre);
  unsigned* err = L.err;
  if (smem_u32(smem) & 1023) {  // the swizzle counts on it
    if (tid == 0) atomicOr(err, kErrConfig);
    return;
  }
  const int nks = L.in / kLinStep, w_tiles = L.out / kLinTile;
  // this CTA's part of a tile's columns: steps k0 to k0 + mine, steps of sums from j0 on
  uint32_t rank = 0;
  if (A.split > 1) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int k0 = nks * rank / A.split, mine = nks * (rank + 1) / A.split - k0;
  const int j0 = sum_steps(nks) * rank / A.split;
  const int steps = mine + (P::kSums ? sum_steps(nks) * (rank + 1) / A.split - j0 : 0);
  const int item0 = blockIdx.x / A.split, items = gridDim.x / A.split;
  const int m_tiles = (L.out + (GLU ? 127 : 255)) / (GLU ? 128 : 256);
  if (tid == 0) {
    for (int i = 0; i < P::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], (P::kSums ? kConvert : kConvert / 2) + 2);
    for (int i = 0; i < P::kUnits; ++i) mbar_init(&a_full[i], kConvert / 2), mbar_init(&a_empty[i], 2);
    for (int i = 0; i < P::kSets; ++i) mbar_init(&d_full[i], 2), mbar_init(&d_empty[i], kResults);
    mbar_init(last, 2);
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
  const uint32_t tmem = *tmem_word;  // (0: all of tensor memory is this CTA's, which the products' addresses count on)
  const int total = pre[L.n];

  if (warp < kConvert) {
    // ---- conversion: the codes of 16 weight rows of a half, a step at a time ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::kRegConvert));
    const int quarter = warp & 3, half = (warp >> 2) & 1, group = warp >> 3;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + P::kA + half * 32;  // (a stage is 64 columns)
    const int wt0 = half * (GLU ? 0 : 8) + quarter * 2;
    bool ok = true;
    // The products wait for the weights only: who hands them over has seen the step's copies, x among them.
    auto hand_over = [&](uint64_t* weights, uint64_t* step) {
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(weights);
        mbar_arrive(step);
      }
    };
    // (of a tile past the last, the stage holds whatever it held; its lanes' results are not used)
    const int from = P::kCodes + half * kHalfCodes + quarter * 2 * kLinStepBytes;
    if constexpr (!P::kSums) {
      // The group's steps, 64 columns: the next one is converted in registers while the products of the one handed over run.
      const uint32_t to = lanes + group * 64;
      int st = group, first = group;  // first: of the tile's steps, this group's first
      uint32_t ph = 0, a_ph = 1;      // (a fresh barrier passes a wait for the phase before its first)
      uint32_t r0[16], r1[16];
      auto next = [&]() {
        ok = wait_warp(&full[st], ph, dead, err);
        const uint8_t* step = smem + st * P::kStage + from;
        convert(*reinterpret_cast<const uint4*>(step + lane * 16), *reinterpret_cast<const uint4*>(step + 512 + (lane >> 2) * 16), r0);
        step += kLinStepBytes;
        convert(*reinterpret_cast<const uint4*>(step + lane * 16), *reinterpret_cast<const uint4*>(step + 512 + (lane >> 2) * 16), r1);
      };
      for (int item = item0; item < total && ok; item += items) {
        int i = first;
        if (i < mine) next();
#pragma unroll 1
        for (; i < mine && ok; i += 2) {
          if (!(ok = wait_warp(&a_empty[group], a_ph, dead, err))) break;
          tc_fence_after();
          tc_st_16x128_x8(to, r0);
          tc_st_16x128_x8(to + (16u << 16), r1);
          hand_over(&a_full[group], &empty[st]);
          a_ph ^= 1;
          if ((st += 2) >= P::kStages) st = group, ph ^= 1;
          if (i + 2 < mine) next();
        }
        first = i - steps;
      }
    } else {
      // The group's block of every step, 32 columns, in two stages in turn; the next one in registers as above.
      int st = 0, turn = 0;
      uint32_t ph = 0, a_ph = 1;
      uint32_t hi[2][8], lo[2][8];
      auto next = [&]() {
        ok = wait_warp(&full[st], ph, dead, err);
        const uint8_t* step = smem + st * P::kStage + from;
#pragma unroll
        for (int h = 0; h < 2; ++h, step += kLinStepBytes)
          convert_two(*reinterpret_cast<const uint2*>(step + lane * 16 + group * 8),
                      *reinterpret_cast<const uint2*>(step + 512 + (lane >> 2) * 16), group, hi[h], lo[h]);
      };
      auto handed = [&]() {
        hand_over(&a_full[turn * 2 + group], &empty[st]);
        if (turn) a_ph ^= 1;
        turn ^= 1;
        if (++st == P::kStages) st = 0, ph ^= 1;
      };
      for (int item = item0; item < total && ok; item += items) {
        next();
#pragma unroll 1
        for (int i = 0; i < mine && ok; ++i) {
          if (!(ok = wait_warp(&a_empty[turn * 2 + group], a_ph, dead, err))) break;
          tc_fence_after();
          const uint32_t to = lanes + (turn * 2 + group) * 64;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tc_st_16x128_x4(to + ((uint32_t)(16 * h) << 16), hi[h]);
            tc_st_16x128_x4(to + ((uint32_t)(16 * h) << 16) + 16, lo[h]);
          }
          handed();
          if (i + 1 < mine) next();
        }
        const Tile t = tile_at<P::kCols>(L, pre, m_tiles, item);
        const int wt = t.mt * (GLU ? 8 : 16) + wt0;
        int stride;
        const uint8_t* recs = lin_tile(L.w[GLU ? half : 0].packed, t.mat, wt, w_tiles, nks, stride) + 512 + (lane >> 2) * 16;
#pragma unroll 1
        for (int i = mine; i < steps && ok; ++i) {
          const int ks = (j0 + i - mine) * kGroup + group * 4 + (lane & 3);  // this lane's step of the sums' group
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 rec = {};
            if (wt + h < w_tiles && ks < nks)
              rec = __ldg(reinterpret_cast<const uint4*>(recs + (long long)ks * stride + h * kLinStepBytes));
            convert_sums(rec, hi[h]);
          }
          if (!(ok = wait_warp(&full[st], ph, dead, err))) break;
          if (!(ok = wait_warp(&a_empty[turn * 2 + group], a_ph, dead, err))) break;
          tc_fence_after();
          const uint32_t to = lanes + (turn * 2 + group) * 64;
#pragma unroll
          for (int h = 0; h < 2; ++h) tc_st_16x128_x4(to + ((uint32_t)(16 * h) << 16), hi[h]);
          handed();
        }
      }
    }
  } else if (warp < kConvert + kResults) {
    // ---- results: 32 weight rows of each half, half of the tile's rows of x ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::kRegResults));
    griddep_wait();  // the rows' powers of two
    const int quarter = warp & 3, side = (warp - kConvert) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)quarter << 21);
    int chunk = 0;
    bool ok = true;
    for (int item = item0; item < total && ok; item += items) {
      const Tile t = tile_at<P::kCols>(L, pre, m_tiles, item);
      const int f0 = (GLU ? t.mt * 128 : t.mt * 256) + quarter * 32 + lane;
      const int halves = GLU || t.mt * 256 + 128 < L.out ? 2 : 1;
      const int r0 = t.row0 + side * (t.cols >> 1), cols = t.cols >> 1;
      float undo[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f = GLU ? f0 : f0 + h * 128;
        undo[h] = f < L.out ? __ldg(L.w[GLU ? h : 0].undo + (long long)t.mat * L.out + f) * (P::kSums ? kTwoUndo : 1.f) : 0.f;
      }
      if constexpr (P::kSets == 1) {
        if (!(ok = wait_warp(&d_full[0], chunk & 1, dead, err))) break;
        tc_fence_after();
        if (A.split > 1) cluster_meet();  // the cluster's stages of copies are free
        for (int c = 0; c < cols; c += 16) {
          if (A.split > 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h >= halves) break;
              uint32_t r[16];
              tc_ld16(lanes + h * P::kCols + side * cols + c, r);
              tc_wait_ld(r);
              float v[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
              give_part(smem_u32(smem), rank, h, t.cols / A.split, side * cols + c, quarter * 32 + lane, v);
            }
            continue;
          }
          float ux[16];
          load16(A.undo_x + r0 + c, ux);
          float v[2][16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h >= halves) break;
            uint32_t r[16];
            tc_ld16(lanes + h * P::kCols + side * cols + c, r);
            tc_wait_ld(r);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              v[h][j] = __uint_as_float(r[j]), v[h][j + 1] = __uint_as_float(r[j + 1]);
              mul2(v[h][j], v[h][j + 1], undo[h], undo[h]);
              mul2(v[h][j], v[h][j + 1], ux[j], ux[j + 1]);
            }
            if constexpr (!GLU) store16<DT>(L, v[h], r0 + c, t.begin, t.end, f0 + h * 128, lane);
          }
          if constexpr (GLU) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[0][j] = lin_silu<DT != kF32>(v[0][j]) * v[1][j];
            store16<DT>(L, v[0], r0 + c, t.begin, t.end, f0, lane);
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
        for (int i = 0; i < steps; i += kChunk, ++chunk) {
          const int set = chunk & 1;
          if (!(ok = wait_warp(&d_full[set], (chunk >> 1) & 1, dead, err))) break;
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (h < halves && c * 16 < cols) {
                uint32_t r[16];
                tc_ld16(lanes + (set * 2 + h) * P::kCols + side * cols + c * 16, r);
                tc_wait_ld(r);
#pragma unroll
                for (int j = 0; j < 16; j += 2)
                  add2(acc[h][c][j], acc[h][c][j + 1], __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
              }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_empty[set]);
        }
        if (!ok) break;
        if (A.split > 1) cluster_meet();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c * 16 >= cols) break;
          if (A.split > 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (h < halves) give_part(smem_u32(smem), rank, h, t.cols / A.split, side * cols + c * 16, quarter * 32 + lane, acc[h][c]);
            continue;
          }
          float ux[16];
          load16(A.undo_x + r0 + c * 16, ux);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              mul2(acc[h][c][j], acc[h][c][j + 1], undo[h], undo[h]);
              mul2(acc[h][c][j], acc[h][c][j + 1], ux[j], ux[j + 1]);
            }
          if constexpr (GLU) {
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[0][c][j] = lin_silu<DT != kF32>(acc[0][c][j]) * acc[1][c][j];
          }
#pragma unroll
          for (int h = 0; h < (GLU ? 1 : 2); ++h)
            if (h < halves) store16<DT>(L, acc[h][c], r0 + c * 16, t.begin, t.end, f0 + h * 128, lane);
        }
      }
    }
    if (A.split > 1) {
      // this CTA's share of the tile's rows of x, added up in the cluster's order
      if (!ok) cluster_meet();  // (the others count on it)
      cluster_meet();
      const Tile t = tile_at<P::kCols>(L, pre, m_tiles, item0);
      const int f0 = (GLU ? t.mt * 128 : t.mt * 256) + quarter * 32 + lane;
      const int halves = GLU || t.mt * 256 + 128 < L.out ? 2 : 1, share = t.cols / A.split;
      float undo[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f = GLU ? f0 : f0 + h * 128;
        undo[h] = f < L.out ? __ldg(L.w[GLU ? h : 0].undo + (long long)t.mat * L.out + f) * (P::kSums ? kTwoUndo : 1.f) : 0.f;
      }
      // 8 rows of x at a time, whose chains of sums, results and stores overlap (a share is 4, 8 or a multiple of 4 rows)
#pragma unroll 1
      for (int c0 = 0; c0 < share && ok; c0 += 16) {
        const int c = c0 + side * 8, r = t.row0 + (int)rank * share + c, n = min(8, share - c);
        float v[2][8] = {};
        float4 ux[2] = {};
#pragma unroll
        for (int j = 0; j < 8; j += 4)
          if (j < n) ux[j / 4] = load4(A.undo_x + r + j);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= halves) break;
          for (int q = 0; q < A.split; ++q) {
            const float* part = reinterpret_cast<const float*>(smem) + part_at(0, q, h, share, c, quarter * 32 + lane) / 4;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j < n) v[h][j] += part[j * 128];
          }
          const float* u = &ux[0].x;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[h][j] = v[h][j] * undo[h] * u[j];  // (undo u may not be finite)
        }
        if constexpr (GLU) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[0][j] = lin_silu<DT != kF32>(v[0][j]) * v[1][j];
        }
#pragma unroll
        for (int h = 0; h < (GLU ? 1 : 2); ++h) {
          if (h >= halves) break;
#pragma unroll
          for (int j = 0; j < 8; j += 2)
            if (j < n) store2<DT>(L, v[h] + j, r + j, t.begin, t.end, f0 + h * 128, lane);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::kRegIssue));
    if (warp == kLoadWarp && lane == 0) {
      // ---- copies ----
      griddep_wait();  // the rows of x in the workspace
      int copies = 0, st = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int item = item0; item < total && ok; item += items) {
        const Tile t = tile_at<P::kCols>(L, pre, m_tiles, item);
        const uint32_t bytes = (uint32_t)t.cols * 128;
        const uint8_t* x = A.xt + ((long long)k0 * A.pad + t.row0) * 128;
        const uint8_t* sums = A.xt + (((long long)P::kXParts * nks + j0) * A.pad + t.row0) * 128;  // (behind the last part's steps)
        // the tiles of a half that there are (of the second half possibly none)
        const int wt = t.mt * (GLU ? 8 : 16), here0 = min(8, w_tiles - wt), here1 = GLU ? here0 : max(0, min(8, w_tiles - wt - 8));
        int s0, s1;
        const uint8_t* w0 = lin_tile(L.w[0].packed, t.mat, wt, w_tiles, nks, s0);
        const uint8_t* w1 = here1 == 0 ? nullptr : lin_tile(L.w[GLU].packed, t.mat, GLU ? wt : wt + 8, w_tiles, nks, s1);
        const uint32_t codes = (here0 + here1) * kLinStepBytes;
        w0 += (long long)k0 * s0;
        if (here1 > 0) w1 += (long long)k0 * s1;
#pragma unroll 1
        for (int i = 0; i < steps; ++i, ++copies) {
          if (!(ok = wait_for(&empty[st], ph, dead, err))) break;
          uint8_t* to = smem + st * P::kStage;
          if (i < mine) {
            mbar_arrive_expect_tx(&full[st], bytes * P::kXParts + codes);
            bulk_g2s(to + P::kCodes, w0, here0 * kLinStepBytes, &full[st]);
            w0 += s0;
            if (here1 > 0) {
              bulk_g2s(to + P::kCodes + kHalfCodes, w1, here1 * kLinStepBytes, &full[st]);
              w1 += s1;
            }
            bulk_g2s(to, x, bytes, &full[st]);
            if constexpr (P::kXParts == 2) bulk_g2s(to + P::kPart, x + nks * A.pad * 128, bytes, &full[st]);
            x += A.pad * 128;
          } else {
            mbar_arrive_expect_tx(&full[st], bytes);
            bulk_g2s(to, sums, bytes, &full[st]);
            sums += A.pad * 128;
          }
          if (++st == P::kStages) st = 0, ph ^= 1;
        }
      }
      for (int i = max(0, copies - P::kStages); i < copies; ++i)  // the copies have landed before the CTA ends
        mbar_wait(&full[i % P::kStages], (i / P::kStages) & 1, err);
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // ---- products: the warp stays together, so that addresses and descriptors are formed in uniform registers, and one
      // lane's predicate is on the instructions ----
      const uint32_t lead = elect_one();
      const int half = warp - kMmaWarp;
      int st = 0, xst = 0, set = 0;
      uint32_t a_ph = 0, d_ph = 1, seen = 0;  // seen: the next stage of weights is there
      bool ok = true;
      for (int item = item0; item < total && ok; item += items) {
        const Tile t = tile_at<P::kCols>(L, pre, m_tiles, item);
        const bool live = half == 0 || GLU || t.mt * 256 + 128 < L.out;
        const uint32_t id = 1u << 4 | (uint32_t)(t.cols >> 3) << 17 | (uint32_t)(128 >> 4) << 24;  // f16, f32, M = 128
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
          const bool first = P::kSets == 2 ? i % kChunk == 0 : i == 0;
          if (first && !(ok = wait_warp(&d_empty[set], d_ph, dead, err))) break;
          const uint64_t b = tc_desc(smem + xst * P::kStage, 1024, 0);
          const uint32_t d = (set * 2 + half) * P::kCols;
          constexpr int kParts = P::kUnits / 2;  // stages of weights to a step
          const bool two = P::kSums && i < mine;
#pragma unroll
          for (int u = 0; u < kParts; ++u) {
            const int at = st * kParts + u;
            if (!__all_sync(0xFFFFFFFFu, seen) && !(ok = wait_warp(&a_full[at], a_ph, dead, err))) break;
            tc_fence_after();
            const uint32_t a = P::kA + at * 64 + half * 32;
            // The next stage's barrier is looked at beside the last products: the tensor cores queue some four of them, less time
            // than a wait takes (f32 rows of 4096 -> 2048 112 -> 108 us, bf16 and f16 rows as before).
            uint64_t* next = &a_full[u + 1 < kParts ? at + 1 : (st ^ 1) * kParts];
            const uint32_t next_ph = u + 1 < kParts || st == 0 ? a_ph : a_ph ^ 1;
            if (!live) {
              seen = 0;
            } else if constexpr (P::kSums) {
              // the small parts first: an add truncates by the accumulator's size
              if (two) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint64_t by = b + (u * 2 + y) * 2;
                  tc_mma_ts_if(lead, d, a + 16 + y * 8, by, id, !first || u > 0 || y > 0);
                  if constexpr (P::kXParts == 2) tc_mma_ts_if(lead, d, a + y * 8, by + (P::kPart >> 4), id, 1);
                }
              }
              seen = tc_mma_pair_look(lead, d, a, b + u * 4, id, two || !first || u > 0, next, next_ph);
            } else {
              tc_mma_ts_if(lead, d, a, b, id, !first);
              tc_mma_ts_if(lead, d, a + 8, b + 2, id, 1);
              seen = tc_mma_pair_look(lead, d, a + 16, b + 4, id, 1, next, next_ph);
            }
            tc_commit_if(lead, &a_empty[at]);
          }
          if (!ok) break;
          tc_commit_if(lead, &empty[xst]);
          if (st) a_ph ^= 1;
          st ^= 1;
          if (++xst == P::kStages) xst = 0;
          if (i == steps - 1 || (P::kSets == 2 && i % kChunk == kChunk - 1)) {
            tc_commit_if(lead, &d_full[set]);
            if (++set == P::kSets) set = 0, d_ph ^= 1;
          }
        }
      }
      tc_commit_if(lead, last);
      __syncwarp();
      mbar_wait(last, 0, err);
    }
    __syncwarp();
  }
  if (A.split > 1 && (warp < kConvert || warp >= kConvert + kResults)) {
    cluster_meet();
    cluster_meet();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int DT>
int smem_bytes(int n) { return ManyPlan<DT>::kPre + (n + 1) * 4; }

// CTAs to a tile: as many as leave every tile a cluster of its own at once and every CTA two steps.
int split_of(int tiles, int nks, const int (&clusters)[3]) {
  for (int i = 2; i >= 0; --i)
    if (tiles <= clusters[i] && nks >= 4 << i) return 2 << i;
  return 1;
}

template <int DT>
cudaError_t launch(ManyArgs A, int nsm, const int (&clusters)[3], cudaStream_t s) {
  const LinArgs& L = A.L;
  int tiles = nsm;
  A.split = 1;
  if (!L.offsets) {  // (with offsets the number of tiles is the device's)
    const long long all = ((long long)L.out + (L.glu ? 127 : 255)) / (L.glu ? 128 : 256) * ((L.T + ManyPlan<DT>::kCols - 1) / ManyPlan<DT>::kCols);
    if (all < nsm) tiles = (int)all, A.split = split_of(tiles, L.in / kLinStep, clusters);
  }
  // warps per row: as many as keep it in registers, at most a CTA's
  int warps = 1;
  constexpr int kRows = DT == kF16Long ? kF16 : DT;
  while (warps < 8 && L.in / 8 > warps * 32 * RowsPlan<kRows>::kOct) warps *= 2;
  const int per = 8 / warps;
  linear_rows_kernel<kRows><<<(unsigned)((L.T + per - 1) / per), 256, 0, s>>>(L.x, L.xs, L.T, L.in, warps, const_cast<uint8_t*>(A.xt),
                                                                             A.pad, const_cast<float*>(A.undo_x));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // launched while the rows are prepared: its start (barriers, tensor memory, the list of tiles, the first codes) needs none
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(nsm), cfg.blockDim = dim3(kManyThreads), cfg.dynamicSmemBytes = smem_bytes<DT>(L.n), cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = A.split, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = A.split > 1 ? 2 : 1;
  if (A.split > 1) cfg.gridDim = dim3(tiles * A.split);
  return L.glu ? cudaLaunchKernelEx(&cfg, linear_many_kernel<DT, true>, A) : cudaLaunchKernelEx(&cfg, linear_many_kernel<DT, false>, A);
}

template <int DT, bool GLU>
cudaError_t setup() {
  auto* fn = linear_many_kernel<DT, GLU>;
  cudaFuncAttributes a;
  const cudaError_t e = cudaFuncGetAttributes(&a, fn);
  if (e != cudaSuccess) return e;
  // the roles' register shares are drawn from what the block is launched with
  if ((a.numRegs + 7) / 8 * 8 < kRegs) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<DT>(kMaxMats));
}

// Bytes of the workspace per row: two parts of f32 rows, the sums, the power of two.
long long row_bytes(int in) { return (2LL * (in / 64) + sum_steps(in / 64)) * 128 + 4; }

// Rows of the workspace: a tile's copies may pass a matrix's last row by less than a tile.
long long pad_rows(int max_rows) { return (((long long)max_rows + 7) & ~7LL) + 192; }

}  // namespace

long long linear_many_workspace(int in, int max_rows) { return pad_rows(max_rows) * row_bytes(in); }

// clusters: how many clusters of 2, 4 and 8 CTAs run at once.
cudaError_t setup_linear_many(int (&clusters)[3]) {
  const cudaError_t e[10] = {setup<kF32, false>(),   setup<kF32, true>(),   setup<kF16, false>(),    setup<kF16, true>(),
                             setup<kBF16, false>(),  setup<kBF16, true>(),  setup<kBF16X, false>(),  setup<kBF16X, true>(),
                             setup<kF16Long, false>(), setup<kF16Long, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  for (int i = 0; i < 3; ++i) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(64 << i), cfg.blockDim = dim3(kManyThreads), cfg.dynamicSmemBytes = smem_bytes<kF16>(kMaxMats);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2 << i, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at, cfg.numAttrs = 1;
    const cudaError_t x = cudaOccupancyMaxActiveClusters(&clusters[i], linear_many_kernel<kF16, false>, &cfg);
    if (x != cudaSuccess) return x;
  }
  return cudaSuccess;
}

cudaError_t launch_linear_many(const LinArgs& L, void* workspace, int max_rows, int nsm, const int (&clusters)[3], cudaStream_t s) {
  ManyArgs A;
  A.L = L;
  A.pad = pad_rows(max_rows);
  A.xt = static_cast<uint8_t*>(workspace);
  A.undo_x = reinterpret_cast<const float*>(A.xt + A.pad * (row_bytes(L.in) - 4));
  if (L.dtype == kF32) return launch<kF32>(A, nsm, clusters, s);
  // An accumulator's adds truncate, some 9 of them a step of 64 columns, by 2^-23 of it at most: while that is below half a step
  // of an f16 result the sum stays in it.  (65536 columns of one sign in one accumulator drifted by 2.3e-4, half of that half step;
  // the registers' sums cost 1280 rows of 32768 -> 4096 1163 us against 735 us.)
  if (L.dtype == kF16) return 9 * (L.in / kLinStep) > 1 << 12 ? launch<kF16Long>(A, nsm, clusters, s) : launch<kF16>(A, nsm, clusters, s);
  return L.rounded ? launch<kBF16>(A, nsm, clusters, s) : launch<kBF16X>(A, nsm, clusters, s);
}

}  // namespace strata
