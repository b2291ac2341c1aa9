// Attention of many rows per slot (prompts and chunks of them) over the 8-bit
// caches, on the 5th-generation tensor cores.
//
// An item is 128 rows (whole tokens x the query heads that share a kv head) of
// one sequence against the positions its last row sees, in units of 128
// positions.  As in kv8_attend.cu all items' units form one list that the CTAs
// (one per SM) share equally, and cut items are joined in CTA order.
//
// Per unit: S = Q K^T (128 x 128) and U = P V (128 x head_dim), both
// tcgen05.mma of f16 operands with f32 accumulators in tensor memory.  Codes
// are exact in f16, so the caches' format costs one conversion per unit; q is
// brought to f16 by a power of two per row, as one part (f16 and bf16 rows) or
// two (f32 rows: hi and lo chain into one accumulator, in S and in U alike).
//
// A unit has its own softmax maximum (over t = s + ev, see kv8_attend.cu); its
// U is scaled into the rows' f32 output registers by the correction warps.  So
// the two softmax warpgroups take units in turn without waiting for each other,
// and no accumulator lives longer than one unit: the tensor core's truncating
// adds do not pile up over a long cache.
//
// q and the weights are rounded to f16 parts as in kv8_attend.cu; f32 rows end
// 8e-7 from 64 bits (rms, prompts and chunks), products in fp32 1.5e-6.
//
// Measured (32 / 8 heads of 128): 8191 bf16 rows from the first token 635 us
// (866 TFLOP/s, 45% of the measured cuBLAS rate); 1531 + 1152 f32 rows at 9001
// and 6776 positions 493 us (two products for each: 69% of that rate).  Bound by
// the roles' per-unit work and hand-overs, not by the tensor cores (27% active
// at 4095 rows).
// Every variant spills at the launch's 80 registers (148 to 232 bytes stored).
//
// Roles (24 warps): two warpgroups of softmax (even and odd units, a row a
// thread), one of correction (a row's output a thread), one of conversion for q
// and K and one for V, and a warp each for the products S, the products U, TMA
// of K (which also makes the list of the CTA's segments) and TMA of V.
// A role sees what another wrote through the chain of barriers between them;
// what a reader does not free by a barrier of its own has slots enough that the
// chain keeps them apart.  S(u) is issued once U(u - 3) is done, so when S(u)
// can be read the softmax of u - 3 is done, and the correction of u - 4 (U has
// one place): 4 slots of statistics, written for u and read for u - 4; 4 of the
// rows' powers of two, written for an item once S of the unit before it is
// done; 8 of the units' factors, written once S(u - 2) is done, that is, after
// the softmax of u - 5.
//   TMA -> raw codes -> conversion -> f16 K, V -> MMA -> S -> softmax -> P (in
//   S's place) -> MMA -> U -> correction
#include "kv8.cuh"

namespace strata {
namespace {

constexpr int kPUnit = 128;      // positions per unit
constexpr int kPRows = 128;      // rows per tile
constexpr int kPThreads = 768;
constexpr int kRegs = 80;        // registers per thread at launch; the roles' shares below sum to 6 x 80
constexpr int kSegs = 8;         // slots of the segment list
constexpr int kMmaWarp = 20, kTmaWarp = 22;  // products: 20 S, 21 U; TMA: 22 K, 23 V
constexpr float kPWeightTop = 14.f;
constexpr float kLeastFactor = 0x1p-100f;
constexpr float kFar = 4096.f;   // rows whose weights need a larger constant than this take unit_shift
constexpr int kRawStages = 3;      // of half a unit's codes, for K and for V
// Barriers of a stage for each half, so that a warp, which takes only its half's copies, waits for every phase of the
// barriers that it reads (one barrier for both would let it take the other half's earlier phase for its own).
constexpr int kRawBars = 2 * kRawStages;
constexpr int kScores = 3;         // places of S (and then P) in tensor memory

template <int HD, bool TWO> struct PromptPlan {
  static constexpr int kTile = kPRows * HD * 2;      // a 128-row f16 tile: panels of 64 halves (one swizzle span)
  static constexpr int kRaw = 64 * HD;               // half a unit's codes of K or V
  static constexpr int kVStages = TWO ? 1 : 2;      // tiles of V: of the one, each half is converted while the other is in use
  static constexpr int kVParts = TWO ? 2 : 1;       // what V's barriers cover: halves, or whole tiles
  static constexpr int kQ = 0;                       // byte offsets from a 1024-byte boundary
  static constexpr int kK = kQ + (TWO ? 2 : 1) * kTile;
  static constexpr int kV = kK + 2 * kTile;
  static constexpr int kRawOff = kV + kVStages * kTile;
  static constexpr int kStats = kRawOff + 2 * kRawStages * kRaw;  // [4][128] float2: a unit's maxima and sums
  static constexpr int kRf = kStats + 4 * kPRows * 8;         // [4][128] the rows' powers of two, by item
  static constexpr int kExp = kRf + 4 * kPRows * 4;           // [8][8] float4: a unit's factors per 16 positions
  static constexpr int kBars = kExp + 8 * 8 * 16;
  static constexpr int kMisc = kBars + 1024;                  // tensor memory address, flags, scan sums
  static constexpr int kSegOff = kMisc + 256;                 // [kSegs] Seg
  static constexpr int kPre = kSegOff + 64 * kSegs;
  // registers per thread by role (softmax keeps the launch's)
  static constexpr int kRegCorrect = 176, kRegConvert = 56, kRegIssue = 32;
  static_assert(2 * kRegs + kRegCorrect + 2 * kRegConvert + kRegIssue <= 6 * kRegs, "register split");
};

// What a CTA does of one item: units u0 to u1 of `units`.  Written once by the
// list's warp, read by every role; a slot is free again when all have passed it.
struct alignas(64) Seg {
  int row0, n, length, slot;   // the sequence
  int head, tile;
  int u0, u1, units;
  int end;                     // the CTA's units up to this segment's end
  long long first;             // the item's first unit in the whole list
};
constexpr int kSegReaders = 8 + 4 + 8 + 1 + 2;  // warps (softmax, correction, conversion, S, TMA)

struct PromptArgs {
  Kv8Dev C;
  Kv8Rows R;
  const void* q;
  void* out;
  long long q_stride, out_stride;
  float scale2;      // |scale| * log2(e)
  float sign;        // of scale
  int dtype, group, layer, tokens;  // tokens per tile: 128 / group
  float* parts;      // [2 grid][(HD + 2) * 128]
  unsigned* count;   // [grid]
};

// --- tcgen05 -----------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// D (+)= A B^T, A and B in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Waits for this thread's tensor memory loads.  The registers they fill are operands, so that no use of them can be
// moved in front of it.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor: 128-byte swizzle, 8-row groups `sbo` bytes
// apart, 64-wide panels `lbo` bytes apart (read for MN-major operands only).
__device__ __forceinline__ uint64_t tc_desc(const void* p, uint32_t sbo, uint32_t lbo) {
  return (uint64_t)((smem_u32(p) >> 4) & 0x3FFF) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFF) << 32 | 1ull << 46 | 2ull << 61;
}
// f16 x f16 -> f32, M = 128.
constexpr uint32_t tc_idesc(int n, bool b_mn_major) {
  return 1u << 4 | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(kPRows >> 4) << 24;
}

// Bounded wait: gives up when it or another role has waited about a second.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* dead, unsigned* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*dead) return false;
    if (clock64() - t0 > (1LL << 31)) {
      *dead = 1;
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
}

// The same for a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* dead, unsigned* err) {
  return __all_sync(0xFFFFFFFFu, wait_for(bar, parity, dead, err));
}

// Barrier of the 128 correction threads: whether all of them say yes.
__device__ __forceinline__ bool all_of_128(bool yes) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.and.pred q, 1, 128, p;\nselp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)yes)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void p_tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float p_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A lane's E neighbouring values of a row of q, as they are in memory (TWO: f32, else f16 or bf16).
template <int E, bool TWO> struct alignas(TWO ? 4 * E : 2 * E) Raw {
  uint32_t w[TWO ? E : E / 2];
  __device__ __forceinline__ void get(float* f, int dtype) const {
    if constexpr (TWO) {
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        if (dtype == 1) {
          const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          f[2 * i] = t.x, f[2 * i + 1] = t.y;
        } else {
          f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      }
    }
  }
};
__device__ __forceinline__ uint32_t pack_out(bool bf16, float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  const __half2 y = __floats2half2_rn(a, b);
  return bf16 ? *reinterpret_cast<const uint32_t*>(&x) : *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void p_store4(void* p, int dtype, long long i, float4 v) {
  if (dtype == 0) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
  } else if (dtype == 1) {
    __half2 h[2] = {__floats2half2_rn(v.x, v.y), __floats2half2_rn(v.z, v.w)};
    *reinterpret_cast<uint2*>(static_cast<__half*>(p) + i) = *reinterpret_cast<uint2*>(h);
  } else {
    __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) = *reinterpret_cast<uint2*>(h);
  }
}

// --- the list of units ----------------------------------------------------------

// sum of floor((a i + b) / m) over i = 0..n-1 (Euclid's steps); a n + b stays below 2^32: a and m are at most 128,
// n at most 2^24 row tiles and b about a cache's length.
__device__ inline long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long sum = 0;
  while (n > 0) {
    sum += (long long)(n - 1) * n / 2 * (a / m) + (long long)n * (b / m);
    a %= m, b %= m;
    const unsigned y = a * n + b;
    if (y < m) break;
    n = y / m, b = y % m;
    const unsigned t = m;
    m = a, a = t;
  }
  return sum;
}

// Row tiles of a sequence, and units of its first `tiles` ones (one kv head).
// Tile t's last row sees base + min(n, tokens (t + 1)) positions, base = length - n.
__device__ __forceinline__ int p_tiles(const Kv8Seq& s, int tokens) { return (s.n + tokens - 1) / tokens; }
__device__ __forceinline__ int p_units(const Kv8Seq& s, int tokens, int t) {
  const int seen = s.length - s.n + min(s.n, tokens * (t + 1));
  return seen <= 0 ? 0 : (seen + kPUnit - 1) / kPUnit;
}
__device__ inline long long p_units_before(const Kv8Seq& s, int tokens, int tiles) {
  if (tiles <= 0) return 0;
  long long sum = 0;
  if (tiles * (long long)tokens > s.n) sum = p_units(s, tokens, --tiles);  // the last tile may be short
  // tiles 0..tiles-1 see base + tokens (t + 1): skip those that see nothing
  const int base = s.length - s.n;
  int t0 = 0;
  if (base + tokens <= 0) t0 = min(tiles, -base / tokens);
  if (tiles > t0) sum += floor_sum(tiles - t0, kPUnit, tokens, base + tokens * (t0 + 1) + kPUnit - 1);
  return sum;
}
__device__ __forceinline__ long long p_head_units(const Kv8Seq& s, int tokens) {
  return s.held_ok && s.n > 0 ? p_units_before(s, tokens, p_tiles(s, tokens)) : 0;
}

// A sequence's row tiles are taken from both ends inwards (first, last, second,
// ...): a tile's units grow with its position, and so every stretch of the list
// has about the same number of items, whose starts cost a CTA time too.
__device__ __forceinline__ int p_tile_at(const Kv8Seq& s, int tokens, int i) {
  return i & 1 ? p_tiles(s, tokens) - 1 - (i >> 1) : i >> 1;
}
// Units of the first k tiles in that order.
__device__ inline long long p_ordered_before(const Kv8Seq& s, int tokens, int k) {
  const int tiles = p_tiles(s, tokens);
  return p_units_before(s, tokens, (k + 1) >> 1) + p_units_before(s, tokens, tiles) -
         p_units_before(s, tokens, tiles - (k >> 1));
}

// The items of a CTA's part of the list in turn; begin() finds the first (a whole warp does, 32 places tried at a time:
// one thread by halves took some 16 us), next() steps.
struct PItem {
  Kv8Seq s;
  int seq, head, i, tile, units;  // i: the tile's place in the order
  int u0, u1;
  long long first;
};

__device__ inline void p_begin(PItem& it, const PromptArgs& A, const long long* pre, long long lo, long long hi) {
  int a = 0, b = A.R.n_seq;
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (pre[m] <= lo)
      a = m;
    else
      b = m;
  }
  it.seq = a;
  it.s = kv8_seq(A.R, A.C, a);
  long long r = lo - pre[a];
  const long long per = p_head_units(it.s, A.tokens);
  it.head = (int)(r / per);
  r -= it.head * per;
  int t0 = 0, t1 = p_tiles(it.s, A.tokens);  // before(t0) <= r < before(t1)
  while (t1 - t0 > 1) {
    const int step = (t1 - t0 + 31) / 32, at = t0 + ((int)(threadIdx.x & 31) + 1) * step;
    const bool below = at < t1 && p_ordered_before(it.s, A.tokens, at) <= r;
    t0 += __popc(__ballot_sync(0xFFFFFFFFu, below)) * step;
    t1 = min(t1, t0 + step);
  }
  it.i = t0;
  it.tile = p_tile_at(it.s, A.tokens, t0);
  it.units = p_units(it.s, A.tokens, it.tile);
  it.u0 = (int)(r - p_ordered_before(it.s, A.tokens, t0));
  it.u1 = (int)min((long long)it.units, it.u0 + (hi - lo));
  it.first = lo - it.u0;
}

// After a part that ended at unit u of the list (u < hi).
__device__ inline void p_next(PItem& it, const PromptArgs& A, const long long* pre, long long u, long long hi) {
  do {
    if (++it.i >= p_tiles(it.s, A.tokens)) {
      it.i = 0;
      if (++it.head >= A.C.kv_heads) {
        it.head = 0;
        do {
          ++it.seq;
        } while (pre[it.seq + 1] <= u);
        it.s = kv8_seq(A.R, A.C, it.seq);
      }
    }
    it.tile = p_tile_at(it.s, A.tokens, it.i);
    it.units = p_units(it.s, A.tokens, it.tile);
  } while (it.units == 0);
  it.u0 = 0;
  it.u1 = (int)min((long long)it.units, hi - u);
  it.first = u;
}

// A stage of a ring of N and the parity of its current round.
template <int N> struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step() {
    if (++st == N) st = 0, ph ^= 1;
  }
};

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The scores of positions that the row does not see become -inf.
__device__ __forceinline__ void unit_mask(uint32_t s_addr, int left) {
#pragma unroll 1
  for (int ch = 0; ch < 8; ++ch) {
    uint32_t r[16];
    tc_ld16(s_addr + ch * 16, r);
    tc_wait_ld(r);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (ch * 16 + i >= left) r[i] = 0xFF800000u;
    tc_st16(s_addr + ch * 16, r);
  }
  tc_wait_st();
}

// The scores of a row whose maximum is far from zero become (t - m - ev) / kLeastFactor, which unit_softmax turns into
// t - m when it goes on with a factor and a maximum of zero.  For the other rows it adds ev, kPWeightTop and -m in one
// rounded constant, whose half step grows with m: from m = 2^25 on it would lift a weight past f16's range, and units
// would disagree on what their weights are relative to.  Not inlined: no trained model's scores come here, and in the
// hot code it cost 2 % of a prompt (as it is: 634 us against 626 for 8191 rows).
__device__ __noinline__ void unit_shift(uint32_t s_addr, const float4* fac, float f_row, bool far, float m) {
#pragma unroll 1
  for (int ch = 0; ch < 8; ++ch) {
    uint32_t r[16];
    tc_ld16(s_addr + ch * 16, r);
    const float4 f = fac[ch];
    const float k = fmaxf(f.x * f_row, kLeastFactor);
    tc_wait_ld(r);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (far) r[i] = __float_as_uint((fmaf(__uint_as_float(r[i]), k, f.y) - m - f.y) * (1.f / kLeastFactor));
    tc_st16(s_addr + ch * 16, r);
  }
  tc_wait_st();
}

// A row's softmax over one unit: the 128 scores at s_addr become weights (16-bit
// parts) relative to the unit's maximum m; l is their sum over 2^ev.  The
// chunks are a rolled loop, and there is one copy of it: the hot code of all
// roles together has to stay within the SM's instruction cache (unrolled,
// instruction fetch was the largest stall and a unit took 9400 cycles).
template <bool TWO>
__device__ __forceinline__ void unit_softmax(uint32_t s_addr, const float4* fac, float f_row, float& m, float& l) {
  m = -INFINITY;
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    uint32_t r[32];
    tc_ld32(s_addr + ch * 32, r);
    const float4 f0 = fac[ch * 2], f1 = fac[ch * 2 + 1];
    tc_wait_ld(r);
    float a0 = -INFINITY, a1 = -INFINITY, b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      a0 = max3(a0, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
      a1 = max3(a1, __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
      b0 = max3(b0, __uint_as_float(r[i + 16]), __uint_as_float(r[i + 17]));
      b1 = max3(b1, __uint_as_float(r[i + 18]), __uint_as_float(r[i + 19]));
    }
    // (a factor of zero would turn -inf into NaN)
    m = max3(m, fmaf(fmaxf(a0, a1), fmaxf(f0.x * f_row, kLeastFactor), f0.y),
             fmaf(fmaxf(b0, b1), fmaxf(f1.x * f_row, kLeastFactor), f1.y));
  }
  float z = m == -INFINITY ? 0.f : kPWeightTop - m;
  const bool far = fabsf(z) >= kFar;
  if (__builtin_expect(__any_sync(0xFFFFFFFFu, far), 0)) {
    unit_shift(s_addr, fac, f_row, far, m);
    if (far) f_row = 0.f, z = kPWeightTop;
  }
  l = 0.f;
#pragma unroll 1
  for (int ch = 0; ch < 8; ++ch) {
    uint32_t r[16];
    tc_ld16(s_addr + ch * 16, r);
    const float4 f = fac[ch];
    const float k = fmaxf(f.x * f_row, kLeastFactor), c = f.y + z;
    const uint64_t k2 = pack2(k, k), c2 = pack2(c, c);
    uint64_t sum = pack2(0.f, 0.f);
    uint32_t hi16[8], lo16[TWO ? 8 : 1];
    tc_wait_ld(r);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      float w0, w1;
      unpack2(fma2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), k2, c2), w0, w1);
      w0 = p_ex2(w0), w1 = p_ex2(w1);
      sum = add2(sum, pack2(w0, w1));
      const __half2 hh = __floats2half2_rn(w0, w1);
      hi16[i / 2] = *reinterpret_cast<const uint32_t*>(&hh);
      if constexpr (TWO) {
        const float2 back = __half22float2(hh);
        lo16[i / 2] = pack_half2(w0 - back.x, w1 - back.y);
      }
    }
    float s0, s1;
    unpack2(sum, s0, s1);
    l = fmaf(s0 + s1, f.z, l);
    // P takes the place of the 16 scores it came from: 8 columns of first parts, 8 of second ones
    tc_st8(s_addr + ch * 16, hi16);
    if constexpr (TWO) tc_st8(s_addr + ch * 16 + 8, lo16);
  }
}

template <int HD, int FMT, bool TWO>
__global__ void __launch_bounds__(kPThreads, 1)
    attend_prompt_kernel(const __grid_constant__ PromptArgs A, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  using P = PromptPlan<HD, TWO>;
  // declared aligned, so that every role's addresses are constants and not registers
  extern __shared__ __align__(1024) uint8_t smem[];
  float2* stats = reinterpret_cast<float2*>(smem + P::kStats);
  float* rf = reinterpret_cast<float*>(smem + P::kRf);
  float4* factors = reinterpret_cast<float4*>(smem + P::kExp);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::kBars);
  uint64_t *v_full = bars, *v_empty = bars + 4, *k_full = bars + 8, *k_empty = bars + 10, *q_full = bars + 12,
           *q_empty = bars + 13, *s_full = bars + 16, *p_full = bars + 19, *u_full = bars + 22, *u_empty = bars + 23,
           *last = bars + 24, *place_free = bars + 26, *seg_full = bars + 32, *seg_empty = bars + 40,
           *raw_full = bars + 48, *raw_empty = bars + 48 + 2 * kRawBars;
  const Seg* segs = reinterpret_cast<const Seg*>(smem + P::kSegOff);
  uint32_t* tmem_word = reinterpret_cast<uint32_t*>(smem + P::kMisc);
  volatile int* dead = reinterpret_cast<volatile int*>(smem + P::kMisc + 8);
  int* flag = reinterpret_cast<int*>(smem + P::kMisc + 12);
  long long* warp_sums = reinterpret_cast<long long*>(smem + P::kMisc + 16);
  long long* span = reinterpret_cast<long long*>(smem + P::kMisc + 192);  // all units; this CTA's first, and end
  long long* pre = reinterpret_cast<long long*>(smem + P::kPre);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned* err = A.C.err;

  if (smem_u32(smem) & 1023) {  // the swizzles count on it
    if (tid == 0) atomicOr(err, kErrConfig);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2 * kRawBars; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_empty[i], 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4), mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&v_full[i], TWO ? 2 : 4), mbar_init(&v_empty[i], 1);
    for (int i = 0; i < kScores; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 4), mbar_init(&place_free[i], 1);
    mbar_init(u_full, 1), mbar_init(u_empty, 4);
    mbar_init(q_full, 4), mbar_init(q_empty, 1), mbar_init(&last[0], 1), mbar_init(&last[1], 1);
    for (int i = 0; i < kSegs; ++i) mbar_init(&seg_full[i], 1), mbar_init(&seg_empty[i], kSegReaders);
    *dead = 0;
    fence_mbar_init();
  }
  // units before each sequence
  const int n_seq = A.R.n_seq;
  {
    constexpr int kScan = 512;
    const int share = (n_seq + kScan - 1) / kScan;
    long long sum = 0;
    if (tid < kScan) {
      for (int i = tid * share; i < min(n_seq, (tid + 1) * share); ++i) {
        const Kv8Seq s = kv8_seq(A.R, A.C, i);
        sum += p_head_units(s, A.tokens) * A.C.kv_heads;
        pre[i + 1] = sum;
        if (!s.held_ok && blockIdx.x == 0) atomicOr(err, kErrIndex);
      }
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31 && warp < kScan / 32) warp_sums[warp] = inc;
    __syncthreads();
    if (tid < kScan) {
      long long before = inc - sum;
      for (int w = 0; w < warp; ++w) before += warp_sums[w];
      for (int i = tid * share; i < min(n_seq, (tid + 1) * share); ++i) pre[i + 1] += before;
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
  }
  // rows that see nothing (or whose slot or length is out of range) are zero
  for (int i = blockIdx.x; i < n_seq; i += gridDim.x) {
    const Kv8Seq s = kv8_seq(A.R, A.C, i);
    if (!s.rows_ok) continue;
    const int blind = s.held_ok ? min(s.n, max(0, s.n - s.length)) : s.n;
    const int w4 = A.C.heads * HD / 4;
    for (long long j = tid; j < (long long)blind * w4; j += kPThreads)
      p_store4(A.out, A.dtype, (s.row0 + j / w4) * A.out_stride + j % w4 * 4, make_float4(0, 0, 0, 0));
  }
  int n_units;
  {
    const long long total = pre[n_seq], G = min((long long)gridDim.x, total);
    if (blockIdx.x >= G) return;
    const long long lo = total * blockIdx.x / G, hi = total * (blockIdx.x + 1) / G;
    n_units = (int)(hi - lo);
    if (tid == 0) span[0] = total, span[1] = lo, span[2] = hi;  // for the roles that need them, now and then
  }

  if (warp == kMmaWarp) {  // all of tensor memory: S in three places (128 columns each), U
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_word)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;

  if (warp < 8) {
    // ---- softmax: warpgroup `odd` takes units odd, odd + 2, ...; a row a thread ----
    const int odd = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
    Ring<kScores> place;
    if (odd) place.step();
    const int row_tok = row < A.tokens * A.group ? row / A.group : 1 << 28;
    Ring<kSegs> seg;
    bool ok = true;
    int n = 0;
    for (int item = 0; n < n_units; ++item) {
      if (!(ok = wait_warp(&seg_full[seg.st], seg.ph, dead, err))) break;
      const Seg* it = segs + seg.st;
      const int tok = it->tile * A.tokens + row_tok, base = it->length - it->n, u0 = it->u0, u1 = it->u1;
      const int lim = tok < it->n ? max(0, base + tok + 1) : 0;  // positions the row sees
      const int all = max(0, base + it->tile * A.tokens + 1);    // positions every row of the tile sees
      float f_row = 1.f;
      bool have = false;
      for (int x = u0 + ((n ^ odd) & 1); x < u1; x += 2) {
        const int at = n + x - u0;
        if (!(ok = wait_warp(&s_full[place.st], place.ph, dead, err))) break;
        tc_fence_after();
        if (!have) f_row = kv8_row_factor(A.scale2, rf[(item & 3) * kPRows + row]), have = true;
        const float4* fac = factors + (at & 7) * 8;  // per 16 positions: 2^ek, ev, 2^-ev
        const int left = lim - x * kPUnit;  // positions of the unit that the row sees
        const bool masked = (x + 1) * kPUnit > all;
        float m, l;
        if (masked) unit_mask(lanes + place.st * 128, left);
        unit_softmax<TWO>(lanes + place.st * 128, fac, f_row, m, l);
        stats[(at & 3) * kPRows + row] = make_float2(m, l);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[place.st]);
        place.step(), place.step();
      }
      if (!ok) break;
      n += u1 - u0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[seg.st]);
      seg.step();
    }
  } else if (warp < 12) {
    // ---- correction: a row's output in registers ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::kRegCorrect));
    const int row = tid & 127;
    const uint32_t u_addr = tmem + kScores * 128 + ((uint32_t)(warp & 3) << 21);
    const int row_tok = row < A.tokens * A.group ? row / A.group : 1 << 28, row_head = row % A.group;
    Ring<kSegs> seg;
    bool ok = true;
    int n = 0;
    while (n < n_units) {
      // all four warps go on or stop together: the barriers below count them all
      if (!all_of_128(wait_warp(&seg_full[seg.st], seg.ph, dead, err))) break;
      const Seg* it = segs + seg.st;
      float o[HD];
#pragma unroll
      for (int i = 0; i < HD; ++i) o[i] = 0.f;
      float m = -INFINITY, l = 0.f;
      for (int x = it->u0; x < it->u1; ++x) {
        const int at = n + x - it->u0;
        if (ok) ok = wait_warp(u_full, at & 1, dead, err);
        if (!ok) break;
        tc_fence_after();
        const float2 st = stats[(at & 3) * kPRows + row];
        const float mn = fmaxf(m, st.x);
        // a NaN row has no maximum but a NaN sum: it stays NaN
        const float a = m == mn ? 1.f : p_ex2(m - mn), b = st.x == -INFINITY && st.y == 0.f ? 0.f : p_ex2(st.x - mn);
        m = mn;
        l = fmaf(st.y, b, l * a);
        const bool grew = __any_sync(0xFFFFFFFFu, a != 1.f);
#pragma unroll
        for (int ch = 0; ch < HD / 32; ++ch) {
          uint32_t r[32];
          tc_ld32(u_addr + ch * 32, r);
          if (grew) {
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              unpack2(mul2(pack2(o[ch * 32 + i], o[ch * 32 + i + 1]), pack2(a, a)), o[ch * 32 + i], o[ch * 32 + i + 1]);
          }
          tc_wait_ld(r);
          if (ch == HD / 32 - 1) {  // the last of U is in registers: its place is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(u_empty);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            unpack2(fma2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), pack2(b, b),
                         pack2(o[ch * 32 + i], o[ch * 32 + i + 1])),
                    o[ch * 32 + i], o[ch * 32 + i + 1]);
        }
      }
      n += it->u1 - it->u0;
      const int tok = it->tile * A.tokens + row_tok;
      const bool on = tok < it->n;
      const long long to = (long long)(it->row0 + tok) * A.out_stride + (long long)(it->head * A.group + row_head) * HD;
      bool write = on && ok;
      if (it->u0 != 0 || it->u1 != it->units) {
        constexpr int kPart = (HD + 2) * kPRows;
        const long long total = span[0], lo = span[1], G = min((long long)gridDim.x, total);
        float* part = A.parts + (long long)(2 * blockIdx.x + (it->first + it->u0 == lo ? 0 : 1)) * kPart + row;
#pragma unroll
        for (int i = 0; i < HD; ++i) part[i * kPRows] = o[i];
        part[HD * kPRows] = m, part[(HD + 1) * kPRows] = l;
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int c0 = (int)(((it->first + 1) * G - 1) / total), c1 = (int)(((it->first + it->units) * G - 1) / total);
        if (row == 0) {
          __threadfence();
          *flag = atomicInc(&A.count[c0], (unsigned)(c1 - c0)) == (unsigned)(c1 - c0);
          __threadfence();
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        write = write && *flag;
        if (write) {
          const int s0 = 2 * c0 + (total * c0 / G == it->first ? 0 : 1);
          m = -INFINITY, l = 0.f;
          for (int y = c0; y <= c1; ++y)
            m = fmaxf(m, __ldcg(A.parts + (long long)(y == c0 ? s0 : 2 * y) * kPart + HD * kPRows + row));
#pragma unroll
          for (int i = 0; i < HD; ++i) o[i] = 0.f;
          for (int y = c0; y <= c1; ++y) {
            const float* from = A.parts + (long long)(y == c0 ? s0 : 2 * y) * kPart + row;
            const float mw = __ldcg(from + HD * kPRows), lw = __ldcg(from + (HD + 1) * kPRows);
            const float f = mw == -INFINITY && lw == 0.f ? 0.f : p_ex2(mw - m);
            l = fmaf(f, lw, l);
#pragma unroll
            for (int i = 0; i < HD; ++i) o[i] = fmaf(f, __ldcg(from + i * kPRows), o[i]);
          }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");  // flag may be written again
      }
      if (write) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if constexpr (TWO) {
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(A.out) + to);
#pragma unroll
          for (int i = 0; i < HD; i += 4) dst[i / 4] = make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.out) + to);
          const bool bf = A.dtype == 2;
#pragma unroll
          for (int i = 0; i < HD; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = pack_out(bf, o[i + 2 * y] * inv, o[i + 2 * y + 1] * inv);
            dst[i / 8] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[seg.st]);
      seg.step();
    }
  } else if (warp < 20) {
    // ---- conversion: q of each item and K of its units, or V, to f16 tiles ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::kRegConvert));
    // two warps take the first half of every tile (64 positions), two the second
    const int t = tid & 127, v_side = warp >> 4, half = (warp >> 1) & 1;  // warps 12..15: K, 16..19: V
    uint64_t *raw_f = raw_full + v_side * kRawBars, *raw_e = raw_empty + v_side * kRawBars;
    Ring<kRawBars> raw;  // copy h is at barrier h % 6, in stage h % 3; this warp's are those with h % 2 = half
    if (half) raw.step();
    bool ok = true;
    // Half a tile (64 positions) of codes to f16: the chunks of 16 codes of a thread are all read, the codes' place is
    // given back, then they are converted.  Rows from `valid` on become 0.
    auto half_tile = [&](uint8_t* dst, int valid) {
      // Eight neighbouring lanes take four chunks of row r and four of row r ^ 5 (mod 8): under both swizzles they meet
      // eight different 16-byte columns, reading the codes and writing either half of the values.  A thread's rows
      // are 8 (16) apart, so its swizzled columns stay.
      constexpr int kMine = HD / 16, kStep = HD == 128 ? 8 : 16;
      const uint8_t* src = smem + P::kRawOff + (v_side * kRawStages + raw.st % kRawStages) * P::kRaw;
      const int w = warp & 1, r7 = ((t >> 3) & 3) ^ ((t >> 2) & 1) * 5;
      const int r0 = (HD == 128 ? 0 : w) * 8 + r7, panel = HD == 128 ? w : 0;
      const int from = HD == 128 ? r0 * 128 + (((panel * 4 + (t & 3)) ^ r7) << 4) : r0 * 64 + (((t & 3) ^ (r7 >> 1)) << 4);
      uint4 cw[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) cw[i] = *reinterpret_cast<const uint4*>(src + from + i * (kStep * HD));
      __syncwarp();
      if (lane == 0) mbar_arrive(&raw_e[raw.st]);
      raw.step(), raw.step();
      if (valid < 64) {
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (r0 + i * kStep >= valid) cw[i] = make_uint4(0, 0, 0, 0);
      }
      uint8_t* to = dst + panel * (kPRows * 128) + r0 * 128;
      const int c0 = ((t & 3) * 2 ^ r7) << 4;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        uint4 h0, h1;
        if constexpr (FMT == 0) {
          e4m3x4_to_f16x4(cw[i].x, h0.x, h0.y), e4m3x4_to_f16x4(cw[i].y, h0.z, h0.w);
          e4m3x4_to_f16x4(cw[i].z, h1.x, h1.y), e4m3x4_to_f16x4(cw[i].w, h1.z, h1.w);
        } else {
          const uint32_t in[4] = {cw[i].x ^ 0x80808080u, cw[i].y ^ 0x80808080u, cw[i].z ^ 0x80808080u, cw[i].w ^ 0x80808080u};
          uint32_t out[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            out[2 * y] = hsub2_u32(__byte_perm(in[y], 0x64646464u, 0x4140), 0x64806480u);
            out[2 * y + 1] = hsub2_u32(__byte_perm(in[y], 0x64646464u, 0x4342), 0x64806480u);
          }
          h0 = make_uint4(out[0], out[1], out[2], out[3]);
          h1 = make_uint4(out[4], out[5], out[6], out[7]);
        }
        uint8_t* at = to + i * (kStep * 128);
        *reinterpret_cast<uint4*>(at + c0) = h0;
        *reinterpret_cast<uint4*>(at + (c0 ^ 16)) = h1;
      }
    };
    // q of a segment: a warp brings in its 32 rows, a row at a time, lane l the dims l E .. l E + E - 1
    auto load_q = [&](const Seg* it, float* powers, int items) {
      constexpr int E = HD / 32, kBatch = TWO ? 4 : 8;
      const int r_first = (warp & 3) * 32;
      int tok = it->tile * A.tokens + r_first / A.group, h = r_first % A.group;
      const int tok_end = min(it->n, (it->tile + 1) * A.tokens);
#pragma unroll 1
      for (int r0 = 0; r0 < 32; r0 += kBatch) {
        Raw<E, TWO> raw_q[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          raw_q[b] = Raw<E, TWO>{};
          if (tok < tok_end)
            raw_q[b] = reinterpret_cast<const Raw<E, TWO>*>(static_cast<const char*>(A.q) +
                ((long long)(it->row0 + tok) * A.q_stride + (long long)(it->head * A.group + h) * HD) * (TWO ? 4 : 2))[lane];
          if (++h == A.group) h = 0, ++tok;
        }
        // the first rows are on their way while the last product with the old q ends
        if (r0 == 0 && items > 0 && !(ok = wait_warp(q_empty, (items - 1) & 1, dead, err))) return;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int row = r_first + r0 + b;
          float f[E];
          raw_q[b].get(f, A.dtype);
          unsigned top = 0;
#pragma unroll
          for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
          top = __reduce_max_sync(0xFFFFFFFFu, top);
          const int e = top == 0 ? 0 : min(max((int)(top >> 23) - 127, -120), 120);
          const float down = pow2i(-e) * A.sign;
          if (lane == 0) powers[row] = pow2i(e);
          uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
          for (int y = 0; y < E / 2; ++y) {
            const float x0 = f[2 * y] * down, x1 = f[2 * y + 1] * down;
            const __half2 hh = __floats2half2_rn(x0, x1);
            hi[y] = *reinterpret_cast<const uint32_t*>(&hh);
            const float2 back = __half22float2(hh);
            lo[y] = pack_half2(x0 - back.x, x1 - back.y);
          }
          const int byte = lane * E * 2;  // within the row's halves
          uint8_t* to = smem + P::kQ + (byte >> 7) * (kPRows * 128) + row * 128 + ((((byte & 127) >> 4) ^ (row & 7)) << 4) + (byte & 15);
          if constexpr (E == 4) {
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
            if constexpr (TWO) *reinterpret_cast<uint2*>(to + P::kTile) = make_uint2(lo[0], lo[1]);
          } else {
            *reinterpret_cast<uint32_t*>(to) = hi[0];
            if constexpr (TWO) *reinterpret_cast<uint32_t*>(to + P::kTile) = lo[0];
          }
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };
    Ring<kSegs> seg;
    int at = 0, items = 0, st = 0;  // st: the tile's place, of 2 (K) or kVStages (V)
    uint32_t ph = 0;
    const int places = v_side ? P::kVStages : 2;
    uint8_t* tiles = smem + (v_side ? P::kV : P::kK);
    while (at < n_units) {
      if (!(ok = wait_warp(&seg_full[seg.st], seg.ph, dead, err))) break;
      const Seg* it = segs + seg.st;
      const int end = it->end, length = it->length;
      int p = it->u0 * kPUnit + half * 64;
      // factors per 16 positions, fetched one unit ahead by 8 threads of the K side
      const long long line = ((long long)it->slot * A.C.kv_heads + it->head) * A.C.n_blocks;
      int e_next = 0;
      auto fetch = [&]() {
        if (!v_side && t < 8 && p + t * 16 < length) {  // (of the first half's warps)
          const long long b = line + ((p + t * 16) >> A.C.block_log2);
          e_next = A.C.k_exp[b] | A.C.v_exp[b] << 8;
        }
      };
      fetch();
      if (!v_side) {
        load_q(it, rf + (items & 3) * kPRows, items);
        if (!ok) break;
        ++items;
      }
#pragma unroll 1
      for (; at < end; ++at) {
        if (at >= places && !(ok = wait_warp(v_side ? &v_empty[TWO ? half : st] : &k_empty[st], ph ^ 1, dead, err))) break;
        if (!v_side && t < 8) {
          const int ek = kv8_exp((uint8_t)e_next), ev = kv8_exp((uint8_t)(e_next >> 8));
          factors[(at & 7) * 8 + t] = make_float4(pow2i(ek), (float)ev, pow2i(-ev), 0.f);
        }
        if (!(ok = wait_warp(&raw_f[raw.st], raw.ph, dead, err))) break;
        half_tile(tiles + st * P::kTile + half * (64 * 128), length - p);
        p += kPUnit;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_side ? &v_full[TWO ? half : st] : &k_full[st]);
        if (at + 1 < end) fetch();
        if (++st == places) st = 0, ph ^= 1;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[seg.st]);
      seg.step();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::kRegIssue));
    // The products: a warp for S and one for U, each kept in step as a whole (so that descriptors stay in uniform
    // registers) with one lane issuing; one warp for both was what bound a unit.
    if (warp == kMmaWarp) {
      // ---- S = Q K^T, up to three units ahead of U ----
      Ring<kSegs> seg;
      Ring<kScores> place;
      int item = 0, q_end = 0;
      bool ok = true;
      const uint64_t q_desc = tc_desc(smem + P::kQ, 1024, 16), k_desc = tc_desc(smem + P::kK, 1024, 16);
      constexpr uint32_t s_id = tc_idesc(kPUnit, false);
      for (int at = 0; at < n_units; ++at) {
        if (at == q_end) {
          if (!(ok = wait_warp(&seg_full[seg.st], seg.ph, dead, err))) break;
          q_end = segs[seg.st].end;
          __syncwarp();
          if (lane == 0) mbar_arrive(&seg_empty[seg.st]);
          seg.step();
          if (!(ok = wait_warp(q_full, item & 1, dead, err))) break;
          ++item;
        }
        if (at >= kScores && !(ok = wait_warp(&place_free[place.st], place.ph ^ 1, dead, err))) break;
        if (!(ok = wait_warp(&k_full[at & 1], (at >> 1) & 1, dead, err))) break;
        tc_fence_after();
        const uint32_t d = tmem + place.st * 128;
        const uint64_t b = k_desc + (((at & 1) * P::kTile) >> 4);
        if (elect_one()) {
#pragma unroll 2
          for (int y = 0; y < HD / 16; ++y) {
            const uint32_t step = ((y >> 2) * (kPRows * 128) + (y & 3) * 32) >> 4;
            tc_mma_ss(d, q_desc + step, b + step, s_id, y > 0);
            if constexpr (TWO) tc_mma_ss(d, q_desc + (P::kTile >> 4) + step, b + step, s_id, 1);
          }
          tc_commit(&s_full[place.st]);
          tc_commit(&k_empty[at & 1]);
          if (at + 1 == q_end) tc_commit(q_empty);
        }
        __syncwarp();
        place.step();
      }
      // every product is done before tensor memory is given back
      if (elect_one()) tc_commit(&last[0]);
      __syncwarp();
      mbar_wait(&last[0], 0, err);
    } else if (warp == kMmaWarp + 1) {
      // ---- U = P V ----
      Ring<kScores> place;
      Ring<P::kVStages * P::kVParts> vst;
      bool ok = true;
      const uint64_t v_desc = tc_desc(smem + P::kV, 1024, kPRows * 128);
      constexpr uint32_t u_id = tc_idesc(HD, true);
      const uint32_t d = tmem + kScores * 128;
      for (int at = 0; at < n_units; ++at) {
        if (!(ok = wait_warp(&p_full[place.st], place.ph, dead, err))) break;
        if (at >= 1 && !(ok = wait_warp(u_empty, (at - 1) & 1, dead, err))) break;
#pragma unroll 1
        for (int part = 0; part < P::kVParts; ++part) {
          if (!(ok = wait_warp(&v_full[vst.st], vst.ph, dead, err))) break;
          tc_fence_after();
          const uint32_t a = tmem + place.st * 128 + part * 64;
          const uint64_t b = v_desc + ((TWO ? part * (64 * 128) : vst.st * P::kTile) >> 4);
          if (elect_one()) {
#pragma unroll 2
            for (int y = 0; y < kPUnit / 16 / P::kVParts; ++y) {
              tc_mma_ts(d, a + y * 16, b + ((y * 16 * 128) >> 4), u_id, part > 0 || y > 0);
              if constexpr (TWO) tc_mma_ts(d, a + y * 16 + 8, b + ((y * 16 * 128) >> 4), u_id, 1);
            }
            if (part == P::kVParts - 1) tc_commit(u_full), tc_commit(&place_free[place.st]);
            tc_commit(&v_empty[vst.st]);
          }
          __syncwarp();
          vst.step();
        }
        if (!ok) break;
        place.step();
      }
      if (elect_one()) tc_commit(&last[1]);
      __syncwarp();
      mbar_wait(&last[1], 0, err);
    } else {
      // ---- TMA of the codes of K, or of V, 64 positions at a time ----
      const int v_side = warp - kTmaWarp;
      PItem item;
      if (!v_side) p_begin(item, A, pre, span[1], span[2]);
      if (lane == 0) {
        const CUtensorMap* map = v_side ? &vmap : &kmap;
        uint64_t *raw_f = raw_full + v_side * kRawBars, *raw_e = raw_empty + v_side * kRawBars;
        uint8_t* dst = smem + P::kRawOff + v_side * kRawStages * P::kRaw;
        Ring<kSegs> seg;
        Ring<kRawBars> raw, freed;  // freed: three copies behind, the last user of raw's stage
        int copies = 0, at = 0;
        bool ok = true;
        for (int i = 0; at < n_units; ++i) {
          if (!v_side) {  // the next segment: K's copies are the first to need it
            if (i > 0) p_next(item, A, pre, span[1] + at, span[2]);
            if (i >= kSegs && !(ok = wait_for(&seg_empty[seg.st], seg.ph ^ 1, dead, err))) break;
            Seg* to = const_cast<Seg*>(segs) + seg.st;
            to->row0 = item.s.row0, to->n = item.s.n, to->length = item.s.length, to->slot = item.s.slot;
            to->head = item.head, to->tile = item.tile;
            to->u0 = item.u0, to->u1 = item.u1, to->units = item.units, to->end = at + item.u1 - item.u0;
            to->first = item.first;
            mbar_arrive(&seg_full[seg.st]);
            // its rows of q on their way to L2
            const int tokens = min(A.tokens, item.s.n - item.tile * A.tokens), size = A.group * HD * (TWO ? 4 : 2);
            const char* q = static_cast<const char*>(A.q) + ((item.s.row0 + (long long)item.tile * A.tokens) * A.q_stride +
                                                             (long long)item.head * A.group * HD) * (TWO ? 4 : 2);
#pragma unroll 1
            for (int y = 0; y < tokens; ++y, q += A.q_stride * (TWO ? 4 : 2))
              asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(q), "r"(size) : "memory");
          } else if (!(ok = wait_for(&seg_full[seg.st], seg.ph, dead, err))) {
            break;
          }
          const Seg* it = segs + seg.st;
          const int y0 = (int)(((long long)it->slot * A.C.kv_heads + it->head) * A.C.max_ctx);
          const int x1 = 2 * it->u1, length = it->length;
          for (int x = 2 * it->u0; x < x1; ++x) {
            if (copies >= kRawStages) {
              if (!(ok = wait_for(&raw_e[freed.st], freed.ph, dead, err))) break;
              freed.step();
            }
            // a half that holds no position of the sequence is not needed (its codes become 0)
            if (x * 64 < length) {
              mbar_arrive_expect_tx(&raw_f[raw.st], P::kRaw);
              p_tma_3d(dst + raw.st % kRawStages * P::kRaw, map, 0, y0 + x * 64, A.layer, &raw_f[raw.st]);
            } else {
              mbar_arrive(&raw_f[raw.st]);
            }
            raw.step();
            ++copies;
          }
          if (!ok) break;
          at = it->end;
          mbar_arrive(&seg_empty[seg.st]);
          seg.step();
        }
        for (int i = max(0, copies - kRawStages); i < copies; ++i)  // the copies have landed before the CTA ends
          mbar_wait(&raw_f[i % kRawBars], (i / kRawBars) & 1, err);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int HD, int FMT, bool TWO>
cudaError_t launch(const PromptArgs& A, const Kv8Maps& M, int nsm, cudaStream_t s) {
  const int smem = PromptPlan<HD, TWO>::kPre + 8 * (A.R.n_seq + 1);
  attend_prompt_kernel<HD, FMT, TWO><<<nsm, kPThreads, smem, s>>>(A, M.k, M.v);
  return cudaGetLastError();
}

template <int HD, int FMT, bool TWO>
cudaError_t setup() {
  auto* fn = attend_prompt_kernel<HD, FMT, TWO>;
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, fn);
  if (e != cudaSuccess) return e;
  // the roles' register shares are drawn from what the block is launched with
  if ((a.numRegs + 7) / 8 * 8 < kRegs) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              PromptPlan<HD, TWO>::kPre + 8 * (kKv8MaxSeq + 1));
}

}  // namespace

int kv8_prompt_part_floats(int head_dim) { return (head_dim + 2) * kPRows; }

cudaError_t setup_kv8_prompt(int head_dim, int format) {
  cudaError_t a, b;
  if (head_dim == 128) {
    a = format == 0 ? setup<128, 0, false>() : setup<128, 1, false>();
    b = format == 0 ? setup<128, 0, true>() : setup<128, 1, true>();
  } else {
    a = format == 0 ? setup<64, 0, false>() : setup<64, 1, false>();
    b = format == 0 ? setup<64, 0, true>() : setup<64, 1, true>();
  }
  return a != cudaSuccess ? a : b;
}

cudaError_t launch_kv8_prompt(const Kv8Dev& C, const Kv8Rows& R, const Kv8Maps& M, int layer, unsigned* count,
                              float* parts, int nsm, const void* q, long long q_stride, void* out,
                              long long out_stride, int dtype, float scale, cudaStream_t s) {
  PromptArgs A;
  A.C = C, A.R = R, A.q = q, A.out = out, A.q_stride = q_stride, A.out_stride = out_stride;
  A.sign = scale < 0.f ? -1.f : 1.f;
  A.scale2 = scale * A.sign * 1.4426950408889634f;
  A.dtype = dtype, A.group = C.heads / C.kv_heads, A.layer = layer, A.tokens = kPRows / A.group;
  A.count = count, A.parts = parts;
  const bool two = dtype == 0;
  if (C.head_dim == 128) {
    if (C.format == 0) return two ? launch<128, 0, true>(A, M, nsm, s) : launch<128, 0, false>(A, M, nsm, s);
    return two ? launch<128, 1, true>(A, M, nsm, s) : launch<128, 1, false>(A, M, nsm, s);
  }
  if (C.format == 0) return two ? launch<64, 0, true>(A, M, nsm, s) : launch<64, 0, false>(A, M, nsm, s);
  return two ? launch<64, 1, true>(A, M, nsm, s) : launch<64, 1, false>(A, M, nsm, s);
}

}  // namespace strata
