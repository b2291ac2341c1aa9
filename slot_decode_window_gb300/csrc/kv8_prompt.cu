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
// Roles (20 warps): two warpgroups of softmax (even and odd units, a row a
// thread), one of correction (a row's output a thread), one of conversion, and
// a warp each for TMA and MMA.
// A role sees what another wrote through the chain of barriers between them;
// what a reader does not free by a barrier of its own (the units' factors and
// statistics, the rows' powers of two) has four slots, of which the chain keeps
// at most three in use.
//   TMA -> raw codes -> conversion -> f16 K, V -> MMA -> S -> softmax -> P (in
//   S's place) -> MMA -> U -> correction
#include "kv8.cuh"

namespace strata {
namespace {

constexpr int kPUnit = 128;      // positions per unit
constexpr int kPRows = 128;      // rows per tile
constexpr int kPThreads = 640;
constexpr int kRegs = 96;        // registers per thread at launch; the roles' shares below sum to 5 x 96
constexpr int kRegSoftmax = 112, kRegCorrect = 168, kRegConvert = 48, kRegIssue = 40;
static_assert(2 * kRegSoftmax + kRegCorrect + kRegConvert + kRegIssue <= 5 * kRegs, "register split");
constexpr float kPWeightTop = 14.f;
constexpr int kRawStages = 3;

template <int HD, bool TWO> struct PromptPlan {
  static constexpr int kTile = kPRows * HD * 2;      // a 128-row f16 tile: panels of 64 halves (one swizzle span)
  static constexpr int kRaw = kPUnit * HD;           // a unit's codes of K or V
  static constexpr int kVStages = TWO ? 1 : 2;
  static constexpr int kParts = TWO ? 2 : 1;
  static constexpr int kQ = 0;                       // byte offsets from a 1024-byte boundary
  static constexpr int kK = kQ + kParts * kTile;
  static constexpr int kV = kK + 2 * kTile;
  static constexpr int kRawOff = kV + kVStages * kTile;
  static constexpr int kStats = kRawOff + kRawStages * kRaw;  // [4][128] float2: a unit's maxima and sums
  static constexpr int kRf = kStats + 4 * kPRows * 8;         // [4][128] the rows' powers of two, by item
  static constexpr int kExp = kRf + 4 * kPRows * 4;           // [4][8] float4: a unit's factors per 16 positions
  static constexpr int kBars = kExp + 4 * 8 * 16;
  static constexpr int kMisc = kBars + 256;                   // tensor memory address, flags, scan sums
  static constexpr int kPre = kMisc + 256;
};

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
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
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
  while (!mbar_try_wait(bar, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > (1LL << 31)) {
      *dead = 1;
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
  return true;
}

// The same for a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* dead, unsigned* err) {
  return __all_sync(0xFFFFFFFFu, wait_for(bar, parity, dead, err));
}

__device__ __forceinline__ void p_tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ float p_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Four neighbouring values of a row.
__device__ __forceinline__ float4 p_load4(const void* p, int dtype, long long i) {
  if (dtype == 0) return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
  if (dtype == 1) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
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

// sum of floor((a i + b) / m) over i = 0..n-1, a, b >= 0 (Euclid's steps)
__device__ inline long long floor_sum(long long n, long long m, long long a, long long b) {
  long long sum = 0;
  while (n > 0) {
    sum += (n - 1) * n / 2 * (a / m) + n * (b / m);
    a %= m, b %= m;
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m, b = y % m;
    const long long t = m;
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
  if (tiles > t0) sum += floor_sum(tiles - t0, kPUnit, tokens, base + (long long)tokens * (t0 + 1) + kPUnit - 1);
  return sum;
}
__device__ __forceinline__ long long p_head_units(const Kv8Seq& s, int tokens) {
  return s.held_ok && s.n > 0 ? p_units_before(s, tokens, p_tiles(s, tokens)) : 0;
}

// The items of a CTA in turn; begin() finds the first, next() steps.
struct PItem {
  Kv8Seq s;
  int seq, head, tile, units;  // units of the whole item
  int u0, u1;                  // the CTA's part of them
  long long first;             // the item's first unit in the whole list
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
  while (pre[a + 1] <= lo) ++a;
  it.seq = a;
  it.s = kv8_seq(A.R, A.C, a);
  long long r = lo - pre[a];
  const long long per = p_head_units(it.s, A.tokens);
  it.head = (int)(r / per);
  r -= it.head * per;
  int t0 = 0, t1 = p_tiles(it.s, A.tokens);  // before(t0) <= r < before(t1)
  while (t1 - t0 > 1) {
    const int m = (t0 + t1) >> 1;
    if (p_units_before(it.s, A.tokens, m) <= r)
      t0 = m;
    else
      t1 = m;
  }
  it.tile = t0;
  it.units = p_units(it.s, A.tokens, t0);
  it.u0 = (int)(r - p_units_before(it.s, A.tokens, t0));
  it.u1 = (int)min((long long)it.units, it.u0 + (hi - lo));
  it.first = lo - it.u0;
}

// After a part that ended at unit u of the list (u < hi).
__device__ inline void p_next(PItem& it, const PromptArgs& A, const long long* pre, long long u, long long hi) {
  do {
    if (++it.tile >= p_tiles(it.s, A.tokens)) {
      it.tile = 0;
      if (++it.head >= A.C.kv_heads) {
        it.head = 0;
        do {
          ++it.seq;
        } while (pre[it.seq + 1] <= u);
        it.s = kv8_seq(A.R, A.C, it.seq);
      }
    }
    it.units = p_units(it.s, A.tokens, it.tile);
  } while (it.units == 0);
  it.u0 = 0;
  it.u1 = (int)min((long long)it.units, hi - u);
  it.first = u;
}

template <int HD, int FMT, bool TWO>
__global__ void __launch_bounds__(kPThreads, 1)
    attend_prompt_kernel(const __grid_constant__ PromptArgs A, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  using P = PromptPlan<HD, TWO>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float2* stats = reinterpret_cast<float2*>(smem + P::kStats);
  float* rf = reinterpret_cast<float*>(smem + P::kRf);
  float4* factors = reinterpret_cast<float4*>(smem + P::kExp);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::kBars);
  uint64_t *raw_full = bars, *raw_empty = bars + 3, *k_full = bars + 6, *k_empty = bars + 8, *v_full = bars + 10,
           *v_empty = bars + 12, *q_full = bars + 14, *q_empty = bars + 15, *s_full = bars + 16, *p_full = bars + 18,
           *u_full = bars + 20, *u_empty = bars + 22, *last = bars + 24;
  uint32_t* tmem_word = reinterpret_cast<uint32_t*>(smem + P::kMisc);
  volatile int* dead = reinterpret_cast<volatile int*>(smem + P::kMisc + 8);
  int* flag = reinterpret_cast<int*>(smem + P::kMisc + 12);
  long long* warp_sums = reinterpret_cast<long long*>(smem + P::kMisc + 16);
  long long* pre = reinterpret_cast<long long*>(smem + P::kPre);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned* err = A.C.err;

  if (tid == 0) {
    for (int i = 0; i < kRawStages; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_empty[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4), mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 4), mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 4);
      mbar_init(&u_full[i], 1), mbar_init(&u_empty[i], 4);
    }
    mbar_init(q_full, 4), mbar_init(q_empty, 1), mbar_init(last, 1);
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
  const long long total = pre[n_seq];
  const int G = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= G) return;
  const long long lo = total * blockIdx.x / G, hi = total * (blockIdx.x + 1) / G;
  const int n_units = (int)(hi - lo);

  if (warp == 16) {  // all of tensor memory: S0 S1 (128 columns each), U0 U1
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_word)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;

  if (warp < 8) {
    // ---- softmax: warpgroup `odd` takes units odd, odd + 2, ...; a row a thread ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax));
    const int odd = warp >> 2, row = tid & 127;
    const uint32_t s_addr = tmem + odd * 128 + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
    PItem it;
    p_begin(it, A, pre, lo, hi);
    bool ok = true;
    int n = 0;
    for (int item = 0; n < n_units && ok; ++item) {
      const int tok = it.tile * A.tokens + row / A.group;
      const bool on = row < A.tokens * A.group && tok < it.s.n;
      const int base = it.s.length - it.s.n;
      const int lim = on ? max(0, base + tok + 1) : 0;          // positions the row sees
      const int all = max(0, base + it.tile * A.tokens + 1);    // positions every row of the tile sees
      float f_row = 1.f;
      bool have = false;
      for (int x = it.u0 + ((n ^ odd) & 1); x < it.u1; x += 2) {
        const int at = n + x - it.u0;
        if (!(ok = wait_warp(&s_full[odd], (at >> 1) & 1, dead, err))) break;
        tc_fence_after();
        if (!have) f_row = rf[(item & 3) * kPRows + row], have = true;
        const float4* fac = factors + (at & 3) * 8;  // per 16 positions: scale 2^ek, ev, 2^-ev
        const int p0 = x * kPUnit;
        const bool masked = p0 + kPUnit > all;
        uint32_t r[32];
        float m = -INFINITY;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          tc_ld32(s_addr + ch * 32, r);
          tc_wait_ld();
          if (masked) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (p0 + ch * 32 + i >= lim) r[i] = 0xFF800000u;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              a = fmaxf(a, __uint_as_float(r[16 * h + i]));
              b = fmaxf(b, __uint_as_float(r[16 * h + i + 1]));
            }
            const float4 f = fac[ch * 2 + h];
            a = fmaxf(a, b);
            m = fmaxf(m, a == -INFINITY ? a : fmaf(a, f.x * f_row, f.y));
          }
        }
        const float z = m == -INFINITY ? 0.f : kPWeightTop - m;
        float l = 0.f;
        uint32_t rest[TWO ? 32 : 1];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          tc_ld32(s_addr + ch * 32, r);
          tc_wait_ld();
          uint32_t hi16[16], lo16[TWO ? 16 : 1];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 f = fac[ch * 2 + h];
            const float k = f.x * f_row, c = f.y + z;
            float sum = 0.f, sum2 = 0.f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float w0 = p_ex2(fmaf(__uint_as_float(r[16 * h + i]), k, c));
              float w1 = p_ex2(fmaf(__uint_as_float(r[16 * h + i + 1]), k, c));
              if (masked) {
                const int p = p0 + ch * 32 + 16 * h + i;
                if (p >= lim) w0 = 0.f;
                if (p + 1 >= lim) w1 = 0.f;
              }
              sum += w0, sum2 += w1;
              const __half2 hh = __floats2half2_rn(w0, w1);
              hi16[8 * h + i / 2] = *reinterpret_cast<const uint32_t*>(&hh);
              if constexpr (TWO) {
                const float2 back = __half22float2(hh);
                lo16[8 * h + i / 2] = pack_half2(w0 - back.x, w1 - back.y);
              }
            }
            l = fmaf(sum + sum2, f.z, l);
          }
          // P's first parts go to columns 0..63 and the second ones to 64..127 of S's 128, each when those have been read
          tc_st16(s_addr + ch * 16, hi16);
          if constexpr (TWO) {
            if (ch < 2) {
#pragma unroll
              for (int i = 0; i < 16; ++i) rest[16 * ch + i] = lo16[i];
            } else {
              if (ch == 2) {
                uint32_t t[16];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                  for (int i = 0; i < 16; ++i) t[i] = rest[16 * y + i];
                  tc_st16(s_addr + 64 + 16 * y, t);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) rest[i] = lo16[i];
              } else {
                uint32_t t[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) t[i] = rest[i];
                tc_st16(s_addr + 96, t);
                tc_st16(s_addr + 112, lo16);
              }
            }
          }
        }
        stats[(at & 3) * kPRows + row] = make_float2(m, l);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[odd]);
      }
      n += it.u1 - it.u0;
      if (n < n_units) p_next(it, A, pre, lo + n, hi);
    }
  } else if (warp < 12) {
    // ---- correction: a row's output in registers ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegCorrect));
    const int row = tid & 127;
    const uint32_t u_addr = tmem + 256 + ((uint32_t)(warp & 3) << 21);
    PItem it;
    p_begin(it, A, pre, lo, hi);
    bool ok = true;
    int n = 0;
    while (n < n_units) {
      float o[HD];
#pragma unroll
      for (int i = 0; i < HD; ++i) o[i] = 0.f;
      float m = -INFINITY, l = 0.f;
      for (int x = it.u0; x < it.u1; ++x) {
        const int at = n + x - it.u0;
        if (ok) ok = wait_warp(&u_full[at & 1], (at >> 1) & 1, dead, err);
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
          tc_ld32(u_addr + (at & 1) * 128 + ch * 32, r);
          if (grew) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[ch * 32 + i] *= a;
          }
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[ch * 32 + i] = fmaf(__uint_as_float(r[i]), b, o[ch * 32 + i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&u_empty[at & 1]);
      }
      n += it.u1 - it.u0;
      const int tok = it.tile * A.tokens + row / A.group;
      const bool on = row < A.tokens * A.group && tok < it.s.n;
      const long long to = (long long)(it.s.row0 + tok) * A.out_stride + (long long)(it.head * A.group + row % A.group) * HD;
      bool write = on && ok;
      if (it.u0 != 0 || it.u1 != it.units) {
        constexpr int kPart = (HD + 2) * kPRows;
        float* part = A.parts + (long long)(2 * blockIdx.x + (it.first + it.u0 == lo ? 0 : 1)) * kPart + row;
#pragma unroll
        for (int i = 0; i < HD; ++i) part[i * kPRows] = o[i];
        part[HD * kPRows] = m, part[(HD + 1) * kPRows] = l;
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int c0 = (int)(((it.first + 1) * G - 1) / total), c1 = (int)(((it.first + it.units) * G - 1) / total);
        if (row == 0) {
          __threadfence();
          *flag = atomicInc(&A.count[c0], (unsigned)(c1 - c0)) == (unsigned)(c1 - c0);
          __threadfence();
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        write = write && *flag;
        if (write) {
          const int s0 = 2 * c0 + (total * c0 / G == it.first ? 0 : 1);
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
#pragma unroll
        for (int i = 0; i < HD; i += 4)
          p_store4(A.out, A.dtype, to + i, make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv));
      }
      if (n < n_units) p_next(it, A, pre, lo + n, hi);
    }
  } else if (warp < 16) {
    // ---- conversion: q of each item, then K and V of its units, to f16 tiles ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegConvert));
    const int t = tid & 127;
    PItem kt;  // the K side runs one unit ahead of the V side
    p_begin(kt, A, pre, lo, hi);
    int k_item = 0, k_at = 0, k_end = kt.u1 - kt.u0;  // units of the list before the K side's item ends
    int k_x = kt.u0, v_x = kt.u0, v_end = k_end;
    int v_len = kt.s.length, k_len = kt.s.length, v_len_next = 0, v_x_next = 0, v_end_next = 0;
    bool ok = true, k_new = true;
    int raw = 0;
    // one tile of codes to f16; positions from `length` on become 0
    auto tile = [&](uint8_t* dst, int p0, int length) {
      const uint8_t* src = smem + P::kRawOff + (raw % kRawStages) * P::kRaw;
      constexpr int kChunks = HD / 16;  // 16-code chunks per row
#pragma unroll 2
      for (int j = 0; j < kChunks; ++j) {
        const int id = j * 128 + t, r = id / kChunks, ch = id % kChunks;
        const uint8_t* from = HD == 128 ? src + r * 128 + ((ch ^ (r & 7)) << 4) : src + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
        uint4 cw = *reinterpret_cast<const uint4*>(from);
        if (p0 + r >= length) cw = make_uint4(0, 0, 0, 0);
        uint4 h0, h1;
        if constexpr (FMT == 0) {
          h0.x = e4m3x2_to_f16x2(cw.x & 0xFFFFu), h0.y = e4m3x2_to_f16x2(cw.x >> 16);
          h0.z = e4m3x2_to_f16x2(cw.y & 0xFFFFu), h0.w = e4m3x2_to_f16x2(cw.y >> 16);
          h1.x = e4m3x2_to_f16x2(cw.z & 0xFFFFu), h1.y = e4m3x2_to_f16x2(cw.z >> 16);
          h1.z = e4m3x2_to_f16x2(cw.w & 0xFFFFu), h1.w = e4m3x2_to_f16x2(cw.w >> 16);
        } else {
          const uint32_t in[4] = {cw.x ^ 0x80808080u, cw.y ^ 0x80808080u, cw.z ^ 0x80808080u, cw.w ^ 0x80808080u};
          uint32_t out[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            out[2 * i] = hsub2_u32(__byte_perm(in[i], 0x64646464u, 0x4140), 0x64806480u);
            out[2 * i + 1] = hsub2_u32(__byte_perm(in[i], 0x64646464u, 0x4342), 0x64806480u);
          }
          h0 = make_uint4(out[0], out[1], out[2], out[3]);
          h1 = make_uint4(out[4], out[5], out[6], out[7]);
        }
        // the two halves' stores alternate so that 8 lanes of a row meet 8 different chunks
        uint8_t* to = dst + (ch >> 2) * (kPRows * 128) + r * 128;
        const int c0 = (ch & 3) * 2, flip = ch >> 2;
        const uint4 first = flip ? h1 : h0, second = flip ? h0 : h1;
        *reinterpret_cast<uint4*>(to + (((c0 + flip) ^ (r & 7)) << 4)) = first;
        *reinterpret_cast<uint4*>(to + (((c0 + 1 - flip) ^ (r & 7)) << 4)) = second;
      }
    };
    auto done = [&](uint64_t* bar) {
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar);
        mbar_arrive(&raw_empty[raw % kRawStages]);
      }
      ++raw;
    };
    for (int v_at = -1; v_at < n_units && ok; ++v_at) {
      if (k_at < n_units) {
        if (k_new) {  // q of the item, once the last product with the old one is done
          if (k_item > 0 && !(ok = wait_warp(q_empty, (k_item - 1) & 1, dead, err))) break;
          const int tok = kt.tile * A.tokens + t / A.group;
          const bool on = t < A.tokens * A.group && tok < kt.s.n;
          const long long from = (long long)(kt.s.row0 + tok) * A.q_stride + (long long)(kt.head * A.group + t % A.group) * HD;
          unsigned top = 0;
          if (on) {
#pragma unroll 8
            for (int i = 0; i < HD; i += 4) {
              const float4 f = p_load4(A.q, A.dtype, from + i);
              top = max(max(top, __float_as_uint(f.x) & 0x7FFFFFFFu), __float_as_uint(f.y) & 0x7FFFFFFFu);
              top = max(max(top, __float_as_uint(f.z) & 0x7FFFFFFFu), __float_as_uint(f.w) & 0x7FFFFFFFu);
            }
          }
          const int e = top == 0 ? 0 : min(max((int)(top >> 23) - 127, -120), 120);
          const float down = pow2i(-e) * A.sign;
          rf[(k_item & 3) * kPRows + t] = pow2i(e);
#pragma unroll 2
          for (int i = 0; i < HD; i += 8) {
            float f[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) f[y] = 0.f;
            if (on) {
              const float4 a = p_load4(A.q, A.dtype, from + i), b = p_load4(A.q, A.dtype, from + i + 4);
              f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
            }
            uint32_t h[4], g[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float x0 = f[2 * y] * down, x1 = f[2 * y + 1] * down;
              const __half2 hh = __floats2half2_rn(x0, x1);
              h[y] = *reinterpret_cast<const uint32_t*>(&hh);
              if constexpr (TWO) {
                const float2 back = __half22float2(hh);
                g[y] = pack_half2(x0 - back.x, x1 - back.y);
              }
            }
            uint8_t* to = smem + P::kQ + (i >> 6) * (kPRows * 128) + t * 128 + ((((i & 63) >> 3) ^ (t & 7)) << 4);
            *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
            if constexpr (TWO) *reinterpret_cast<uint4*>(to + P::kTile) = make_uint4(g[0], g[1], g[2], g[3]);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full);
          k_new = false;
        }
        const int st = k_at & 1;
        if (k_at >= 2 && !(ok = wait_warp(&k_empty[st], ((k_at >> 1) - 1) & 1, dead, err))) break;
        if (t < 8) {  // factors per 16 positions
          const int p = k_x * kPUnit + t * 16;
          int ek = 0, ev = 0;
          if (p < k_len) {
            const long long line = (long long)kt.s.slot * A.C.kv_heads + kt.head;
            ek = kv8_exp(A.C.k_exp[line * A.C.n_blocks + (p >> A.C.block_log2)]);
            ev = kv8_exp(A.C.v_exp[line * A.C.n_blocks + (p >> A.C.block_log2)]);
          }
          factors[(k_at & 3) * 8 + t] = make_float4(A.scale2 * pow2i(ek), (float)ev, pow2i(-ev), 0.f);
        }
        if (!(ok = wait_warp(&raw_full[raw % kRawStages], (raw / kRawStages) & 1, dead, err))) break;
        tile(smem + P::kK + st * P::kTile, k_x * kPUnit, k_len);
        done(&k_full[st]);
        ++k_at, ++k_x;
      }
      if (v_at >= 0) {
        const int st = v_at % P::kVStages;
        if (v_at >= P::kVStages && !(ok = wait_warp(&v_empty[st], (v_at / P::kVStages - 1) & 1, dead, err))) break;
        if (!(ok = wait_warp(&raw_full[raw % kRawStages], (raw / kRawStages) & 1, dead, err))) break;
        tile(smem + P::kV + st * P::kTile, v_x * kPUnit, v_len);
        done(&v_full[st]);
        ++v_x;
        if (v_at + 1 == v_end && v_at + 1 < n_units) v_x = v_x_next, v_len = v_len_next, v_end = v_end_next;
      }
      if (k_at == k_end && k_at < n_units) {
        p_next(kt, A, pre, lo + k_at, hi);
        k_end += kt.u1 - kt.u0;
        k_x = kt.u0, k_len = kt.s.length, k_new = true, ++k_item;
        v_x_next = k_x, v_len_next = k_len, v_end_next = k_end;  // the V side changes over one step later
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegIssue));
    if (warp == 16 && lane == 0) {
      // ---- MMA ----
      PItem it;
      p_begin(it, A, pre, lo, hi);
      int item = 0, q_end = it.u1 - it.u0;
      bool ok = true, fresh = true;
      const uint64_t q_desc = tc_desc(smem + P::kQ, 1024, 16), k_desc = tc_desc(smem + P::kK, 1024, 16),
                     v_desc = tc_desc(smem + P::kV, 1024, kPRows * 128);
      constexpr uint32_t s_id = tc_idesc(kPUnit, false), u_id = tc_idesc(HD, true);
      auto scores = [&](int at) {  // S(at) = Q K(at)^T
        if (fresh) {
          if (!(ok = wait_for(q_full, item & 1, dead, err))) return;
          fresh = false;
        }
        if (!(ok = wait_for(&k_full[at & 1], (at >> 1) & 1, dead, err))) return;
        tc_fence_after();
        const uint32_t d = tmem + (at & 1) * 128;
#pragma unroll
        for (int part = 0; part < P::kParts; ++part)
#pragma unroll
          for (int y = 0; y < HD / 16; ++y) {
            const uint64_t step = ((y >> 2) * (kPRows * 128) + (y & 3) * 32) >> 4;
            tc_mma_ss(d, q_desc + step + ((part * P::kTile) >> 4), k_desc + step + (((at & 1) * P::kTile) >> 4), s_id,
                      part > 0 || y > 0);
          }
        tc_commit(&s_full[at & 1]);
        tc_commit(&k_empty[at & 1]);
        if (at + 1 == q_end) {
          tc_commit(q_empty);
          if (at + 1 < n_units) {
            p_next(it, A, pre, lo + at + 1, hi);
            q_end += it.u1 - it.u0;
            ++item, fresh = true;
          }
        }
      };
      scores(0);
      if (ok && n_units > 1) scores(1);
      for (int at = 0; at < n_units && ok; ++at) {
        if (!(ok = wait_for(&p_full[at & 1], (at >> 1) & 1, dead, err))) break;
        if (!(ok = wait_for(&v_full[at % P::kVStages], (at / P::kVStages) & 1, dead, err))) break;
        if (at >= 2 && !(ok = wait_for(&u_empty[at & 1], ((at >> 1) - 1) & 1, dead, err))) break;
        tc_fence_after();
        const uint32_t a = tmem + (at & 1) * 128, d = tmem + 256 + (at & 1) * 128;
#pragma unroll
        for (int part = 0; part < P::kParts; ++part)
#pragma unroll
          for (int y = 0; y < kPUnit / 16; ++y)
            tc_mma_ts(d, a + part * 64 + y * 8,
                      v_desc + ((y * 16 * 128) >> 4) + (((at % P::kVStages) * P::kTile) >> 4), u_id, part > 0 || y > 0);
        tc_commit(&u_full[at & 1]);
        tc_commit(&v_empty[at % P::kVStages]);
        if (at + 2 < n_units) scores(at + 2);
      }
      // every product is done before tensor memory is given back
      tc_commit(last);
      mbar_wait(last, 0, err);
    } else if (warp == 17 && lane == 0) {
      // ---- TMA: K0, K1, V0, K2, V1, ..., two boxes of 64 positions each ----
      PItem kt, vt;
      p_begin(kt, A, pre, lo, hi);
      vt = kt;
      int k_at = 0, k_end = kt.u1 - kt.u0, v_end = k_end, k_x = kt.u0, v_x = kt.u0, raw = 0;
      bool ok = true;
      auto copy = [&](const CUtensorMap* map, const PItem& it, int x) {
        const int st = raw % kRawStages;
        if (raw >= kRawStages && !(ok = wait_for(&raw_empty[st], (raw / kRawStages - 1) & 1, dead, err))) return;
        uint8_t* dst = smem + P::kRawOff + st * P::kRaw;
        const int y = (int)(((long long)it.s.slot * A.C.kv_heads + it.head) * A.C.max_ctx + (long long)x * kPUnit);
        // the second box only where it holds positions of the sequence: the rows of the next head or past the end
        // of the array are never needed (their codes become 0)
        const bool both = x * kPUnit + 64 < it.s.length;
        mbar_arrive_expect_tx(&raw_full[st], both ? P::kRaw : P::kRaw / 2);
        p_tma_3d(dst, map, 0, y, A.layer, &raw_full[st]);
        if (both) p_tma_3d(dst + P::kRaw / 2, map, 0, y + 64, A.layer, &raw_full[st]);
        ++raw;
      };
      for (int v_at = -1; v_at < n_units && ok; ++v_at) {
        if (k_at < n_units) {
          if (k_at == k_end) {
            p_next(kt, A, pre, lo + k_at, hi);
            k_end += kt.u1 - kt.u0, k_x = kt.u0;
          }
          copy(&kmap, kt, k_x++);
          ++k_at;
        }
        if (v_at >= 0 && ok) {
          if (v_at == v_end) {
            p_next(vt, A, pre, lo + v_at, hi);
            v_end += vt.u1 - vt.u0, v_x = vt.u0;
          }
          copy(&vmap, vt, v_x++);
        }
      }
      for (int i = max(0, raw - kRawStages); i < raw; ++i)  // the copies have landed before the CTA ends
        mbar_wait(&raw_full[i % kRawStages], (i / kRawStages) & 1, err);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int HD, int FMT, bool TWO>
cudaError_t launch(const PromptArgs& A, const Kv8Maps& M, int nsm, cudaStream_t s) {
  const int smem = 1024 + PromptPlan<HD, TWO>::kPre + 8 * (A.R.n_seq + 1);
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
                              1024 + PromptPlan<HD, TWO>::kPre + 8 * (kKv8MaxSeq + 1));
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
