// Attention of a call's rows over the slots' 8-bit caches.
#include "kv8.cuh"

namespace strata {
namespace {

// ---------------------------------------------------------------------------
// Few rows per slot: the cache is read once, at the memory's rate.
//
// The rows of a sequence that share a kv head (its rows x group query heads)
// are the N side of mma.sync m16n8k16 products whose M side is the cache: S^T =
// K Q^T (16 positions x rows) and O^T = V^T P^T (16 dims x rows), so that a
// tile of 8 rows wastes nothing and a lane's accumulators are few.  The weights
// turn from S^T's layout to P^T's by movmatrix.
// Positions are cut into units of 64 (128 for
// heads of 64, so that a copy and a step of a warp stay as long).  All units of all (sequence, row tile, kv
// head) items form one list, and each CTA (one per SM) takes an equal
// contiguous part of it, so that one long conversation and many short ones fill
// the GPU alike.  A producer thread streams the units' codes by TMA into a
// ring; four warps share a unit, groups of four take units
// in turn, and every warp keeps its own softmax state; the warps join once per
// item.  An item cut by a CTA border leaves its parts (maximum, sum,
// unnormalised output) in the workspace; the last CTA to finish joins them in
// CTA order, so the bits do not depend on timing.
//
// Weights: with scores s_j (base 2) and a block's value exponent ev, the state
// follows t_j = s_j + ev: w_j = 2^(t_j - max t), O = sum w_j code_j,
// l = sum w_j 2^-ev, out = O / l.  Whatever the exponents, the largest weight
// that meets a code is 1 (held times 2^14 so that 16-bit weights keep 38 bits
// below it), and no block needs its own accumulator.
// What is rounded to 16 bits, for the matrix unit's sake: codes are exact in
// f16.  16-bit rows: q after a power of two per row (bf16 elements below 2^-17
// of the row's largest lose bits, a 2^-25 of it at most) and the weights (11
// bits, on their way into O only: a relative 2^-11 at most, to both sides, that
// averages out over positions; l sums them in f32), against the 8 or 11 bits
// that the result is rounded to.  f32 rows: both as two f16 parts (22 bits) that
// chain into one accumulator: 1.6e-7 off at 512 positions, fp32 products 1.1e-7.
// Scores, statistics and sums are f32; t_j is one f32 sum, so weights resolve
// 2^-24 of the largest |t_j|.
// Measured (32 / 8 heads of 128, bf16): 64 rows over 1.6 k to 8.2 k positions
// 112.5 us (84% of the measured HBM rate), one over 131071 52.8 us (75%; the
// start and the join of 19 parts are the rest).  With the rows on the M side
// and 8 warps of 168 registers these took 164 and 62 us.
// Registers: heads of 128 spill at the limits below (bytes stored, one tile of
// rows / two: 24 to 28 / 152 for 16-bit rows, 152 to 160 / 320 for f32 rows);
// heads of 64 none for 16-bit rows, up to 24 for f32 rows.
// ---------------------------------------------------------------------------
constexpr float kWeightTop = 14.f;  // weights are scaled by 2^14

// HD: head_dim; NT: tiles of 8 rows (1 or 2); PARTS: f16 parts of q and of the weights (1, or 2 for f32 rows).
template <int HD, int NT, int PARTS> struct SplitPlan {
  static constexpr int kRows = 8 * NT;
  // consumers: as many as their registers allow (with the producer, 13 warps leave 128 a thread, 9 leave 168; 16 + 1
  // would leave 96)
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kGroups = kWarps / 4;                // units under way at a time
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kSlabs = 128 / HD;                   // of 16 positions: a warp's part of a unit
  static constexpr int kUnit = 64 * kSlabs;                 // positions of a ring stage
  static constexpr int kFold = 16 / kSlabs;                 // units of a warp between folds of O (f32 rows)
  static constexpr int kTile = kUnit * HD;                  // bytes of one unit's K (or V) codes: 8 KB
  static constexpr int kStages = NT == 1 ? 9 : 8;           // 144 or 128 KB in flight; a multiple of kGroups
  static constexpr int kJoin = kWarps * kRows * (HD + 4) * 4;  // the warps' O (rows padded by 4 floats)
  static constexpr int kRing = 1024;                        // offsets in dynamic shared memory
  static constexpr int kJoinOff = kRing + kStages * 2 * kTile;
  static constexpr int kMlOff = kJoinOff + kJoin;           // [kWarps][kRows][2] maximum, sum
  static constexpr int kSeqOff = kMlOff + kWarps * kRows * 2 * 4;  // [n_seq] first row, rows, slot, length
};
constexpr int split_part(int hd) { return 16 * hd + 32; }  // floats of a part in the workspace: O, maxima, sums

struct AttendArgs {
  Kv8Dev C;
  Kv8Rows R;
  const void* q;
  void* out;
  long long q_stride, out_stride;
  float scale2;      // scale * log2(e)
  int dtype, group, layer, tile_rows, unit, grid;
  float* parts;      // [2 grid][split_part]
  unsigned* count;   // [grid] parts done of the item that starts last in a CTA; back to 0 when joined
};

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Units of row tile mt: positions that its last row sees.
__device__ __forceinline__ int tile_units(int n, int length, const AttendArgs& A, int mt) {
  const int last = min(n, (A.tile_rows * (mt + 1) - 1) / A.group + 1);
  const int seen = length - n + last;
  return seen <= 0 ? 0 : (seen + A.unit - 1) / A.unit;
}

// Cost of all row tiles of one kv head: their units, and `start` more for each tile that has any.
__device__ __forceinline__ int head_cost(int n, int length, const AttendArgs& A, int start) {
  const int tiles = (n * A.group + A.tile_rows - 1) / A.tile_rows;
  int sum = 0;
  for (int mt = 0; mt < tiles; ++mt) {
    const int u = tile_units(n, length, A, mt);
    sum += u > 0 ? u + start : 0;
  }
  return sum;
}

__device__ __forceinline__ void store_value4(void* p, int dtype, long long i, float4 v) {
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

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Four codes to two f16x2, exactly.  int8: 0x6400 | (code ^ 0x80) is 1152 + code.
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == 0) {
    e4m3x4_to_f16x4(w, lo, hi);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    lo = hsub2_u32(prmt(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2_u32(prmt(u, 0x64646464u, 0x4342), 0x64806480u);
  }
}

__device__ __forceinline__ void mma_acc(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// An 8 x 8 matrix of 16-bit values across the warp, transposed.
__device__ __forceinline__ uint32_t turn(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Weight of a part with maximum mw and sum lw under the joint maximum m: 0 for a
// part that saw nothing (a row of NaN has no maximum but a NaN sum, and stays NaN).
__device__ __forceinline__ float join_factor(float mw, float lw, float m) {
  return mw == -INFINITY && lw == 0.f ? 0.f : ex2(mw - m);
}

// A CTA's next item.  The list that the CTAs share is one of costs: an item's is `start` (what beginning an item costs a
// CTA, in units) and then its units.  A CTA whose share ends within the start does nothing of the item (u0 = u1 = 0).
struct Item {
  int row0, n, slot, length;  // the sequence
  int seq, head, mt;
  int u0, u1, units;          // the CTA's part, of the item's units
  int cost;                   // what the part takes up of the list
  long long first;            // the place of the item's first unit in the list
};

__device__ __forceinline__ Item next_item(const AttendArgs& A, const long long* pre, const int4* seqs, long long u,
                                          long long end, int seq, int start) {
  Item it;
  while (pre[seq + 1] <= u) ++seq;
  it.seq = seq;
  const int4 s = seqs[seq];
  it.row0 = s.x, it.n = s.y, it.slot = s.z, it.length = s.w;
  long long r = u - pre[seq];
  const int per_head = head_cost(it.n, it.length, A, start);
  it.head = (int)(r / per_head);
  r -= (long long)it.head * per_head;
  it.mt = 0;
  it.units = tile_units(it.n, it.length, A, 0);
  while (it.units == 0 || r >= it.units + start) {
    if (it.units > 0) r -= it.units + start;
    it.units = tile_units(it.n, it.length, A, ++it.mt);
  }
  it.first = u - r + start;
  it.u0 = (int)max(0ll, r - start);
  it.u1 = (int)min((long long)it.units, max(0ll, end - it.first));
  it.cost = (int)(min(end, it.first + it.units) - u);
  return it;
}

// Units that beginning an item is worth (its q, its join), where every CTA has at least kStartFrom units to do.  With 64
// conversations of other lengths, 3.4 items a CTA, equal units alone left the slowest CTA 20 us behind the median.  A
// start of 0, 4, 8, 12, 16 units: 124.4, 116.3, 112.6, 108.0, 108.0 us there, and 37.4, 35.3, 33.3, 34.8, 33.8 us with 24
// slots x 2 rows of 16 heads of 64; the same from 8 to 96 conversations (12 up to 4 % below 8, 0 up to 10 % above).  Short
// lists keep equal units: there a start would leave CTAs without any (from 12, 24, 48 units: 111.6, 112.6, 112.1 and
// 33.8, 33.3, 37.4 us).
constexpr int kStart = 8, kStartFrom = 24;

template <int HD, int FMT, int NT, int PARTS>
__global__ void __launch_bounds__(SplitPlan<HD, NT, PARTS>::kThreads, 1)
    attend_split_kernel(const __grid_constant__ AttendArgs A, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using P = SplitPlan<HD, NT, PARTS>;
  constexpr int kSteps = HD / 16;   // k-steps of K Q^T, m-tiles of V^T P^T
  constexpr int kPart = split_part(HD);
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + P::kStages;
  int* shared_word = reinterpret_cast<int*>(empty + P::kStages);
  long long* warp_sums = reinterpret_cast<long long*>(smem + 512);
  float* join = reinterpret_cast<float*>(smem + P::kJoinOff);
  float* ml = reinterpret_cast<float*>(smem + P::kMlOff);
  Item* cur = reinterpret_cast<Item*>(smem + 640);  // the consumers' item, for the join: not held in registers meanwhile
  int4* seqs = reinterpret_cast<int4*>(smem + P::kSeqOff);
  long long* pre = reinterpret_cast<long long*>(seqs + A.R.n_seq);  // costs before each sequence
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;

  if (smem_u32(smem) & 1023) {  // the swizzles count on it
    if (tid == 0) atomicOr(A.C.err, kErrConfig);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < P::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    fence_mbar_init();
  }
  // the cost of all before each sequence: a contiguous share per thread, joined by a scan
  const int n_seq = A.R.n_seq;
  int start;  // what an item's start counts for
  {
    constexpr int kScan = 256;
    const int share = (n_seq + kScan - 1) / kScan;
    int blind = 0;  // whether some rows see nothing
    long long units = 0;
    if (tid < kScan) {
      for (int i = tid * share; i < min(n_seq, (tid + 1) * share); ++i) {
        const Kv8Seq s = kv8_seq(A.R, A.C, i);
        seqs[i] = make_int4(s.row0, s.held_ok ? s.n : 0, s.slot, s.length);
        if (s.held_ok) units += head_cost(s.n, s.length, A, 0);
        blind |= s.rows_ok && (!s.held_ok || s.length < s.n);
        if (!s.held_ok && blockIdx.x == 0) atomicOr(A.C.err, kErrIndex);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xFFFFFFFFu, units, o);
    if (lane == 0 && warp < kScan / 32) warp_sums[kScan / 32 + warp] = units;
    blind = __syncthreads_or(blind);
    units = 0;
    for (int w = 0; w < kScan / 32; ++w) units += warp_sums[kScan / 32 + w];
    start = units * A.C.kv_heads >= (long long)kStartFrom * gridDim.x ? kStart : 0;
    long long sum = 0;
    if (tid < kScan) {
      for (int i = tid * share; i < min(n_seq, (tid + 1) * share); ++i) {
        const int4 s = seqs[i];
        sum += (long long)head_cost(s.y, s.w, A, start) * A.C.kv_heads;
        pre[i + 1] = sum;
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
    // rows that see nothing (or whose slot or length is out of range) are zero
    for (int i = blockIdx.x; blind && i < n_seq; i += gridDim.x) {
      const Kv8Seq s = kv8_seq(A.R, A.C, i);
      if (!s.rows_ok) continue;
      const int rows = s.held_ok ? min(s.n, max(0, s.n - s.length)) : s.n;
      const int w4 = A.C.heads * HD / 4;
      for (int j = tid; j < rows * w4; j += P::kThreads)
        store_value4(A.out, A.dtype, (long long)(s.row0 + j / w4) * A.out_stride + j % w4 * 4, make_float4(0, 0, 0, 0));
    }
  }

  const long long total = pre[n_seq];
  // as many CTAs as give each group of warps a unit: more would only make more parts to join
  const int G = (int)min((long long)gridDim.x, (total + P::kGroups - 1) / P::kGroups);
  if ((int)blockIdx.x >= G) return;
  const long long lo = total * blockIdx.x / G, hi = total * (blockIdx.x + 1) / G;
  int seq0 = 0;
  {
    int a = 0, b = n_seq;  // the sequence that holds place lo: pre[seq0] <= lo < pre[seq0 + 1]
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (pre[m] <= lo)
        a = m;
      else
        b = m;
    }
    seq0 = a;
  }

  if (warp == P::kWarps) {
    // ---- producer ----
    if (lane != 0) return;
    int n = 0, seq = seq0;
    bool ok = true;
    for (long long u = lo; u < hi && ok;) {
      const Item it = next_item(A, pre, seqs, u, hi, seq, start);
      seq = it.seq;
      const long long line = (long long)it.slot * A.C.kv_heads + it.head, row = line * A.C.max_ctx;
      // what the consumers will load when they come to the item, on its way to L2: q's rows, the first exponents
      if (it.u0 < it.u1) {
        const int size = PARTS == 2 ? 4 : 2, t0 = it.mt * P::kRows / A.group;
        const int t1 = min(it.n, (it.mt * P::kRows + P::kRows - 1) / A.group + 1);
        const char* q = static_cast<const char*>(A.q) +
                        ((it.row0 + t0) * A.q_stride + (long long)it.head * A.group * HD) * size;
#pragma unroll 1
        for (int t = t0; t < t1; ++t, q += A.q_stride * size)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(q), "r"(A.group * HD * size) : "memory");
        const long long e = line * A.C.n_blocks + ((it.u0 * P::kUnit) >> A.C.block_log2);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(A.C.k_exp + e));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(A.C.v_exp + e));
      }
      for (int x = it.u0; x < it.u1; ++x, ++n) {
        const int st = n % P::kStages;
        if (n >= P::kStages && !mbar_wait(&empty[st], (n / P::kStages - 1) & 1, A.C.err)) {
          ok = false;
          break;
        }
        uint8_t* dst = smem + P::kRing + st * 2 * P::kTile;
        // boxes of 64 positions; one that holds none of the sequence's is left out (its place is not read)
        const int boxes = P::kSlabs == 1 || x * P::kUnit + 64 < it.length ? P::kSlabs : 1;
        mbar_arrive_expect_tx(&full[st], 2 * boxes * 64 * HD);
#pragma unroll
        for (int b = 0; b < P::kSlabs; ++b) {
          if (b >= boxes) break;
          const int y = (int)(row + (long long)x * P::kUnit + 64 * b);
          tma_3d(dst + b * 64 * HD, &kmap, 0, y, A.layer, &full[st]);
          tma_3d(dst + P::kTile + b * 64 * HD, &vmap, 0, y, A.layer, &full[st]);
        }
      }
      u += it.cost;
    }
    if (!ok)  // the copies in flight land before this thread leaves
      for (int i = max(0, n - P::kStages); i < n; ++i)
        mbar_wait(&full[i % P::kStages], (i / P::kStages) & 1, A.C.err);
    return;
  }

  // ---- consumers: warp w takes quarter w mod 4 of the positions of units w / 4, w / 4 + kGroups, ... of the CTA's list.
  // (Stages are a multiple of the groups, so a stage's units are all of one group, which waits for every phase of it.)
  static_assert(P::kStages % P::kGroups == 0, "a stage belongs to one group of warps");
  const int mine = warp >> 2, slab0 = (warp & 3) * 16 * P::kSlabs;
  int n = 0, seq = seq0;
  bool ok = true;
  for (long long u = lo; u < hi;) {
    int u0, u1, length, min_pos, cost;
    long long line;
    uint32_t qb[PARTS][NT][kSteps][2];  // q as the B operand
    float rf[NT][2];                    // score factors of rows 8 nt + 2c and + 1 (the columns of S^T that this lane holds)
    int lim[NT][2];                     // positions that they see
    {
      const Item it = next_item(A, pre, seqs, u, hi, seq, start);
      seq = it.seq, cost = it.cost;
      if (it.u0 >= it.u1) {
        u += cost;
        continue;
      }
      if (tid == 0) *cur = it;
      u0 = it.u0, u1 = it.u1, length = it.length;
      line = ((long long)it.slot * A.C.kv_heads + it.head) * A.C.n_blocks;
      const int rows = min(P::kRows, it.n * A.group - it.mt * P::kRows);  // of this tile
      const int p_first = length - it.n;                                 // position of the sequence's first row
      min_pos = p_first + it.mt * P::kRows / A.group;                    // position of the tile's first row
      // lane (g, c) of k-step y holds dims c HD/4 + 4y .. + 3 of row 8 nt + g; all loads are on their way at once
      // (rows past the tile's load its last one, and become 0)
      constexpr int kVec = HD / 4 * (PARTS == 2 ? 4 : 2) / 16;
      uint4 raw[NT][kVec];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int m = it.mt * P::kRows + min(8 * nt + g, rows - 1);
        const long long at = (long long)(it.row0 + m / A.group) * A.q_stride +
                             (long long)(it.head * A.group + m % A.group) * HD + c * (HD / 4);
        const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(A.q) + at * (PARTS == 2 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < kVec; ++i) raw[nt][i] = from[i];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[HD / 4];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if constexpr (PARTS == 2)
            Val<float>::unpack(raw[nt][i], f + 4 * i);
          else if (A.dtype == 1)
            Val<__half>::unpack(raw[nt][i], f + 8 * i);
          else
            Val<__nv_bfloat16>::unpack(raw[nt][i], f + 8 * i);
        }
        if (8 * nt + g >= rows) {
#pragma unroll
          for (int d = 0; d < HD / 4; ++d) f[d] = 0.f;
        }
        // a power of two per row brings its largest element to [1, 2)
        unsigned top = 0;
#pragma unroll
        for (int d = 0; d < HD / 4; ++d) top = max(top, __float_as_uint(f[d]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const int e = top == 0 ? 0 : min(max((int)(top >> 23) - 127, -120), 120);
        const float down = pow2i(-e);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int r = 8 * nt + 2 * c + y;
          rf[nt][y] = kv8_row_factor(A.scale2, pow2i(__shfl_sync(0xFFFFFFFFu, e, (2 * c + y) * 4)));
          lim[nt][y] = r < rows ? max(0, p_first + (it.mt * P::kRows + r) / A.group + 1) : 0;
        }
#pragma unroll
        for (int y = 0; y < kSteps; ++y) {
          float h[4], l[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            h[d] = f[4 * y + d] * down;
            l[d] = h[d] - __half2float(__float2half_rn(h[d]));
          }
          qb[0][nt][y][0] = pack_half2(h[0], h[1]), qb[0][nt][y][1] = pack_half2(h[2], h[3]);
          if constexpr (PARTS == 2) qb[1][nt][y][0] = pack_half2(l[0], l[1]), qb[1][nt][y][1] = pack_half2(l[2], l[3]);
        }
      }
    }
    // this warp's units of the part, and the exponent bytes of its slabs, fetched a step ahead
    int x = u0 + (mine + P::kGroups - n % P::kGroups) % P::kGroups;
    int ek_next[P::kSlabs], ev_next[P::kSlabs];
    auto fetch = [&](int unit) {
#pragma unroll
      for (int b = 0; b < P::kSlabs; ++b) {
        const int p = unit * P::kUnit + slab0 + 16 * b;
        ek_next[b] = ev_next[b] = kKv8Bias;
        if (p < length) {
          ek_next[b] = A.C.k_exp[line + (p >> A.C.block_log2)];
          ev_next[b] = A.C.v_exp[line + (p >> A.C.block_log2)];
        }
      }
    };
    fetch(x);

    // O^T: lane (g, c) of m-tile i holds dims g HD/8 + 2i and + 1 of rows 8 nt + 2c and + 1
    float o[kSteps][NT][4];
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    // m: what the weights are relative to, kWeightTop below the maximum of t.  Rounded up, so that no weight exceeds
    // 2^kWeightTop where a step of m is larger than that (from m = 2^25 on; f16 holds 2^kWeightTop but not four times it).
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
    constexpr int kRowF = HD + 4;
    float* own = join + warp * P::kRows * kRowF;
    // f32 rows: every kFold units O goes to the warp's place of the join, relative to the m that stands behind each row
    // there, and starts anew.  The tensor core's adds cut off: a sum left in one accumulator is up to 7e-8 short for each
    // of them, without end (a CTA's 131071 positions came out 1e-4 short, folded 2e-7 at any length).  64 f32 rows over
    // 4 k to 8.2 k positions: 173.6 us, 164.4 without; folded every 8 units 176.1, every 4 181.3, each unit's sum added by
    // itself 195.1.  16-bit rows, with half the adds, stay as they are: their sums are 5e-5 short after 131071 positions
    // in one CTA and half a step of f16 short after 1.3 million, and even folds 256 units apart cost 64 bf16 rows 4 %.
    int held = 0;  // units that this warp has seen of the item
    auto fold = [&](bool first) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float* row = own + (8 * nt + 2 * c + y) * kRowF;
          const float then = first ? -INFINITY : row[HD], a = then == m[nt][y] ? 1.f : ex2(then - m[nt][y]);
#pragma unroll
          for (int i = 0; i < kSteps; i += 2) {
            float4* to = reinterpret_cast<float4*>(row + g * (HD / 8) + 2 * i);
            const float4 v = first ? make_float4(0, 0, 0, 0) : *to;
            *to = make_float4(fmaf(v.x, a, o[i][nt][y]), fmaf(v.y, a, o[i][nt][y + 2]), fmaf(v.z, a, o[i + 1][nt][y]),
                              fmaf(v.w, a, o[i + 1][nt][y + 2]));
            o[i][nt][y] = o[i][nt][y + 2] = o[i + 1][nt][y] = o[i + 1][nt][y + 2] = 0.f;
          }
        }
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (g == 0) own[(8 * nt + 2 * c + y) * kRowF + HD] = m[nt][y];
      __syncwarp();
    };

#pragma unroll 1
    for (; x < u1; x += P::kGroups) {
      const int at = n + x - u0, st = at % P::kStages;
      int ek[P::kSlabs], ev[P::kSlabs];
#pragma unroll
      for (int b = 0; b < P::kSlabs; ++b) ek[b] = kv8_exp((uint8_t)ek_next[b]), ev[b] = kv8_exp((uint8_t)ev_next[b]);
      fetch(x + P::kGroups);
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[st], (at / P::kStages) & 1, A.C.err));
      const int p0 = x * P::kUnit + slab0;
      if (ok && p0 < length) {
        const uint8_t* kt = smem + P::kRing + st * 2 * P::kTile;
        const uint8_t* vt = kt + P::kTile;
        // S^T: positions p0 + 16 b + g and + 8 (y / 2), rows 2c, 2c + 1 (y mod 2)
        float sc[P::kSlabs][NT][4];
#pragma unroll
        for (int b = 0; b < P::kSlabs; ++b) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sc[b][nt][0] = sc[b][nt][1] = sc[b][nt][2] = sc[b][nt][3] = 0.f;
          uint32_t kw[2][kSteps];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = slab0 + 16 * b + 8 * h + g;
            if constexpr (HD == 128) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint4 w = *reinterpret_cast<const uint4*>(kt + row * 128 + (((2 * c + y) ^ (row & 7)) << 4));
                kw[h][4 * y] = w.x, kw[h][4 * y + 1] = w.y, kw[h][4 * y + 2] = w.z, kw[h][4 * y + 3] = w.w;
              }
            } else {
              const uint4 w = *reinterpret_cast<const uint4*>(kt + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
              kw[h][0] = w.x, kw[h][1] = w.y, kw[h][2] = w.z, kw[h][3] = w.w;
            }
          }
#pragma unroll
          for (int y = 0; y < kSteps; ++y) {
            uint32_t a[4];
            codes_to_f16<FMT>(kw[0][y], a[0], a[2]);
            codes_to_f16<FMT>(kw[1][y], a[1], a[3]);
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_acc(sc[b][nt], a, qb[part][nt][y][0], qb[part][nt][y][1]);
          }
          // t = score * log2(e) + ev, masked where a row does not see the position
          const float kf = pow2i(ek[b]), evf = (float)ev[b];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 4; ++y) sc[b][nt][y] = fmaf(sc[b][nt][y], kf * rf[nt][y & 1], evf);
          if (p0 + 16 * b + 15 > min_pos) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                if (p0 + 16 * b + g + 8 * (y >> 1) >= lim[nt][y & 1]) sc[b][nt][y] = -INFINITY;
          }
        }
        float mx[NT][2];
        bool grew = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float v = fmaxf(sc[0][nt][y], sc[0][nt][y + 2]);
#pragma unroll
            for (int b = 1; b < P::kSlabs; ++b) v = fmaxf(v, fmaxf(sc[b][nt][y], sc[b][nt][y + 2]));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
            mx[nt][y] = v = __fsub_ru(v, kWeightTop);
            grew |= v > m[nt][y];
          }
        if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float to = fmaxf(m[nt][y], mx[nt][y]), a = to == -INFINITY ? 1.f : ex2(m[nt][y] - to);
              m[nt][y] = to, l[nt][y] *= a;
#pragma unroll
              for (int i = 0; i < kSteps; ++i) o[i][nt][y] *= a, o[i][nt][y + 2] *= a;
            }
        }
#pragma unroll
        for (int b = 0; b < P::kSlabs; ++b) {
          const float back = pow2i(-ev[b]);
          uint32_t pb[PARTS][NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = ex2(sc[b][nt][y] - (m[nt][y & 1] == -INFINITY ? 0.f : m[nt][y & 1]));
            l[nt][0] = fmaf(w[0] + w[2], back, l[nt][0]), l[nt][1] = fmaf(w[1] + w[3], back, l[nt][1]);
            pb[0][nt][0] = turn(pack_half2(w[0], w[1])), pb[0][nt][1] = turn(pack_half2(w[2], w[3]));
            if constexpr (PARTS == 2) {
              auto rest = [](float v) { return v - __half2float(__float2half_rn(v)); };
              pb[1][nt][0] = turn(pack_half2(rest(w[0]), rest(w[1])));
              pb[1][nt][1] = turn(pack_half2(rest(w[2]), rest(w[3])));
            }
          }
          // O^T += V^T P^T: lane (g, c) reads HD/8 dims from dim g HD/8 of positions 2c, 2c+1, 2c+8, 2c+9
          constexpr int kWords = HD / 32;
          uint32_t vw[4][kWords];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int row = slab0 + 16 * b + 2 * c + (y & 1) + 8 * (y >> 1);
            if constexpr (HD == 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(vt + row * 128 + ((g ^ (row & 7)) << 4));
              vw[y][0] = w.x, vw[y][1] = w.y, vw[y][2] = w.z, vw[y][3] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(vt + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
              vw[y][0] = w.x, vw[y][1] = w.y;
            }
          }
          if (p0 + 16 * b + 16 > length) {  // positions that nothing has been written to: any bits, NaN among them
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (p0 + 16 * b + 2 * c + (y & 1) + 8 * (y >> 1) >= length)
#pragma unroll
                for (int i = 0; i < kWords; ++i) vw[y][i] = 0;
          }
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // bytes 2h, 2h + 1 of the word: dims g and g + 8 of m-tile 2i + h
              const uint32_t sel = h ? 0x7362 : 0x5140;
              uint32_t a[4];
              codes_to_f16<FMT>(prmt(vw[0][i], vw[1][i], sel), a[0], a[1]);
              codes_to_f16<FMT>(prmt(vw[2][i], vw[3][i], sel), a[2], a[3]);
#pragma unroll
              for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_acc(o[2 * i + h][nt], a, pb[part][nt][0], pb[part][nt][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if constexpr (PARTS == 2)
        if (++held % P::kFold == 0) fold(held == P::kFold);
    }
    n += u1 - u0;

    // ---- join the warps ----
    if constexpr (PARTS == 2) fold(held < P::kFold);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float v = l[nt][y];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
        const int r = 8 * nt + 2 * c + y;
        if (g == 0) ml[(warp * P::kRows + r) * 2] = m[nt][y], ml[(warp * P::kRows + r) * 2 + 1] = v;
#pragma unroll
        for (int i = 0; PARTS == 1 && i < kSteps; i += 2)
          *reinterpret_cast<float4*>(own + r * kRowF + g * (HD / 8) + 2 * i) =
              make_float4(o[i][nt][y], o[i][nt][y + 2], o[i + 1][nt][y], o[i + 1][nt][y + 2]);
      }
    asm volatile("bar.sync 1, %0;" ::"n"(P::kWarps * 32) : "memory");
    const Item it = *cur;
    const int rows = min(P::kRows, it.n * A.group - it.mt * P::kRows);
    const bool whole = it.u0 == 0 && it.u1 == it.units;
    const int c0 = (int)(((it.first + 1) * G - 1) / total);
    float* part = A.parts + (long long)(2 * blockIdx.x + (u == lo ? 0 : 1)) * kPart;
    constexpr int kQ = HD / 4;  // float4s of a row
    for (int j = tid; j < rows * kQ; j += P::kWarps * 32) {
      const int r = j / kQ, d = j % kQ * 4;
      float mj = -INFINITY;
#pragma unroll
      for (int w = 0; w < P::kWarps; ++w) mj = fmaxf(mj, ml[(w * P::kRows + r) * 2]);
      float4 acc = make_float4(0, 0, 0, 0);
      float lj = 0.f;
#pragma unroll 4
      for (int w = 0; w < P::kWarps; ++w) {
        const float mw = ml[(w * P::kRows + r) * 2], lw = ml[(w * P::kRows + r) * 2 + 1];
        const float f = join_factor(mw, lw, mj);
        const float4 v = *reinterpret_cast<const float4*>(join + (w * P::kRows + r) * kRowF + d);
        lj = fmaf(f, lw, lj);
        acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y), acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
      }
      if (whole) {
        const int mm = it.mt * P::kRows + r;
        const float inv = lj == 0.f ? 0.f : 1.f / lj;
        acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
        store_value4(A.out, A.dtype,
                     (long long)(it.row0 + mm / A.group) * A.out_stride + (long long)(it.head * A.group + mm % A.group) * HD + d, acc);
      } else {
        *reinterpret_cast<float4*>(part + r * HD + d) = acc;
        if (d == 0) part[16 * HD + r] = mj, part[16 * HD + 16 + r] = lj;
      }
    }
    if (!whole) {
      // the last CTA to finish its part joins them, in CTA order
      __threadfence();
      asm volatile("bar.sync 1, %0;" ::"n"(P::kWarps * 32) : "memory");
      const int c1 = (int)(((it.first + it.units) * G - 1) / total);
      if (tid == 0) {
        __threadfence();
        *shared_word = atomicInc(&A.count[c0], (unsigned)(c1 - c0)) == (unsigned)(c1 - c0);
        __threadfence();
      }
      asm volatile("bar.sync 1, %0;" ::"n"(P::kWarps * 32) : "memory");
      if (*shared_word) {
        const int s0 = 2 * c0 + (total * c0 / G >= it.first - start ? 0 : 1), np = c1 - c0 + 1;
        auto part_of = [&](int y) { return A.parts + (long long)(y == 0 ? s0 : 2 * (c0 + y)) * kPart; };
        // all parts' statistics at once, then each part's weight for each row
        float* stat = join;  // [np][rows][2]
        for (int j = tid; j < np * rows; j += P::kWarps * 32) {
          const float* from = part_of(j / rows) + 16 * HD + j % rows;
          stat[2 * j] = __ldcg(from), stat[2 * j + 1] = __ldcg(from + 16);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(P::kWarps * 32) : "memory");
        for (int j = tid; j < rows * kQ; j += P::kWarps * 32) {
          const int r = j / kQ, d = j % kQ * 4;
          float mj = -INFINITY;
          for (int y = 0; y < np; ++y) mj = fmaxf(mj, stat[2 * (y * rows + r)]);
          float4 acc = make_float4(0, 0, 0, 0);
          float lj = 0.f;
          for (int y0 = 0; y0 < np; y0 += 4) {
            float4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (y0 + y < np) v[y] = __ldcg(reinterpret_cast<const float4*>(part_of(y0 + y) + r * HD + d));
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              if (y0 + y >= np) break;
              const float mw = stat[2 * ((y0 + y) * rows + r)], lw = stat[2 * ((y0 + y) * rows + r) + 1];
              const float f = join_factor(mw, lw, mj);
              lj = fmaf(f, lw, lj);
              acc.x = fmaf(f, v[y].x, acc.x), acc.y = fmaf(f, v[y].y, acc.y);
              acc.z = fmaf(f, v[y].z, acc.z), acc.w = fmaf(f, v[y].w, acc.w);
            }
          }
          const int mm = it.mt * P::kRows + r;
          const float inv = lj == 0.f ? 0.f : 1.f / lj;
          acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
          store_value4(A.out, A.dtype,
                       (long long)(it.row0 + mm / A.group) * A.out_stride + (long long)(it.head * A.group + mm % A.group) * HD + d, acc);
        }
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(P::kWarps * 32) : "memory");  // join and ml may be written again
    u += cost;
  }
}

template <int HD, int FMT, int NT, int PARTS>
struct Split {
  using P = SplitPlan<HD, NT, PARTS>;
  static int smem(int n_seq) { return P::kSeqOff + 16 * n_seq + 8 * (n_seq + 1); }
  static cudaError_t setup() {
    return cudaFuncSetAttribute(attend_split_kernel<HD, FMT, NT, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem(kKv8MaxSeq));
  }
  static cudaError_t launch(const AttendArgs& A, const Kv8Maps& M, cudaStream_t s) {
    attend_split_kernel<HD, FMT, NT, PARTS><<<A.grid, P::kThreads, smem(A.R.n_seq), s>>>(A, M.k, M.v);
    return cudaGetLastError();
  }
};

template <int HD, int FMT>
cudaError_t setup_split() {
  cudaError_t e = Split<HD, FMT, 1, 1>::setup();
  if (e == cudaSuccess) e = Split<HD, FMT, 1, 2>::setup();
  if (e == cudaSuccess) e = Split<HD, FMT, 2, 1>::setup();
  if (e == cudaSuccess) e = Split<HD, FMT, 2, 2>::setup();
  return e;
}

template <int HD, int FMT>
cudaError_t launch_split(const AttendArgs& A, const Kv8Maps& M, cudaStream_t s) {
  const bool two = A.dtype == 0;
  if (A.tile_rows == 8) return two ? Split<HD, FMT, 1, 2>::launch(A, M, s) : Split<HD, FMT, 1, 1>::launch(A, M, s);
  return two ? Split<HD, FMT, 2, 2>::launch(A, M, s) : Split<HD, FMT, 2, 1>::launch(A, M, s);
}

}  // namespace

cudaError_t setup_kv8_attend(int head_dim, int format) {
  cudaError_t e;
  if (head_dim == 128)
    e = format == 0 ? setup_split<128, 0>() : setup_split<128, 1>();
  else
    e = format == 0 ? setup_split<64, 0>() : setup_split<64, 1>();
  return e != cudaSuccess ? e : setup_kv8_prompt(head_dim, format);
}

long long kv8_attend_zeroed(int nsm) { return 256 + ((long long)nsm * 4 + 255) / 256 * 256; }

long long kv8_attend_workspace(int nsm, int head_dim) {  // two parts per CTA
  return kv8_attend_zeroed(nsm) + 2LL * nsm * max(split_part(head_dim), kv8_prompt_part_floats(head_dim)) * 4;
}

cudaError_t launch_kv8_attend(const Kv8Dev& C, const Kv8Rows& R, const Kv8Maps& M, int layer, void* workspace, int nsm,
                              const void* q, long long q_stride, void* out, long long out_stride, int dtype,
                              float scale, cudaStream_t s) {
  const int group = C.heads / C.kv_heads;
  uint8_t* w = static_cast<uint8_t*>(workspace) + 256;
  unsigned* count = reinterpret_cast<unsigned*>(w);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kv8_attend_zeroed(nsm));
  // Few rows or many: the rows that the host knows, max_rows x group.  Measured few / many in us, 32 / 4 heads of 128, for
  // 16, 24, 32, 40, 48, 64, 128 of them.  4 sequences of 1002 positions: bf16 23/31, 23/31, 24/31, 25/31, 27/31, 26/31,
  // 33/33, f32 29/32, 29/33, 31/33, 33/33, 33/33, 36/33, 44/35.  Of 16000: bf16 34/62, 41/63, 41/64, 54/64, 54/64, 65/63,
  // 103/64, f32 50/68, 64/70, 64/70, 87/70, 87/70, 109/72, 178/72.  24 of 8000, where every SM has enough to read: bf16
  // 58/76, 92/76, 93/77, 131/76, 132/76, 169/77, 281/78, f32 92/93, 157/93, 159/95, 227/94, 229/95, 298/95, 504/97.  So
  // long lists cross at 16, where a second row tile reads the caches again, and short ones at 40 to 128; the lengths that
  // would tell them apart are on the device, and 32 lies between.
  if ((long long)R.max_rows * group > 32)
    return launch_kv8_prompt(C, R, M, layer, count, parts, nsm, q, q_stride, out, out_stride, dtype, scale, s);
  AttendArgs A;
  A.C = C, A.R = R, A.q = q, A.out = out, A.q_stride = q_stride, A.out_stride = out_stride;
  A.scale2 = scale * 1.4426950408889634f;
  A.dtype = dtype, A.group = group, A.layer = layer, A.grid = nsm;
  A.tile_rows = R.max_rows * group <= 8 ? 8 : 16;
  A.unit = 64 * (128 / C.head_dim);
  A.count = count, A.parts = parts;
  if (C.head_dim == 128) return C.format == 0 ? launch_split<128, 0>(A, M, s) : launch_split<128, 1>(A, M, s);
  return C.format == 0 ? launch_split<64, 0>(A, M, s) : launch_split<64, 1>(A, M, s);
}

}  // namespace strata
