// Attention of a call's rows over the slots' 8-bit caches.
#include "kv8.cuh"

namespace strata {
namespace {

// ---------------------------------------------------------------------------
// Few rows per slot: the cache is read once, at the memory's rate.
//
// The rows of a sequence that share a kv head (its rows x group query heads)
// are the M side of mma.sync tiles; positions are cut into units of 64.  All
// units of all (sequence, row tile, kv head) items form one list, and each CTA
// (one per SM) takes an equal contiguous part of it, so that one long
// conversation and many short ones fill the GPU alike.  A producer thread
// streams the units' codes by TMA into a ring; each of 8 warps takes 16
// positions of every second unit and keeps its own softmax state, and the
// warps join once per item.  An item cut by a CTA border leaves its parts
// (maximum, sum, unnormalised output) in the workspace; the last CTA to finish
// joins them in CTA order, so the bits do not depend on timing.
//
// Weights: with scores s_j (base 2) and a block's value exponent ev, the state
// follows t_j = s_j + ev: w_j = 2^(t_j - max t), O = sum w_j code_j,
// l = sum w_j 2^-ev, out = O / l.  Whatever the exponents, the largest weight
// that meets a code is 1 (held times 2^14 so that 16-bit weights keep 38 bits
// below it), and no block needs its own accumulator.
// f32 rows: q and the weights enter as two f16 parts (22 bits).  With at most 8
// rows per tile (kPaired) the parts are rows g and g + 8 of one MMA; above
// that two MMAs chain into one accumulator (kChained).
// ---------------------------------------------------------------------------
enum { kSingle = 0, kPaired = 1, kChained = 2 };

constexpr int kUnit = 64;       // positions per ring stage
constexpr int kWarps = 8;       // consumer warps
constexpr int kSplitThreads = (kWarps + 1) * 32;
constexpr float kWeightTop = 14.f;  // weights are scaled by 2^14

template <int HD> struct SplitPlan {
  static constexpr int kTile = kUnit * HD;                  // bytes of one unit's K (or V) codes
  static constexpr int kStages = HD == 128 ? 8 : 16;        // 128 KB in flight
  static constexpr int kJoin = kWarps * 16 * (HD + 4) * 4;  // the warps' O (rows padded by 4 floats)
  static constexpr int kRing = 1024;                        // offsets in dynamic shared memory
  static constexpr int kJoinOff = kRing + kStages * 2 * kTile;
  static constexpr int kMlOff = kJoinOff + kJoin;           // [kWarps][16][2] maximum, sum
  static constexpr int kQloOff = kMlOff + kWarps * 16 * 2 * 4;  // low parts of q (kChained): [HD / 16][32] uint4
  static constexpr int kPreOff = kQloOff + HD / 16 * 32 * 16;
  static constexpr int kPart = 16 * HD + 32;                // floats of a part in the workspace: O, maxima, sums
};

struct AttendArgs {
  Kv8Dev C;
  Kv8Rows R;
  const void* q;
  void* out;
  long long q_stride, out_stride;
  float scale2;      // scale * log2(e)
  int dtype, group, layer, tile_rows, grid;
  float* parts;      // [2 grid][kPart]
  unsigned* count;   // [grid] parts done of the item that starts last in a CTA; back to 0 when joined
};

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Units of row tile mt: positions that its last row sees.
__device__ __forceinline__ int tile_units(const Kv8Seq& s, int group, int tile_rows, int mt) {
  const int last = min(s.n, (tile_rows * (mt + 1) - 1) / group + 1);
  const int seen = s.length - s.n + last;
  return seen <= 0 ? 0 : (seen + kUnit - 1) / kUnit;
}

__device__ __forceinline__ int row_tiles(const Kv8Seq& s, int group, int tile_rows) {
  return (s.n * group + tile_rows - 1) / tile_rows;
}

// Units of all row tiles of one kv head.
__device__ __forceinline__ int head_units(const Kv8Seq& s, int group, int tile_rows) {
  if (!s.held_ok) return 0;
  int sum = 0;
  for (int mt = 0; mt < row_tiles(s, group, tile_rows); ++mt) sum += tile_units(s, group, tile_rows, mt);
  return sum;
}

__device__ __forceinline__ float load_value(const void* p, int dtype, long long i) {
  if (dtype == 0) return static_cast<const float*>(p)[i];
  if (dtype == 1) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Four neighbouring values (the address is a multiple of four values).
__device__ __forceinline__ float4 load_value4(const void* p, int dtype, long long i) {
  if (dtype == 0) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  if (dtype == 1) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
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

// Weight of a part with maximum mw and sum lw under the joint maximum m: 0 for a
// part that saw nothing (a row of NaN has no maximum but a NaN sum, and stays NaN).
__device__ __forceinline__ float join_factor(float mw, float lw, float m) {
  return mw == -INFINITY && lw == 0.f ? 0.f : ex2(mw - m);
}

// A CTA's next item: the part [u0, u1) of its units, positions counted from the item's first unit.
struct Item {
  Kv8Seq s;
  int seq, head, mt;
  int u0, u1, units;     // within the item
  long long first;       // the item's first unit in the whole list
};

template <int HD>
__device__ __forceinline__ Item next_item(const AttendArgs& A, const long long* pre, long long u, long long end,
                                          int seq) {
  Item it;
  while (pre[seq + 1] <= u) ++seq;
  it.seq = seq;
  it.s = kv8_seq(A.R, A.C, seq);
  long long r = u - pre[seq];
  const int per_head = head_units(it.s, A.group, A.tile_rows);
  it.head = (int)(r / per_head);
  r -= (long long)it.head * per_head;
  it.mt = 0;
  it.units = tile_units(it.s, A.group, A.tile_rows, 0);
  while (r >= it.units) {
    r -= it.units;
    it.units = tile_units(it.s, A.group, A.tile_rows, ++it.mt);
  }
  it.u0 = (int)r;
  it.u1 = (int)min((long long)it.units, r + (end - u));
  it.first = u - r;
  return it;
}

template <int HD, int FMT, int MODE>
__global__ void __launch_bounds__(kSplitThreads, 1)
    attend_split_kernel(AttendArgs A, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using P = SplitPlan<HD>;
  constexpr int kSteps = HD / 16;   // k-steps of q.K, and half the n-tiles of P.V
  constexpr int kNt = HD / 8;       // n-tiles of P.V
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + P::kStages;
  int* shared_word = reinterpret_cast<int*>(empty + P::kStages);
  long long* warp_sums = reinterpret_cast<long long*>(smem + 512);
  float* join = reinterpret_cast<float*>(smem + P::kJoinOff);
  float* ml = reinterpret_cast<float*>(smem + P::kMlOff);
  uint4* qlo = reinterpret_cast<uint4*>(smem + P::kQloOff);
  long long* pre = reinterpret_cast<long long*>(smem + P::kPreOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;

  if (tid == 0) {
    for (int i = 0; i < P::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps / 2);
    }
    fence_mbar_init();
  }
  // units before each sequence: a contiguous share per thread, joined by a scan
  const int n_seq = A.R.n_seq;
  {
    constexpr int kScan = kWarps * 32;
    const int share = (n_seq + kScan - 1) / kScan;
    long long sum = 0;
    if (tid < kScan) {
      for (int i = tid * share; i < min(n_seq, (tid + 1) * share); ++i) {
        const Kv8Seq s = kv8_seq(A.R, A.C, i);
        const int u = head_units(s, A.group, A.tile_rows);
        sum += (long long)u * A.C.kv_heads;
        pre[i + 1] = sum;
        if (!s.held_ok && blockIdx.x == 0) atomicOr(A.C.err, kErrIndex);
      }
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31 && warp < kWarps) warp_sums[warp] = inc;
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
    for (int j = tid; j < blind * w4; j += kSplitThreads)
      store_value4(A.out, A.dtype, (long long)(s.row0 + j / w4) * A.out_stride + j % w4 * 4, make_float4(0, 0, 0, 0));
  }

  const long long total = pre[n_seq];
  const int G = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= G) return;
  const long long lo = total * blockIdx.x / G, hi = total * (blockIdx.x + 1) / G;
  int seq0 = 0;
  {
    int a = 0, b = n_seq;  // the sequence that holds unit lo: pre[seq0] <= lo < pre[seq0 + 1]
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (pre[m] <= lo)
        a = m;
      else
        b = m;
    }
    seq0 = a;
  }

  if (warp == kWarps) {
    // ---- producer ----
    if (lane != 0) return;
    int n = 0, seq = seq0;
    bool ok = true;
    for (long long u = lo; u < hi && ok;) {
      const Item it = next_item<HD>(A, pre, u, hi, seq);
      seq = it.seq;
      const long long row = ((long long)it.s.slot * A.C.kv_heads + it.head) * A.C.max_ctx;
      for (int x = it.u0; x < it.u1; ++x, ++n) {
        const int st = n % P::kStages;
        if (n >= P::kStages && !mbar_wait(&empty[st], (n / P::kStages - 1) & 1, A.C.err)) {
          ok = false;
          break;
        }
        uint8_t* dst = smem + P::kRing + st * 2 * P::kTile;
        mbar_arrive_expect_tx(&full[st], 2 * P::kTile);
        tma_3d(dst, &kmap, 0, (int)(row + (long long)x * kUnit), A.layer, &full[st]);
        tma_3d(dst + P::kTile, &vmap, 0, (int)(row + (long long)x * kUnit), A.layer, &full[st]);
      }
      u += it.u1 - it.u0;
    }
    if (!ok)  // the copies in flight land before this thread leaves
      for (int i = max(0, n - P::kStages); i < n; ++i)
        mbar_wait(&full[i % P::kStages], (i / P::kStages) & 1, A.C.err);
    return;
  }

  // ---- consumers ----
  const int half = warp >> 2, slab = (warp & 3) * 16;
  int n = 0, seq = seq0;
  bool ok = true;
  for (long long u = lo; u < hi;) {
    const Item it = next_item<HD>(A, pre, u, hi, seq);
    seq = it.seq;
    const Kv8Seq& s = it.s;
    const int rows = min(A.tile_rows, s.n * A.group - it.mt * A.tile_rows);  // of this tile
    const int p_first = s.length - s.n;                                     // position of the sequence's first row

    // q fragments: lane (g, c) of k-step x holds dims c HD/4 + 4x .. + 3 of rows g and g + 8
    uint32_t qa[kSteps][4];
    float rf[2];
    int lim[2];  // positions that rows g, g + 8 see
    {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int rr = MODE == kPaired ? g : g + 8 * r;
        const bool on = rr < rows && !(MODE == kPaired && r);
        const int m = it.mt * A.tile_rows + rr, tok = m / A.group;
        lim[r] = rr < rows ? max(0, p_first + tok + 1) : 0;
        float f[HD / 4];
#pragma unroll
        for (int d = 0; d < HD / 4; ++d) f[d] = 0.f;
        if (on) {
          const long long at =
              (long long)(s.row0 + tok) * A.q_stride + (long long)(it.head * A.group + m % A.group) * HD + c * (HD / 4);
#pragma unroll
          for (int d = 0; d < HD / 4; d += 4) {
            const float4 v = load_value4(A.q, A.dtype, at + d);
            f[d] = v.x, f[d + 1] = v.y, f[d + 2] = v.z, f[d + 3] = v.w;
          }
        }
        // a power of two per row brings its largest element to [1, 2)
        unsigned top = 0;
#pragma unroll
        for (int d = 0; d < HD / 4; ++d) top = max(top, __float_as_uint(f[d]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const int e = top == 0 ? 0 : min(max((int)(top >> 23) - 127, -120), 120);
        const float down = pow2i(-e);
        if (!(MODE == kPaired && r)) rf[r] = pow2i(e);
#pragma unroll
        for (int x = 0; x < kSteps; ++x) {
          float h[4], l[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            h[d] = f[4 * x + d] * down;
            l[d] = h[d] - __half2float(__float2half_rn(h[d]));
          }
          if (!(MODE == kPaired && r)) {
            qa[x][r] = pack_half2(h[0], h[1]);
            qa[x][2 + r] = pack_half2(h[2], h[3]);
            if constexpr (MODE == kPaired) {
              qa[x][1] = pack_half2(l[0], l[1]);
              qa[x][3] = pack_half2(l[2], l[3]);
            }
            if constexpr (MODE == kChained) {  // every warp holds the same low parts: warp 0 keeps them
              if (warp == 0) {
                uint32_t* w = reinterpret_cast<uint32_t*>(&qlo[x * 32 + lane]);
                w[r] = pack_half2(l[0], l[1]);
                w[2 + r] = pack_half2(l[2], l[3]);
              }
            }
          }
        }
      }
      if constexpr (MODE == kPaired) rf[1] = rf[0];
      if constexpr (MODE == kChained) asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    }
    const int min_pos = p_first + it.mt * A.tile_rows / A.group;  // position of the tile's first row

    float o[kNt][4];
#pragma unroll
    for (int i = 0; i < kNt; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    const long long line = (long long)s.slot * A.C.kv_heads + it.head;
    const uint8_t* keb = A.C.k_exp + line * A.C.n_blocks;
    const uint8_t* veb = A.C.v_exp + line * A.C.n_blocks;
    // this warp's units of the part: every second one of the CTA's list
    int x = it.u0 + ((n ^ half) & 1);
    auto exps = [&](int unit, int& ek, int& ev) {
      const int p = unit * kUnit + slab;
      ek = ev = 0;
      if (unit < it.u1 && p < s.length) {
        ek = keb[p >> A.C.block_log2];
        ev = veb[p >> A.C.block_log2];
      }
    };
    int ek_next, ev_next;
    exps(x, ek_next, ev_next);
    for (; x < it.u1; x += 2) {
      const int at = n + x - it.u0, st = at % P::kStages;
      const int ek = kv8_exp((uint8_t)ek_next), ev = kv8_exp((uint8_t)ev_next);
      exps(x + 2, ek_next, ev_next);
      if (ok) ok = mbar_wait(&full[st], (at / P::kStages) & 1, A.C.err);
      const int p0 = x * kUnit + slab;
      if (ok && p0 < s.length) {
        const uint8_t* kt = smem + P::kRing + st * 2 * P::kTile;
        const uint8_t* vt = kt + P::kTile;
        // scores of 16 positions: n-tile j, column g is position p0 + 8j + g
        float sc[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t kw[kSteps];
          const int row = slab + 8 * j + g;
          if constexpr (HD == 128) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 w = *reinterpret_cast<const uint4*>(kt + row * 128 + (((2 * c + h) ^ (row & 7)) << 4));
              kw[4 * h] = w.x, kw[4 * h + 1] = w.y, kw[4 * h + 2] = w.z, kw[4 * h + 3] = w.w;
            }
          } else {
            const uint4 w = *reinterpret_cast<const uint4*>(kt + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
            kw[0] = w.x, kw[1] = w.y, kw[2] = w.z, kw[3] = w.w;
          }
          sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
          for (int y = 0; y < kSteps; ++y) {
            uint32_t b0, b1;
            codes_to_f16<FMT>(kw[y], b0, b1);
            mma_acc(sc[j], qa[y], b0, b1);
            if constexpr (MODE == kChained) {
              const uint4 w = qlo[y * 32 + lane];
              const uint32_t ql[4] = {w.x, w.y, w.z, w.w};
              mma_acc(sc[j], ql, b0, b1);
            }
          }
        }
        // t = score * log2(e) + ev, masked where a row does not see the position
        const float kf = A.scale2 * pow2i(ek), evf = (float)ev;
        float t[2][4];
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (MODE == kPaired) {
            t[j][0] = fmaf(sc[j][0] + sc[j][2], kf * rf[0], evf);
            t[j][1] = fmaf(sc[j][1] + sc[j][3], kf * rf[0], evf);
          } else {
            t[j][0] = fmaf(sc[j][0], kf * rf[0], evf);
            t[j][1] = fmaf(sc[j][1], kf * rf[0], evf);
            t[j][2] = fmaf(sc[j][2], kf * rf[1], evf);
            t[j][3] = fmaf(sc[j][3], kf * rf[1], evf);
          }
        }
        if (p0 + 15 > min_pos) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int p = p0 + 8 * j + 2 * c + y;
              if (p >= lim[0]) t[j][y] = -INFINITY;
              if (MODE != kPaired && p >= lim[1]) t[j][2 + y] = -INFINITY;
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mx0 = fmaxf(mx0, fmaxf(t[j][0], t[j][1]));
          if constexpr (MODE != kPaired) mx1 = fmaxf(mx1, fmaxf(t[j][2], t[j][3]));
        }
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, 2));
        if constexpr (MODE != kPaired) {
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, 1));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, 2));
        }
        if (__any_sync(0xFFFFFFFFu, mx0 > m0 || mx1 > m1)) {
          const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
          const float a0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0), a1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
          m0 = n0, m1 = n1, l0 *= a0, l1 *= a1;
#pragma unroll
          for (int i = 0; i < kNt; ++i) {
            o[i][0] *= a0, o[i][1] *= a0;
            o[i][2] *= MODE == kPaired ? a0 : a1, o[i][3] *= MODE == kPaired ? a0 : a1;
          }
        }
        const float z0 = m0 == -INFINITY ? 0.f : kWeightTop - m0, z1 = m1 == -INFINITY ? 0.f : kWeightTop - m1;
        const float back = pow2i(-ev);
        uint32_t pa[4], pl[4];
        {
          float w[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            w[j][0] = ex2(t[j][0] + z0), w[j][1] = ex2(t[j][1] + z0);
            if constexpr (MODE != kPaired) w[j][2] = ex2(t[j][2] + z1), w[j][3] = ex2(t[j][3] + z1);
          }
          l0 = fmaf((w[0][0] + w[0][1]) + (w[1][0] + w[1][1]), back, l0);
          if constexpr (MODE != kPaired) l1 = fmaf((w[0][2] + w[0][3]) + (w[1][2] + w[1][3]), back, l1);
          auto rest = [](float v) { return v - __half2float(__float2half_rn(v)); };
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            pa[2 * j] = pack_half2(w[j][0], w[j][1]);
            if constexpr (MODE == kPaired) {
              pa[2 * j + 1] = pack_half2(rest(w[j][0]), rest(w[j][1]));
            } else {
              pa[2 * j + 1] = pack_half2(w[j][2], w[j][3]);
            }
            if constexpr (MODE == kChained) {
              pl[2 * j] = pack_half2(rest(w[j][0]), rest(w[j][1]));
              pl[2 * j + 1] = pack_half2(rest(w[j][2]), rest(w[j][3]));
            }
          }
        }
        // O += P V: lane (g, c) reads HD/8 dims from dim g HD/8 of positions 2c, 2c+1, 2c+8, 2c+9
        constexpr int kWords = HD / 32;
        uint32_t vw[4][kWords];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int row = slab + 2 * c + (y & 1) + 8 * (y >> 1);
          if constexpr (HD == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(vt + row * 128 + ((g ^ (row & 7)) << 4));
            vw[y][0] = w.x, vw[y][1] = w.y, vw[y][2] = w.z, vw[y][3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(vt + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
            vw[y][0] = w.x, vw[y][1] = w.y;
          }
        }
        if (p0 + 16 > s.length) {  // positions that nothing has been written to: any bits, NaN among them
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (p0 + 2 * c + (y & 1) + 8 * (y >> 1) >= s.length)
#pragma unroll
              for (int i = 0; i < kWords; ++i) vw[y][i] = 0;
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // bytes 2h, 2h + 1 of the word: n-tiles 4i + 2h, 4i + 2h + 1
            const uint32_t sel = h ? 0x7362 : 0x5140;
            uint32_t b0a, b0b, b1a, b1b;
            codes_to_f16<FMT>(prmt(vw[0][i], vw[1][i], sel), b0a, b0b);
            codes_to_f16<FMT>(prmt(vw[2][i], vw[3][i], sel), b1a, b1b);
            mma_acc(o[4 * i + 2 * h], pa, b0a, b1a);
            mma_acc(o[4 * i + 2 * h + 1], pa, b0b, b1b);
            if constexpr (MODE == kChained) {
              mma_acc(o[4 * i + 2 * h], pl, b0a, b1a);
              mma_acc(o[4 * i + 2 * h + 1], pl, b0b, b1b);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    n += it.u1 - it.u0;

    // ---- join the warps ----
    l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 1);
    l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 2);
    l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 1);
    l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 2);
    constexpr int kRowF = HD + 4;
    float* mine = join + warp * 16 * kRowF;
    if (c == 0) {
      ml[(warp * 16 + g) * 2] = m0, ml[(warp * 16 + g) * 2 + 1] = l0;
      ml[(warp * 16 + g + 8) * 2] = MODE == kPaired ? -INFINITY : m1, ml[(warp * 16 + g + 8) * 2 + 1] = MODE == kPaired ? 0.f : l1;
    }
    // o[i][0], o[i][1] are dims 2c kNt + i and (2c + 1) kNt + i
#pragma unroll
    for (int i = 0; i < kNt; i += 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4 a = make_float4(o[i][h], o[i + 1][h], o[i + 2][h], o[i + 3][h]);
        const float4 b = make_float4(o[i][2 + h], o[i + 1][2 + h], o[i + 2][2 + h], o[i + 3][2 + h]);
        const int d = (2 * c + h) * kNt + i;
        if constexpr (MODE == kPaired) {
          a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        } else {
          *reinterpret_cast<float4*>(mine + (g + 8) * kRowF + d) = b;
        }
        *reinterpret_cast<float4*>(mine + g * kRowF + d) = a;
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    const bool whole = it.u0 == 0 && it.u1 == it.units;
    const int c0 = (int)(((it.first + 1) * G - 1) / total);
    float* part = A.parts + (long long)(2 * blockIdx.x + (u == lo ? 0 : 1)) * P::kPart;
    constexpr int kQ = HD / 4;  // float4s of a row
    for (int j = tid; j < rows * kQ; j += kWarps * 32) {
      const int r = j / kQ, d = j % kQ * 4;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[(w * 16 + r) * 2]);
      float4 acc = make_float4(0, 0, 0, 0);
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = ml[(w * 16 + r) * 2], lw = ml[(w * 16 + r) * 2 + 1];
        const float f = join_factor(mw, lw, m);
        const float4 v = *reinterpret_cast<const float4*>(join + (w * 16 + r) * kRowF + d);
        l = fmaf(f, lw, l);
        acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y), acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
      }
      if (whole) {
        const int mm = it.mt * A.tile_rows + r;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
        store_value4(A.out, A.dtype,
                     (long long)(s.row0 + mm / A.group) * A.out_stride + (long long)(it.head * A.group + mm % A.group) * HD + d, acc);
      } else {
        *reinterpret_cast<float4*>(part + r * HD + d) = acc;
        if (d == 0) part[16 * HD + r] = m, part[16 * HD + 16 + r] = l;
      }
    }
    if (!whole) {
      // the last CTA to finish its part joins them, in CTA order
      __threadfence();
      asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
      const int c1 = (int)(((it.first + it.units) * G - 1) / total);
      if (tid == 0) {
        __threadfence();
        *shared_word = atomicInc(&A.count[c0], (unsigned)(c1 - c0)) == (unsigned)(c1 - c0);
        __threadfence();
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
      if (*shared_word) {
        const int s0 = 2 * c0 + (total * c0 / G == it.first ? 0 : 1);
        for (int j = tid; j < rows * kQ; j += kWarps * 32) {
          const int r = j / kQ, d = j % kQ * 4;
          float m = -INFINITY;
          for (int y = c0; y <= c1; ++y)
            m = fmaxf(m, __ldcg(A.parts + (long long)(y == c0 ? s0 : 2 * y) * P::kPart + 16 * HD + r));
          float4 acc = make_float4(0, 0, 0, 0);
          float l = 0.f;
#pragma unroll 4
          for (int y = c0; y <= c1; ++y) {
            const float* from = A.parts + (long long)(y == c0 ? s0 : 2 * y) * P::kPart;
            const float mw = __ldcg(from + 16 * HD + r), lw = __ldcg(from + 16 * HD + 16 + r);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(from + r * HD + d));
            const float f = join_factor(mw, lw, m);
            l = fmaf(f, lw, l);
            acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y), acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
          }
          const int mm = it.mt * A.tile_rows + r;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
          store_value4(A.out, A.dtype,
                       (long long)(s.row0 + mm / A.group) * A.out_stride + (long long)(it.head * A.group + mm % A.group) * HD + d, acc);
        }
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");  // join, ml and qlo may be written again
    u += it.u1 - it.u0;
  }
}

template <int HD>
int split_smem(int n_seq) {
  return 1024 + SplitPlan<HD>::kPreOff + 8 * (n_seq + 1);
}

template <int HD, int FMT, int MODE>
cudaError_t launch_split(const AttendArgs& A, const Kv8Maps& M, cudaStream_t s) {
  attend_split_kernel<HD, FMT, MODE><<<A.grid, kSplitThreads, split_smem<HD>(A.R.n_seq), s>>>(A, M.k, M.v);
  return cudaGetLastError();
}

template <int HD, int FMT>
cudaError_t setup_split() {
  const int smem = split_smem<HD>(kKv8MaxSeq);
  cudaError_t e = cudaSuccess;
  auto set = [&](auto* fn) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  set(attend_split_kernel<HD, FMT, kSingle>);
  set(attend_split_kernel<HD, FMT, kPaired>);
  set(attend_split_kernel<HD, FMT, kChained>);
  return e;
}

template <int HD, int FMT>
cudaError_t launch_split_mode(const AttendArgs& A, const Kv8Maps& M, int mode, cudaStream_t s) {
  if (mode == kSingle) return launch_split<HD, FMT, kSingle>(A, M, s);
  if (mode == kPaired) return launch_split<HD, FMT, kPaired>(A, M, s);
  return launch_split<HD, FMT, kChained>(A, M, s);
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

// After the error word's 256 bytes: a counter per CTA, then two parts per CTA.
long long kv8_attend_workspace(int nsm, int head_dim) {
  const int split = head_dim == 128 ? SplitPlan<128>::kPart : SplitPlan<64>::kPart;
  const int part = max(split, kv8_prompt_part_floats(head_dim));
  return 256 + ((long long)nsm * 4 + 255) / 256 * 256 + 2LL * nsm * part * 4;
}

cudaError_t launch_kv8_attend(const Kv8Dev& C, const Kv8Rows& R, const Kv8Maps& M, int layer, void* workspace, int nsm,
                              const void* q, long long q_stride, void* out, long long out_stride, int dtype,
                              float scale, cudaStream_t s) {
  const int group = C.heads / C.kv_heads;
  uint8_t* w = static_cast<uint8_t*>(workspace) + 256;
  unsigned* count = reinterpret_cast<unsigned*>(w);
  float* parts = reinterpret_cast<float*>(w + ((size_t)nsm * 4 + 255) / 256 * 256);
  if ((long long)R.max_rows * group > 32)
    return launch_kv8_prompt(C, R, M, layer, count, parts, nsm, q, q_stride, out, out_stride, dtype, scale, s);
  AttendArgs A;
  A.C = C, A.R = R, A.q = q, A.out = out, A.q_stride = q_stride, A.out_stride = out_stride;
  A.scale2 = scale * 1.4426950408889634f;
  A.dtype = dtype, A.group = group, A.layer = layer, A.grid = nsm;
  const int mode = dtype != 0 ? kSingle : R.max_rows * group <= 8 ? kPaired : kChained;
  A.tile_rows = mode == kPaired ? 8 : 16;
  A.count = count, A.parts = parts;
  if (C.head_dim == 128)
    return C.format == 0 ? launch_split_mode<128, 0>(A, M, mode, s) : launch_split_mode<128, 1>(A, M, mode, s);
  return C.format == 0 ? launch_split_mode<64, 0>(A, M, mode, s) : launch_split_mode<64, 1>(A, M, mode, s);
}

}  // namespace strata
