// C ABI and kernels of the tokens sorted by expert and back: the router's
// choice, the order of the entries, rows to the experts' order, rows back with
// weights, and the gradient of that.
#include <cooperative_groups.h>

#include <cmath>
#include <new>

#include "handle.h"
#include "kv8.cuh"
#include "strata_window.h"

using namespace strata;
namespace cg = cooperative_groups;

struct strata_sort {
  strata_sort_desc desc;
  int device = 0, nsm = 0;
};

namespace {

constexpr int kSortMaxExperts = 1024, kSortMaxK = 16;
constexpr unsigned kAll = 0xFFFFFFFFu;

// --- the router's choice ---------------------------------------------------------

// A float's order as an unsigned's; 0 for what is never chosen (-inf, NaN).
__device__ __forceinline__ unsigned logit_key(float f) {
  if (!(f > -INFINITY)) return 0;
  const unsigned b = __float_as_uint(f + 0.f);  // -0 is +0: they are equal
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(unsigned k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// A warp owns a row: expert i * 32 + lane in register i of the lane, as a key.  The largest key of the warp is one
// redux, its lowest holder another, so equal logits go to the lower expert.  8191 rows of 128 logits, 8 of each: 8 us.
template <int NI>
__global__ void __launch_bounds__(128) route_kernel(const float* logits, long long stride, const float* bias, int T, int E,
                                                    int k, int renorm, int* idx, float* w) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= T) return;
  const float* src = logits + (long long)row * stride;
  unsigned key[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = i * 32 + lane;
    float f = e < E ? src[e] + (bias ? bias[e] : 0.f) : -INFINITY;
    if (f > 3.402823466e38f) f = 3.402823466e38f;
    key[i] = logit_key(f);
  }
  unsigned best = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) best = max(best, key[i]);
  const unsigned top = __reduce_max_sync(kAll, best);
  const float most = key_logit(top);
  float total = 0.f;
  if (!renorm) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (key[i]) total += expf(key_logit(key[i]) - most);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  }
  int mine = -1;
  float part = 0.f;  // lane j holds the j-th choice
  for (int j = 0; j < k; ++j) {
    best = 0;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (key[i] > best) best = key[i], at = i * 32 + lane;
    const unsigned m = __reduce_max_sync(kAll, best);
    if (m == 0) break;  // nothing is left
    const int e = __reduce_min_sync(kAll, best == m ? at : 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (e == i * 32 + lane) key[i] = 0;
    if (lane == j) mine = e, part = expf(key_logit(m) - most);
  }
  if (renorm) {
    total = part;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  }
  if (lane < k) {
    idx[(long long)row * k + lane] = mine;
    w[(long long)row * k + lane] = mine < 0 ? 0.f : part / total;
  }
}

// --- the order -------------------------------------------------------------------

// A stable counting sort in one launch of one cluster.  The entries are cut into equal stretches, one for each warp of
// the cluster in turn, so that an expert's entries of an earlier warp come first: a warp counts its stretch (lanes with
// the same expert find each other by a ballot for each bit of it, the first of them adds), the CTAs exchange their totals through
// distributed shared memory, and each warp walks its stretch again with running positions.  No atomics: the same order
// always.  Latency bound (a prompt's 65528 entries are 256 a warp: 14.7 us, 20.5 us with match in place of the ballots; 512
// entries in one CTA 4.3 us).
constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32, kPlanCluster = 8;
constexpr int kHeld = 8;  // entries of a lane loaded at once

// The lanes that have this lane's value, of `bits` bits.
__device__ __forceinline__ unsigned same_lanes(int v, int bits) {
  unsigned same = kAll;
  for (int b = 0; b < bits; ++b) {
    const unsigned set = __ballot_sync(kAll, v >> b & 1);
    same &= v >> b & 1 ? set : ~set;
  }
  return same;
}

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const int* __restrict__ idx, int n, int E, int* counts, int* offsets,
                                                               int* entries, int* place) {
  extern __shared__ int sm[];
  int* run = sm;                        // [kPlanWarps][E] a warp's counts, then its running positions
  int* total = sm + kPlanWarps * E;     // [E] the CTA's counts, read by the others
  __shared__ int scan[kPlanWarps];
  cg::cluster_group cl = cg::this_cluster();
  const int ctas = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * E; i += kPlanThreads) run[i] = 0;
  const int warps = ctas * kPlanWarps;
  const int stretch = ((n + warps - 1) / warps + 31) & ~31;
  const long long lo = (long long)(rank * kPlanWarps + warp) * stretch;
  const int begin = (int)(lo < n ? lo : n), end = (int)(lo + stretch < n ? lo + stretch : n);
  int* mine = run + warp * E;
  __syncthreads();
  // kHeld loads at a time; of a stretch of at most that many the values stay for the second walk
  int held[kHeld];
  unsigned same[kHeld];
  const int bits = 32 - __clz(E);
  auto fetch = [&](int base) {
#pragma unroll
    for (int y = 0; y < kHeld; ++y) {
      const int i = base + y * 32 + lane;
      held[y] = i < end ? idx[i] : -1;
      if (held[y] < 0 || held[y] >= E) held[y] = E;
    }
  };
  for (int base = begin; base < end; base += 32 * kHeld) {
    fetch(base);
#pragma unroll
    for (int y = 0; y < kHeld; ++y) {
      if (base + y * 32 >= end) break;
      same[y] = same_lanes(held[y], bits);
      if (held[y] < E && lane == __ffs(same[y]) - 1) mine[held[y]] += __popc(same[y]);
      __syncwarp();
    }
  }
  __syncthreads();
  const int e = threadIdx.x;  // E <= 1024
  if (e < E) {
    int s = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = run[w * E + e];
      run[w * E + e] = s;
      s += c;
    }
    total[e] = s;
  }
  cl.sync();
  int before = 0, all = 0;
  if (e < E) {
    for (int c = 0; c < ctas; ++c) {
      const int v = *cl.map_shared_rank(total + e, c);
      if (c < rank) before += v;
      all += v;
    }
  }
  int upto = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kAll, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  int add = lane < warp ? scan[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) add += __shfl_xor_sync(kAll, add, o);
  const int first = upto - all + add;  // entries of lower experts
  if (e < E) {
    for (int w = 0; w < kPlanWarps; ++w) run[w * E + e] += first + before;
    if (rank == 0) {
      if (counts) counts[e] = all;
      offsets[e] = first;
      if (e == E - 1) offsets[E] = first + all;
    }
  }
  int live = 0;  // entries that are an expert's
  for (int w = 0; w < kPlanWarps; ++w) live += scan[w];
  cl.sync();  // the runs are written, and no CTA leaves while its totals are read
  for (int base = begin; base < end; base += 32 * kHeld) {
    const bool again = end - begin > 32 * kHeld;
    if (again) fetch(base);
#pragma unroll
    for (int y = 0; y < kHeld; ++y) {
      if (base + y * 32 >= end) break;
      const int i = base + y * 32 + lane, x = held[y];
      const unsigned us = again ? same_lanes(x, bits) : same[y];
      int at = -1;
      if (x < E) at = mine[x] + __popc(us & ((1u << lane) - 1));
      __syncwarp();
      if (x < E && lane == __ffs(us) - 1) mine[x] += __popc(us);
      __syncwarp();
      if (i < end) {
        place[i] = at;
        if (x < E) entries[at] = i;
      }
    }
  }
  for (long long i = (long long)live + rank * kPlanThreads + threadIdx.x; i < n; i += (long long)ctas * kPlanThreads)
    entries[i] = -1;
}

// --- rows to the experts' order and back -----------------------------------------

struct MoveArgs {
  const int* place;
  const float* w;
  const uint4 *a, *b;   // gather: x; combine: z, base; backward: dy, z
  uint4* out;           // xs; y; dz
  float* dw;
  long long as, bs, os; // row strides in 16-byte pieces
  int T, k, pieces;     // 16-byte pieces of a row
  long long n;          // T k
};

__device__ __forceinline__ bool placed(int p, long long n) { return p >= 0 && p < n; }

// A thread moves one piece of a row to its k places: x is read once and each copy written once.  HBM bound: 8191 bf16 rows of 2048
// to 8 places each 47 us, 94% of the measured rate.
__global__ void __launch_bounds__(256) gather_kernel(MoveArgs A) {
  const long long items = (long long)A.T * A.pieces;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < items; i += (long long)gridDim.x * 256) {
    const long long t = i / A.pieces;
    const int c = (int)(i - t * A.pieces);
    const uint4 v = A.a[t * A.as + c];
    const int* p = A.place + t * A.k;
    for (int j = 0; j < A.k; ++j)
      if (placed(p[j], A.n)) A.out[p[j] * A.os + c] = v;
  }
}

// A thread sums one piece of a row over its k places, in the row's order, four loads at a time.  HBM bound: the same rows back onto a
// base 54 us, 89% of the measured rate.
template <typename T>
__global__ void __launch_bounds__(256) combine_kernel(MoveArgs A) {
  constexpr int E = Val<T>::kPer;
  const long long items = (long long)A.T * A.pieces;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < items; i += (long long)gridDim.x * 256) {
    const long long t = i / A.pieces;
    const int c = (int)(i - t * A.pieces);
    float s[E];
#pragma unroll
    for (int u = 0; u < E; ++u) s[u] = 0.f;
    if (A.b) Val<T>::unpack(A.b[t * A.bs + c], s);
    const int* p = A.place + t * A.k;
    for (int j0 = 0; j0 < A.k; j0 += 4) {
      uint4 v[4];
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = j0 + j < A.k ? p[j0 + j] : -1;
        const bool ok = placed(at, A.n);
        v[j] = ok ? A.a[at * A.as + c] : make_uint4(0, 0, 0, 0);
        w[j] = !ok ? 0.f : A.w ? A.w[t * A.k + j0 + j] : 1.f;
        if (!ok) w[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j0 + j >= A.k) break;
        float f[E];
        Val<T>::unpack(v[j], f);
#pragma unroll
        for (int u = 0; u < E; ++u) s[u] = fmaf(w[j], f[u], s[u]);
      }
    }
    A.out[t * A.os + c] = Val<T>::pack(s);
  }
}

// A CTA takes a row: a thread its pieces of dy against the k places' rows of z; the k products are summed over the CTA
// in a fixed order.  HBM bound: 2047 f32 rows of 4096 at 8 places 97 us, 87% of the measured rate.
constexpr int kBackThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kBackThreads) combine_backward_kernel(MoveArgs A) {
  constexpr int E = Val<T>::kPer;
  __shared__ float part[kBackThreads / 32][kSortMaxK];
  const long long t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int* p = A.place + t * A.k;
  float dot[kSortMaxK];
#pragma unroll
  for (int j = 0; j < kSortMaxK; ++j) dot[j] = 0.f;
  for (int c = threadIdx.x; c < A.pieces; c += kBackThreads) {
    float d[E];
    Val<T>::unpack(A.a[t * A.as + c], d);
#pragma unroll
    for (int j = 0; j < kSortMaxK; ++j) {
      if (j >= A.k) break;
      const int at = p[j];
      if (!placed(at, A.n)) continue;
      if (A.dw) {
        float f[E];
        Val<T>::unpack(A.b[at * A.bs + c], f);
#pragma unroll
        for (int u = 0; u < E; ++u) dot[j] = fmaf(d[u], f[u], dot[j]);
      }
      if (A.out) {
        const float w = A.w ? A.w[t * A.k + j] : 1.f;
        float f[E];
#pragma unroll
        for (int u = 0; u < E; ++u) f[u] = w * d[u];
        A.out[at * A.os + c] = Val<T>::pack(f);
      }
    }
  }
  if (!A.dw) return;
#pragma unroll
  for (int j = 0; j < kSortMaxK; ++j) {
    if (j >= A.k) break;
    float s = dot[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (lane == 0) part[warp][j] = s;
  }
  __syncthreads();
  if ((int)threadIdx.x < A.k) {
    float s = 0.f;
    for (int w = 0; w < kBackThreads / 32; ++w) s += part[w][threadIdx.x];
    A.dw[t * A.k + threadIdx.x] = s;
  }
}

// --- checks ----------------------------------------------------------------------

bool rows_ok(const void* p, long long stride, int width, int size) {
  return p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride >= width && stride <= (1LL << 40) &&
         (stride * size) % 16 == 0;
}
bool words_ok(const void* p) { return p && reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// What gather, combine and its gradient check alike.
strata_status check_move(const strata_sort* h, const int32_t* place, int32_t dtype, int32_t T, int32_t width, int* size) {
  if (!h || T < 0 || width < 1 || dtype < STRATA_F32 || dtype > STRATA_BF16) return STRATA_EINVAL;
  *size = dtype == STRATA_F32 ? 4 : 2;
  if ((long long)width * *size % 16 != 0) return STRATA_EINVAL;
  if ((long long)T * h->desc.top_k > (1 << 28) || width > (1 << 24)) return STRATA_EUNSUPPORTED;
  if (T > 0 && !words_ok(place)) return STRATA_EINVAL;
  return STRATA_OK;
}

MoveArgs move_args(const strata_sort* h, const int32_t* place, int T, int width, int size) {
  MoveArgs A{};
  A.place = place, A.T = T, A.k = h->desc.top_k, A.pieces = width * size / 16, A.n = (long long)T * h->desc.top_k;
  return A;
}

strata_status launched() {
  if (cudaGetLastError() != cudaSuccess) return STRATA_ECUDA;
  return STRATA_OK;
}

// CTAs of 256 threads for `items` of them: at most what the SMs hold at once, eight each.
unsigned move_grid(const strata_sort* h, long long items) {
  const long long want = (items + 255) / 256, most = 8LL * h->nsm;
  return (unsigned)(want < most ? want : most);
}

}  // namespace

extern "C" {

strata_status strata_sort_create(const strata_sort_desc* d, strata_sort** out) {
  if (!out) return STRATA_EINVAL;
  *out = nullptr;
  if (!d || d->n_experts < 1 || d->top_k < 1 || d->top_k > d->n_experts || (d->renorm_topk != 0 && d->renorm_topk != 1))
    return STRATA_EINVAL;
  if (d->n_experts > kSortMaxExperts || d->top_k > kSortMaxK) return STRATA_EUNSUPPORTED;
  if (fault_is("alloc")) return STRATA_ENOMEM;
  strata_sort* h = new (std::nothrow) strata_sort();
  if (!h) return STRATA_ENOMEM;
  h->desc = *d;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->nsm, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
      cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (kPlanWarps + 1) * kSortMaxExperts * 4) != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return STRATA_ECUDA;
  }
  *out = h;
  return STRATA_OK;
}

strata_status strata_sort_route(strata_sort* h, const float* logits, int64_t stride, const float* bias, int32_t T,
                                int32_t* topk_idx, float* topk_w, void* cuda_stream) {
  if (!h || T < 0) return STRATA_EINVAL;
  if (T == 0) return STRATA_OK;
  const int E = h->desc.n_experts, k = h->desc.top_k;
  if (!words_ok(logits) || stride < E || stride > (1LL << 40) || !words_ok(topk_idx) || !words_ok(topk_w) ||
      (bias && !words_ok(bias)))
    return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const unsigned grid = (unsigned)(((long long)T + 3) / 4);
  const int r = h->desc.renorm_topk;
  if (E <= 128)
    route_kernel<4><<<grid, 128, 0, s>>>(logits, stride, bias, T, E, k, r, topk_idx, topk_w);
  else if (E <= 256)
    route_kernel<8><<<grid, 128, 0, s>>>(logits, stride, bias, T, E, k, r, topk_idx, topk_w);
  else
    route_kernel<32><<<grid, 128, 0, s>>>(logits, stride, bias, T, E, k, r, topk_idx, topk_w);
  return launched();
}

strata_status strata_sort_plan(strata_sort* h, const int32_t* topk_idx, int32_t T, const strata_sort_order* o,
                               void* cuda_stream) {
  if (!h || !o || T < 0) return STRATA_EINVAL;
  const int E = h->desc.n_experts;
  const long long n = (long long)T * h->desc.top_k;
  if (n > (1 << 28)) return STRATA_EUNSUPPORTED;
  if (!words_ok(o->offsets) || (o->counts && !words_ok(o->counts))) return STRATA_EINVAL;
  if (T > 0 && (!words_ok(topk_idx) || !words_ok(o->entries) || !words_ok(o->place))) return STRATA_EINVAL;
  if (T > 0 && (o->entries == o->place || o->place == topk_idx || o->entries == topk_idx)) return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  // one CTA up to 64 entries a warp, where a cluster's exchange costs more than it saves
  const size_t smem = (size_t)(kPlanWarps + 1) * E * 4;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (n <= kPlanWarps * 64) {
    plan_kernel<<<1, kPlanThreads, smem, s>>>(topk_idx, (int)n, E, o->counts, o->offsets, o->entries, o->place);
    return launched();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kPlanCluster), cfg.blockDim = dim3(kPlanThreads), cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kPlanCluster, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, plan_kernel, topk_idx, (int)n, E, o->counts, o->offsets, o->entries, o->place) != cudaSuccess) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  return STRATA_OK;
}

strata_status strata_sort_gather(strata_sort* h, const int32_t* place, const void* x, int64_t x_stride, void* xs,
                                 int64_t xs_stride, int32_t dtype, int32_t T, int32_t width, void* cuda_stream) {
  int size;
  const strata_status st = check_move(h, place, dtype, T, width, &size);
  if (st != STRATA_OK || T == 0) return st;
  if (!rows_ok(x, x_stride, width, size) || !rows_ok(xs, xs_stride, width, size) || x == xs) return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  MoveArgs A = move_args(h, place, T, width, size);
  A.a = static_cast<const uint4*>(x), A.as = x_stride * size / 16;
  A.out = static_cast<uint4*>(xs), A.os = xs_stride * size / 16;
  gather_kernel<<<move_grid(h, (long long)T * A.pieces), 256, 0, static_cast<cudaStream_t>(cuda_stream)>>>(A);
  return launched();
}

strata_status strata_sort_combine(strata_sort* h, const int32_t* place, const void* z, int64_t z_stride, const float* w,
                                  const void* base, int64_t base_stride, void* y, int64_t y_stride, int32_t dtype,
                                  int32_t T, int32_t width, void* cuda_stream) {
  int size;
  const strata_status st = check_move(h, place, dtype, T, width, &size);
  if (st != STRATA_OK || T == 0) return st;
  if (!rows_ok(z, z_stride, width, size) || !rows_ok(y, y_stride, width, size) || y == z) return STRATA_EINVAL;
  if (base && (!rows_ok(base, base_stride, width, size) || (T > 1 && base == y && base_stride != y_stride)))
    return STRATA_EINVAL;
  if (w && !words_ok(w)) return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  MoveArgs A = move_args(h, place, T, width, size);
  A.w = w;
  A.a = static_cast<const uint4*>(z), A.as = z_stride * size / 16;
  A.b = static_cast<const uint4*>(base), A.bs = base_stride * size / 16;
  A.out = static_cast<uint4*>(y), A.os = y_stride * size / 16;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const unsigned grid = move_grid(h, (long long)T * A.pieces);
  if (dtype == STRATA_F32)
    combine_kernel<float><<<grid, 256, 0, s>>>(A);
  else if (dtype == STRATA_F16)
    combine_kernel<__half><<<grid, 256, 0, s>>>(A);
  else
    combine_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(A);
  return launched();
}

strata_status strata_sort_combine_backward(strata_sort* h, const int32_t* place, const void* dy, int64_t dy_stride,
                                           const void* z, int64_t z_stride, const float* w, void* dz, int64_t dz_stride,
                                           float* dw, int32_t dtype, int32_t T, int32_t width, void* cuda_stream) {
  int size;
  const strata_status st = check_move(h, place, dtype, T, width, &size);
  if (st != STRATA_OK || T == 0) return st;
  if (!rows_ok(dy, dy_stride, width, size) || (!dz && !dw)) return STRATA_EINVAL;
  if (dw && (!words_ok(dw) || !rows_ok(z, z_stride, width, size) || dw == w)) return STRATA_EINVAL;
  if (dz && (!rows_ok(dz, dz_stride, width, size) || dz == dy || (dz == z && dz_stride != z_stride)))
    return STRATA_EINVAL;
  if (w && !words_ok(w)) return STRATA_EINVAL;
  if (fault_is("launch")) return STRATA_ECUDA;
  DeviceScope on(h->device);
  if (!on.ok) {
    cudaGetLastError();
    return STRATA_ECUDA;
  }
  MoveArgs A = move_args(h, place, T, width, size);
  A.w = w, A.dw = dw;
  A.a = static_cast<const uint4*>(dy), A.as = dy_stride * size / 16;
  A.b = static_cast<const uint4*>(z), A.bs = z_stride * size / 16;
  A.out = static_cast<uint4*>(dz), A.os = dz_stride * size / 16;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (dtype == STRATA_F32)
    combine_backward_kernel<float><<<(unsigned)T, kBackThreads, 0, s>>>(A);
  else if (dtype == STRATA_F16)
    combine_backward_kernel<__half><<<(unsigned)T, kBackThreads, 0, s>>>(A);
  else
    combine_backward_kernel<__nv_bfloat16><<<(unsigned)T, kBackThreads, 0, s>>>(A);
  return launched();
}

strata_status strata_sort_destroy(strata_sort* h) {
  delete h;
  return STRATA_OK;
}

}  // extern "C"
