// Writing a call's keys and values into the 8-bit caches, and reading them
// back.
#include "kv8.cuh"

namespace strata {
namespace {

constexpr int kThreads = 256;

// Largest magnitudes of 16 bytes of values as they are in memory: for the 16-bit types two at a time (their bits
// without the sign are ordered as their magnitudes).  bits(): as an f32's.
template <typename T> struct Abs;
template <> struct Abs<float> {
  static __device__ __forceinline__ unsigned most(unsigned a, const uint4& u) {
    return max(max(max(a, u.x & 0x7FFFFFFFu), u.y & 0x7FFFFFFFu), max(u.z & 0x7FFFFFFFu, u.w & 0x7FFFFFFFu));
  }
  static __device__ __forceinline__ unsigned bits(unsigned a) { return a; }
};
template <> struct Abs<__nv_bfloat16> {
  static __device__ __forceinline__ unsigned most(unsigned a, const uint4& u) {
    return __vmaxu2(__vmaxu2(__vmaxu2(a, u.x & 0x7FFF7FFFu), u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
  }
  static __device__ __forceinline__ unsigned bits(unsigned a) { return max(a >> 16, a & 0xFFFFu) << 16; }
};
template <> struct Abs<__half> {
  static __device__ __forceinline__ unsigned most(unsigned a, const uint4& u) { return Abs<__nv_bfloat16>::most(a, u); }
  static __device__ __forceinline__ unsigned bits(unsigned a) {
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)max(a >> 16, a & 0xFFFFu))));
  }
};

// --- append -------------------------------------------------------------------
//
// One CTA owns one block of one head, of the keys or of the values: it finds
// the largest new magnitude, fixes the exponent, requantises what the block
// holds if the exponent grew, and writes the new codes.  Its new values stay in
// registers between the two passes (NP 16-byte loads a thread, all in flight),
// so they are read once.  24 k bf16 rows of 8 heads of 128 (150 MB in and out): 34.2 us, 64% of the measured HBM rate;
// issue bound (68% of the slots), so magnitudes are taken two at a time and what is not finite has a path of its own
// (43.1 us before both).  A window's rows: 2.2 us.
template <typename T, int NP>
__device__ __forceinline__ void append_block(const Kv8Dev& C, const Kv8Rows& R, const T* __restrict__ kin,
                                             long long k_stride, const T* __restrict__ vin, long long v_stride, int i,
                                             int b_at, int head, bool is_v) {
  constexpr int kPer = Val<T>::kPer;
  __shared__ unsigned red[kThreads / 32];
  const Kv8Seq q = kv8_seq(R, C, i);
  const bool lead = threadIdx.x == 0 && b_at == 0 && head == 0 && !is_v;
  if (!q.held_ok || q.length < q.n) {
    if (lead) atomicOr(C.err, kErrIndex);
    return;
  }
  if (q.n == 0) return;
  const int p0 = q.length - q.n;  // first new position
  const int B = 1 << C.block_log2;
  const int blk = (p0 >> C.block_log2) + b_at;
  const int lo = max(p0, blk << C.block_log2), hi = min(q.length, (blk + 1) << C.block_log2);
  if (lo >= hi) return;
  // the new values, all on their way before anything waits
  const int hd = C.head_dim;
  const int tpt_log2 = (hd == 128 ? 7 : 6) - (kPer == 4 ? 2 : 3);  // threads per token
  const int per_pass = kThreads >> tpt_log2;
  const int t0 = threadIdx.x >> tpt_log2, d = (threadIdx.x & ((1 << tpt_log2) - 1)) * kPer;
  const T* src = is_v ? vin : kin;
  const long long stride = is_v ? v_stride : k_stride;
  const T* base = src + (long long)(q.row0 + lo - p0) * stride + (long long)head * hd + d;
  const int n = hi - lo;
  uint4 raw[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int t = t0 + p * per_pass;
    raw[p] = t < n ? __ldcs(reinterpret_cast<const uint4*>(base + (long long)t * stride)) : make_uint4(0, 0, 0, 0);
  }
  const long long line = (long long)q.slot * C.kv_heads + head;
  uint8_t* codes = (is_v ? C.v : C.k) + (line * C.max_ctx + (blk << C.block_log2)) * hd;
  uint8_t* ep = (is_v ? C.v_exp : C.k_exp) + line * C.n_blocks + blk;
  const int held = lo - (blk << C.block_log2);
  const int e_held = held > 0 ? kv8_exp(*ep) : kKv8EMin;
  // an earlier sequence with rows that names the same slot owns it, unless it is itself left out
  int taken = 0;
  for (int j = threadIdx.x; j < i; j += kThreads)
    if (R.slot[j] == q.slot) {
      const Kv8Seq other = kv8_seq(R, C, j);
      if (other.held_ok && other.n > 0 && other.length >= other.n) taken = 1;
    }
  unsigned a = 0;
#pragma unroll
  for (int p = 0; p < NP; ++p) a = Abs<T>::most(a, raw[p]);
  a = Abs<T>::bits(a);
  const bool odd = a >= 0x7F800000u;
  if (odd) {  // something is not finite: the largest of the others
    a = 0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      float f[kPer];
      Val<T>::unpack(raw[p], f);
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const unsigned m = __float_as_uint(f[x]) & 0x7FFFFFFFu;
        if (m < 0x7F800000u) a = max(a, m);
      }
    }
  }
  a = __reduce_max_sync(0xFFFFFFFFu, a);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  // one barrier: the maxima are there, and every thread has read the held exponent
  if (__syncthreads_or(taken)) {
    if (lead) atomicOr(C.err, kErrIndex);
    return;
  }
  if (odd) atomicOr(C.err, kErrNonFinite);
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) a = max(a, red[w]);

  int e = kv8_least_exp(__uint_as_float(a), C.format);
  if (held > 0) {
    if (e > e_held) {
      const float f = pow2i(e_held - e);
      uint32_t* w = reinterpret_cast<uint32_t*>(codes);
      for (int j = threadIdx.x; j < held * hd / 4; j += kThreads) {
        float x[4];
        kv8_decode4(w[j], C.format, x);
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] = x[y] == x[y] ? x[y] * f : 0.f;
        w[j] = kv8_encode4(x, C.format);
      }
    } else {
      e = e_held;
    }
  }
  if (threadIdx.x == 0) *ep = (uint8_t)(e + kKv8Bias);
  const float f = pow2i(-e);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int t = t0 + p * per_pass;
    if (t >= n) break;
    float x[kPer];
    Val<T>::unpack(raw[p], x);
#pragma unroll
    for (int y = 0; y < kPer; ++y) x[y] *= f;
    if (odd) {
#pragma unroll
      for (int y = 0; y < kPer; ++y) x[y] = x[y] == x[y] ? x[y] : 0.f;
    }
    uint8_t* to = codes + (held + t) * hd + d;
    if constexpr (kPer == 4)
      *reinterpret_cast<uint32_t*>(to) = kv8_encode4(x, C.format);
    else
      *reinterpret_cast<uint2*>(to) = make_uint2(kv8_encode4(x, C.format), kv8_encode4(x + 4, C.format));
  }
}

// Blocks that n consecutive positions can touch.
__host__ __device__ constexpr long long append_pieces(int n, int B) { return n > 0 ? (n + (long long)B - 2) / B + 1 : 0; }

// kList: the CTAs share the list of all sequences' blocks; else each sequence has nb places.
template <typename T, int NP, bool kList>
__global__ void __launch_bounds__(kThreads) append_kernel(Kv8Dev C, Kv8Rows R, const T* __restrict__ kin,
                                                          long long k_stride, const T* __restrict__ vin,
                                                          long long v_stride, int nb) {
  const int lines = 2 * C.kv_heads;  // keys and values of each head
  if constexpr (kList) {
    for (long long id = blockIdx.x;; id += gridDim.x) {
      const Kv8Piece p = kv8_find<kThreads>(R, id / lines, [&](int n) { return append_pieces(n, 1 << C.block_log2); });
      if (p.seq < 0) return;
      const int line = (int)(id % lines);
      append_block<T, NP>(C, R, kin, k_stride, vin, v_stride, p.seq, p.at, line >> 1, line & 1);
      if (id + gridDim.x >= p.all * lines) return;
    }
  } else {
    int id = blockIdx.x;
    const int b_at = id % nb;
    id /= nb;
    const int head = id % C.kv_heads;
    id /= C.kv_heads;
    append_block<T, NP>(C, R, kin, k_stride, vin, v_stride, id >> 1, b_at, head, id & 1);
  }
}

// CTAs of a launch over pieces of sequences: `each` places for every sequence, or a list of `most` pieces (which the
// rows cannot need more of unless sequences lie over one another; the CTAs go on until the list's end).  A sequence's
// place is found without a search, so short and even batches take the first; the second once the first would start
// more than twice the CTAs.  8 heads of 128, bf16, blocks of 16, places / list in us: 64 sequences of 256 rows, append 46 /
// 73 and read 17.5 / 23.5; 63 of 256 and one of 512, 60 / 74 and 21 / 24; one of 1024 (2.9 and 3.9 times the CTAs), 88 /
// 77 and 30 / 25.5; 63 single rows and one prompt of 8129, 437 / 42 and 138 / 17; 1023 and one of 100000, read 25 ms /
// 205 us.
constexpr long long kMaxGrid = 0x7FFFFFFF;
struct PieceGrid { bool list; unsigned grid; };
PieceGrid piece_grid(const Kv8Dev& C, const Kv8Rows& R, long long each, long long most) {
  const long long lines = 2LL * C.kv_heads;
  const bool list = R.n_seq * each > 2 * most || lines * R.n_seq * each > kMaxGrid;
  return {list, (unsigned)min(lines * (list ? most : R.n_seq * each), kMaxGrid)};
}

template <typename T>
cudaError_t append_typed(const Kv8Dev& C, const Kv8Rows& R, const void* k, long long k_stride, const void* v,
                         long long v_stride, cudaStream_t s) {
  const int B = 1 << C.block_log2;
  const int nb = (int)append_pieces(min(R.max_rows, C.max_ctx), B);
  const PieceGrid g = piece_grid(C, R, nb, R.n_rows / B + 2LL * R.n_seq);
  const T *kk = static_cast<const T*>(k), *vv = static_cast<const T*>(v);
  // passes of the CTA over the tokens that a block can gain in this call
  const int most = min(B, R.max_rows);
  const int per_pass = kThreads * Val<T>::kPer / C.head_dim;
  const int np = (most + per_pass - 1) / per_pass;
#define STRATA_APPEND(NP)                                                                              \
  do {                                                                                                 \
    if (g.list)                                                                                        \
      append_kernel<T, NP, true><<<g.grid, kThreads, 0, s>>>(C, R, kk, k_stride, vv, v_stride, nb);    \
    else                                                                                               \
      append_kernel<T, NP, false><<<g.grid, kThreads, 0, s>>>(C, R, kk, k_stride, vv, v_stride, nb);   \
  } while (0)
  if (np <= 1)
    STRATA_APPEND(1);
  else if (np <= 2)
    STRATA_APPEND(2);
  else if (np <= 4)
    STRATA_APPEND(4);
  else if (np <= 8)
    STRATA_APPEND(8);
  else
    STRATA_APPEND(16);
#undef STRATA_APPEND
  return cudaGetLastError();
}

// --- read -----------------------------------------------------------------------
//
// A CTA turns up to kReadPasses passes of tokens of one head into values: a
// thread reads as many codes as fill a 16-byte store, so that both sides are
// contiguous across a warp.  HBM bound (codes in, values out): 99 k positions of 8 heads of 128 to bf16 (606 MB) in
// 91.9 us, 97% of the measured rate.
constexpr int kReadPasses = 8;

template <typename T>
__device__ __forceinline__ void read_chunk(const Kv8Dev& C, const Kv8Rows& R, T* __restrict__ kout, long long k_stride,
                                           T* __restrict__ vout, long long v_stride, int i, int chunk, int head,
                                           bool is_v) {
  constexpr int kPer = Val<T>::kPer;
  const Kv8Seq q = kv8_seq(R, C, i);
  const bool ok = q.held_ok && q.length >= q.n;
  if (!ok && threadIdx.x == 0 && chunk == 0 && head == 0 && !is_v) atomicOr(C.err, kErrIndex);
  if (!q.rows_ok) return;
  const int hd = C.head_dim;
  const int tpt_log2 = (hd == 128 ? 7 : 6) - (kPer == 4 ? 2 : 3);
  const int per_pass = kThreads >> tpt_log2;
  const int d = (threadIdx.x & ((1 << tpt_log2) - 1)) * kPer;
  const int t0 = chunk * (per_pass * kReadPasses) + (threadIdx.x >> tpt_log2);
  const long long line = (long long)q.slot * C.kv_heads + head;
  const int p0 = q.length - q.n;
  const uint8_t* codes = (is_v ? C.v : C.k);
  const uint8_t* eb = (is_v ? C.v_exp : C.k_exp);
  if (ok) {
    codes += (line * C.max_ctx + p0) * hd + d;
    eb += line * C.n_blocks;
  }
  T* dst = is_v ? vout : kout;
  const long long stride = is_v ? v_stride : k_stride;
  dst += (long long)q.row0 * stride + (long long)head * hd + d;
  uint2 raw[kReadPasses];
  uint8_t ex[kReadPasses];
#pragma unroll
  for (int p = 0; p < kReadPasses; ++p) {
    const int t = t0 + p * per_pass;
    raw[p] = make_uint2(0, 0);
    ex[p] = 0;
    if (ok && t < q.n) {
      if constexpr (kPer == 4)
        raw[p].x = *reinterpret_cast<const uint32_t*>(codes + (long long)t * hd);
      else
        raw[p] = *reinterpret_cast<const uint2*>(codes + (long long)t * hd);
      ex[p] = eb[(p0 + t) >> C.block_log2];
    }
  }
#pragma unroll
  for (int p = 0; p < kReadPasses; ++p) {
    const int t = t0 + p * per_pass;
    if (t >= q.n) break;
    const float f = pow2i(kv8_exp(ex[p]));
    float x[8];
    kv8_decode4(raw[p].x, C.format, x);
    if constexpr (kPer == 8) kv8_decode4(raw[p].y, C.format, x + 4);
#pragma unroll
    for (int y = 0; y < kPer; ++y) x[y] = ok ? x[y] * f : 0.f;
    *reinterpret_cast<uint4*>(dst + (long long)t * stride) = Val<T>::pack(x);
  }
}

// kList: as append_kernel's.
template <typename T, bool kList>
__global__ void __launch_bounds__(kThreads) read_kernel(Kv8Dev C, Kv8Rows R, T* __restrict__ kout, long long k_stride,
                                                        T* __restrict__ vout, long long v_stride, int nchunk) {
  const int lines = 2 * C.kv_heads;
  if constexpr (kList) {
    const int per_cta = kThreads * Val<T>::kPer / C.head_dim * kReadPasses;
    for (long long id = blockIdx.x;; id += gridDim.x) {
      const Kv8Piece p = kv8_find<kThreads>(R, id / lines, [&](int n) { return (n + (long long)per_cta - 1) / per_cta; });
      if (p.seq < 0) return;
      const int line = (int)(id % lines);
      read_chunk<T>(C, R, kout, k_stride, vout, v_stride, p.seq, p.at, line >> 1, line & 1);
      if (id + gridDim.x >= p.all * lines) return;
    }
  } else {
    int id = blockIdx.x;
    const int chunk = id % nchunk;
    id /= nchunk;
    const int head = id % C.kv_heads;
    id /= C.kv_heads;
    read_chunk<T>(C, R, kout, k_stride, vout, v_stride, id >> 1, chunk, head, id & 1);
  }
}

template <typename T>
cudaError_t read_typed(const Kv8Dev& C, const Kv8Rows& R, void* k, long long k_stride, void* v, long long v_stride,
                       cudaStream_t s) {
  const int per_cta = kThreads * Val<T>::kPer / C.head_dim * kReadPasses;
  const int nchunk = (R.max_rows + per_cta - 1) / per_cta;
  const PieceGrid g = piece_grid(C, R, nchunk, R.n_rows / per_cta + (long long)R.n_seq);
  T *kk = static_cast<T*>(k), *vv = static_cast<T*>(v);
  if (g.list)
    read_kernel<T, true><<<g.grid, kThreads, 0, s>>>(C, R, kk, k_stride, vv, v_stride, nchunk);
  else
    read_kernel<T, false><<<g.grid, kThreads, 0, s>>>(C, R, kk, k_stride, vv, v_stride, nchunk);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Dev& C, const Kv8Rows& R, const void* k, long long k_stride, const void* v,
                              long long v_stride, int dtype, cudaStream_t s) {
  if (dtype == 0) return append_typed<float>(C, R, k, k_stride, v, v_stride, s);
  if (dtype == 1) return append_typed<__half>(C, R, k, k_stride, v, v_stride, s);
  return append_typed<__nv_bfloat16>(C, R, k, k_stride, v, v_stride, s);
}

cudaError_t launch_kv8_read(const Kv8Dev& C, const Kv8Rows& R, void* k, long long k_stride, void* v,
                            long long v_stride, int dtype, cudaStream_t s) {
  if (dtype == 0) return read_typed<float>(C, R, k, k_stride, v, v_stride, s);
  if (dtype == 1) return read_typed<__half>(C, R, k, k_stride, v, v_stride, s);
  return read_typed<__nv_bfloat16>(C, R, k, k_stride, v, v_stride, s);
}

}  // namespace strata
