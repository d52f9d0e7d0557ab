// Softmax statistics of logits rows, cut into slices over many workgroups: the common first pass
// of draft verification (verify.h) and distillation (distill.h).
//
// With c = log2(e) / T, a row's softmax is 2^((x_i - m) c) / s, m the maximum and s the sum of
// the numerators. One pass gives both: each thread keeps a running maximum and the sum relative
// to it, rescaled when the maximum grows; partial states merge the same way.
#pragma once

#include "tsc_device.h"

namespace tsc {

constexpr int kOpThreads = 256;
constexpr int kOpWaves = kOpThreads / kWaveSize;
constexpr int kMaxSlices = 64;  // one lane of a wave holds one slice's state when they are merged

// Rows are read in chunks of 8 elements from the row's first element on, whatever its address:
// gfx950 loads 16 bytes from any element boundary, so rows of odd strides need no other path.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_by2 __attribute__((aligned(2)));
typedef u32x4 u32x4_by4 __attribute__((aligned(4)));

template <int DT>
struct Row;

template <>
struct Row<TSC_DTYPE_BF16> {
  using Bits = uint16_t;
  struct Chunk {
    u32x4 v;
  };
  __device__ static inline Chunk load(const Bits* p) {
    return {*reinterpret_cast<const u32x4_by2*>(p)};
  }
  // For rows that are not read again: leaves the caches to others.
  __device__ static inline Chunk load_once(const Bits* p) {
    return {__builtin_nontemporal_load(reinterpret_cast<const u32x4_by2*>(p))};
  }
  __device__ static inline void unpack(const Chunk& c, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(c.v[i] << 16);
      x[2 * i + 1] = __uint_as_float(c.v[i] & 0xFFFF0000u);
    }
  }
  __device__ static inline float get(const Bits* p) { return __uint_as_float((uint32_t)*p << 16); }
  // Results are rounded once, to nearest even, from the 32-bit value. Whole chunks are stored
  // nontemporally: a gradient is not read again soon, and what the caches keep instead (a row that
  // the loss has read) the gradient's pass reads again.
  __device__ static inline void put(Bits* p, float x) { *p = __builtin_bit_cast(uint16_t, (__bf16)x); }
  __device__ static inline void store(Bits* p, const float (&x)[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16;
    __builtin_nontemporal_store((u32x4_by2)v, reinterpret_cast<u32x4_by2*>(p));
  }
};

template <>
struct Row<TSC_DTYPE_F32> {
  using Bits = float;
  struct Chunk {
    u32x4 v[2];
  };
  __device__ static inline Chunk load(const Bits* p) {
    const u32x4_by4* q = reinterpret_cast<const u32x4_by4*>(p);
    return {{q[0], q[1]}};
  }
  __device__ static inline Chunk load_once(const Bits* p) {
    const u32x4_by4* q = reinterpret_cast<const u32x4_by4*>(p);
    return {{__builtin_nontemporal_load(q), __builtin_nontemporal_load(q + 1)}};
  }
  __device__ static inline void unpack(const Chunk& c, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(c.v[i >> 2][i & 3]);
  }
  __device__ static inline float get(const Bits* p) { return *p; }
  __device__ static inline void put(Bits* p, float x) { *p = x; }
  __device__ static inline void store(Bits* p, const float (&x)[8]) {
    u32x4_by4* q = reinterpret_cast<u32x4_by4*>(p);
    u32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(x[i]), b[i] = __float_as_uint(x[i + 4]);
    __builtin_nontemporal_store((u32x4_by4)a, q);
    __builtin_nontemporal_store((u32x4_by4)b, q + 1);
  }
};

// The 8 elements from position `at`; those at or past `end` read as -inf (the last chunk of a row
// whose length is no multiple of 8).
template <int DT>
__device__ inline void load8(const typename Row<DT>::Bits* row, int64_t at, int64_t end,
                             float (&x)[8]) {
  if (at + 8 <= end) {
    Row<DT>::unpack(Row<DT>::load(row + at), x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = at + e < end ? Row<DT>::get(row + at + e) : -__builtin_inff();
  }
}

template <int DT>
__device__ inline void store8(typename Row<DT>::Bits* row, int64_t at, int64_t end,
                              const float (&x)[8]) {
  if (at + 8 <= end) {
    Row<DT>::store(row + at, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e < end) Row<DT>::put(row + at + e, x[e]);
  }
}

// A temperature the sampler takes for sampling: normal, positive, finite.
__device__ inline bool temperature_ok(float T) {
  return __builtin_isfinite(T) && T >= 1.1754943508222875e-38f;
}

// c = log2(e) / T as hi + lo, hi rounded down, so that an exponent (x - m) c keeps the rounding
// error of one float32 operation: a single float32 c would shift all exponents of a row by up to
// 2^-25 of their size, the same way for every element. lo > 0, so that d = -inf gives -inf and
// never -inf + inf.
struct Scale {
  float hi, lo;
};

__device__ inline Scale make_scale(float T) {
  const double c = 1.4426950408889634074 / (double)T;
  float hi = (float)c;
  if ((double)hi > c) hi = __uint_as_float(__float_as_uint(hi) - 1u);
  const float lo = (float)(c - (double)hi);
  return {hi, lo > 0.0f ? lo : 0x1p-149f};
}

// 2^(d c) for d <= 0 (d = x - m); NaN stays NaN.
__device__ inline float exp2_scaled(float d, Scale c) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(d, c.lo, d * c.hi));
}

// With c = log2(e) / T in one float32: one operation less, and an error of 2^-24 |d c| from c
// itself beside the product's rounding. For losses and gradients, which are float32 or less;
// decisions between probabilities take the Scale.
__device__ inline float exp2_scaled(float d, float c) { return __builtin_amdgcn_exp2f(d * c); }
__device__ inline float plain_scale(float T) { return (float)(1.4426950408889634074 / (double)T); }

// State of a slice of a row. `s` is NaN when the slice holds a NaN or a +inf. `at` (greedy rows
// only, whose s is otherwise 1) is the first index of the maximum.
struct RowPart {
  float m;
  int32_t at;
  double s;
};

// Running state of a thread: sums of up to 32 numerators in float32, all else in float64.
struct LseState {
  float m = -__builtin_inff();
  double s = 0.0;
  template <int N, class C>
  __device__ inline void add(const float (&x)[N], C c) {
    float b = m;
#pragma unroll
    for (int i = 0; i < N; ++i) b = __builtin_fmaxf(b, x[i]);
    const float base = b == -__builtin_inff() ? 0.0f : b;
    float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) t[i & 3] += exp2_scaled(x[i] - base, c);
    if (b != m) {  // m = -inf: s is 0
      s *= (double)exp2_scaled(m - b, c);
      m = b;
    }
    s += (double)((t[0] + t[1]) + (t[2] + t[3]));
  }
};

// s relative to m, relative to M >= m instead (both may be -inf: s is 0 then, or NaN).
template <class C>
__device__ inline double rescaled(double s, float m, float M, C c) {
  return m == M ? s : s * (double)exp2_scaled(m - M, c);
}

__device__ inline float wave_max(float v) {
  return wave_reduce(v, [](float p, float q) { return __builtin_fmaxf(p, q); });
}

// The workgroup's state from its threads', the same for every thread. kW waves; sh_m and sh_s
// hold one entry each.
template <int kW, class C>
__device__ inline void block_lse(float& m, double& s, C c, float* sh_m, double* sh_s) {
  const uint32_t w = threadIdx.x / kWaveSize, lane = threadIdx.x & (kWaveSize - 1);
  const float wm = wave_max(m);
  const double ws = wave_reduce(rescaled(s, m, wm, c), SumOp());
  if (lane == 0) sh_m[w] = wm, sh_s[w] = ws;
  lds_barrier();
  float M = sh_m[0];
#pragma unroll
  for (int i = 1; i < kW; ++i) M = __builtin_fmaxf(M, sh_m[i]);
  double S = 0.0;
#pragma unroll
  for (int i = 0; i < kW; ++i) S += rescaled(sh_s[i], sh_m[i], M, c);
  m = M, s = S;
}

// A value over a workgroup of 16 waves under op, the same for every thread; sh holds one entry per
// wave.
template <class T, class Op>
__device__ inline T block_all(T v, Op op, T* sh) {
  v = wave_reduce(v, op);
  lds_barrier();  // sh may still be read by an earlier call
  if ((threadIdx.x & (kWaveSize - 1)) == 0) sh[threadIdx.x / kWaveSize] = v;
  lds_barrier();
  return row16_reduce(sh[threadIdx.x & 15], op);
}

// ---- Writing a row with a few scattered entries --------------------------------------------------
// A gradient row is a stream over the vocabulary plus a term at each of a few thousand ids. The
// row is written window by window, a chunk per thread: the entries of a window are added up in
// LDS in float32 and join the stream's chunks there, so that each result is rounded once and
// stored in whole chunks. (Writing the entries over a finished row instead costs a read and a
// write of their lines each: for 1000 entries in a row of 151936, more traffic than the row.) The
// entries are sorted by window first, so that a window looks at its own only.
constexpr int kMaxWindows = 64;

// kThr * 8 elements. The halves of a thread's chunk lie apart, so that the 16-byte reads of
// neighbouring lanes neighbour each other.
template <int kThr>
struct Window {
  static constexpr int kSize = kThr * 8;
  float* f;
  __device__ inline void clear() const {
    for (int i = (int)threadIdx.x * 4; i < kSize; i += kThr * 4)
      *reinterpret_cast<float4*>(f + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  __device__ inline void add(uint32_t at, float v) const {  // at < kSize
    atomicAdd(f + ((at >> 2) & 1u) * (kThr * 4) + (at >> 3) * 4 + (at & 3u), v);
  }
  // Chunk t, left cleared for the window after the next.
  __device__ inline void take(int t, float (&d)[8]) const {
    float4* p = reinterpret_cast<float4*>(f + t * 4);
    const float4 a = p[0], b = p[kThr];
    d[0] = a.x, d[1] = a.y, d[2] = a.z, d[3] = a.w;
    d[4] = b.x, d[5] = b.y, d[6] = b.z, d[7] = b.w;
    uint32_t any = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) any |= __float_as_uint(d[e]);
    if (any != 0u) p[0] = p[kThr] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
};

// LDS of a workgroup that writes such rows: the entries, and two windows, which take turns so that
// one barrier separates a window's entries from its chunks; or one window, where that lets a second
// workgroup on the CU, or where two do not fit.
template <int kThr>
struct Entries {
  static constexpr int kSize = Window<kThr>::kSize;
  // Counters of a window: lanes that count into the same window at the same time mostly meet
  // different ones.
  static constexpr int kCopies = 4;
  static constexpr int64_t kFixed = (kMaxWindows + 4 + kMaxWindows * kCopies) * 4;
  static constexpr int64_t kHalf = 78 * 1024, kAll = 156 * 1024;  // of a CU's LDS, beside static LDS
  bool two;
  float* window;     // [1 or 2][kSize]
  uint32_t* start;   // [kMaxWindows + 1]
  uint32_t* cursor;  // [kMaxWindows][kCopies]
  float* val;        // [W]
  uint16_t* rel;     // [W]
  __host__ __device__ static constexpr int64_t with(int windows, int64_t W) {
    return windows * kSize * 4 + W * 4 + kFixed + (W + 1) / 2 * 4;
  }
  // `more`: bytes that the kernel needs behind them.
  __host__ __device__ static constexpr bool takes_two(int64_t W, int64_t more) {
    return with(2, W) + more <= (with(1, W) + more <= kHalf ? kHalf : kAll);
  }
  __host__ __device__ static constexpr size_t bytes(int64_t W, int64_t more = 0) {
    return (size_t)(with(takes_two(W, more) ? 2 : 1, W) + more);
  }
  __device__ inline explicit Entries(void* lds, int32_t W, int64_t more = 0) {
    two = takes_two(W, more);
    window = reinterpret_cast<float*>(lds);
    start = reinterpret_cast<uint32_t*>(window + (two ? 2 : 1) * kSize);
    cursor = start + kMaxWindows + 4;  // 16-byte aligned, as `lds` and the window's size are
    val = reinterpret_cast<float*>(cursor + kMaxWindows * kCopies);
    rel = reinterpret_cast<uint16_t*>(val + W);
  }
  // In this order, with a barrier between any two: begin, count of every entry, offsets, place of
  // every entry. `at` counts from the segment's first element and is below kMaxWindows * kSize.
  __device__ inline void begin() const {
    Window<kThr>{window}.clear();
    if (two) Window<kThr>{window + kSize}.clear();
    if (threadIdx.x < kMaxWindows * kCopies) cursor[threadIdx.x] = 0u;
  }
  __device__ inline uint32_t* counter(uint32_t at) const {
    return &cursor[at / kSize * kCopies + (threadIdx.x & (kCopies - 1))];
  }
  __device__ inline void count(uint32_t at) const { atomicAdd(counter(at), 1u); }
  __device__ inline void offsets() const {
    if (threadIdx.x < kMaxWindows) {  // the first wave, a window per lane
      uint4 n = *reinterpret_cast<uint4*>(cursor + threadIdx.x * kCopies);
      const uint32_t sum = n.x + n.y + n.z + n.w, incl = wave_incl_scan(sum, SumOp(), 0u), at = incl - sum;
      start[threadIdx.x] = at;
      *reinterpret_cast<uint4*>(cursor + threadIdx.x * kCopies) =
          make_uint4(at, at + n.x, at + n.x + n.y, at + n.x + n.y + n.z);
      if (threadIdx.x == kMaxWindows - 1) start[kMaxWindows] = incl;
    }
  }
  __device__ inline void place(uint32_t at, float v) const {
    const uint32_t i = atomicAdd(counter(at), 1u);
    val[i] = v, rel[i] = (uint16_t)(at % kSize);
  }
  __device__ inline Window<kThr> at_window(int k) const { return {window + (two ? (k & 1) * kSize : 0)}; }
  // Window k's turn: use() takes its chunks; put(k + 1) adds the entries of the next.
  template <class Put, class Use>
  __device__ inline void turn(int k, Put put, Use use) const {
    if (two) put(k + 1);
    use();
    lds_barrier();
    if (!two) {
      put(k + 1);
      lds_barrier();
    }
  }
  // The entries of window k (none past the last).
  __device__ inline void add(int k) const {
    if (k >= kMaxWindows) return;
    const Window<kThr> win = at_window(k);
    for (uint32_t i = start[k] + threadIdx.x; i < start[k + 1]; i += kThr) win.add(rel[i], val[i]);
  }
};

// A thread's state of row[lo, hi) in a workgroup of kThr threads. passing(b, e) is called when the
// workgroup has asked for the elements [b, e): what it reads there is on its way or in the caches.
struct NoVisit {
  __device__ inline void operator()(int64_t, int64_t) const {}
};
template <int DT, int kThr, class C, class Passing = NoVisit>
__device__ inline LseState thread_stats(const typename Row<DT>::Bits* row, int64_t lo, int64_t hi, C c,
                                        Passing passing = Passing()) {
  constexpr int kU = 4;  // chunks in flight per thread
  constexpr int64_t kStep = (int64_t)kThr * 8;
  LseState st;
  const int64_t first = (int64_t)threadIdx.x * 8;
  int64_t base = lo;
  for (; base + kU * kStep <= hi; base += kU * kStep) {
    typename Row<DT>::Chunk v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) v[u] = Row<DT>::load(row + base + u * kStep + first);
    passing(base, base + kU * kStep);
    float f[kU * 8];
#pragma unroll
    for (int u = 0; u < kU; ++u) Row<DT>::unpack(v[u], reinterpret_cast<float(&)[8]>(f[u * 8]));
    st.add(f, c);
  }
  if (base < hi) {
    passing(base, hi);
    for (int64_t at = base + first; at < hi; at += kStep) {
      float x[8];
      load8<DT>(row, at, hi, x);
      st.add(x, c);
    }
  }
  return st;
}

// Statistics of row[lo, hi) into *out (threads of one workgroup of kOpThreads).
template <int DT, class C>
__device__ inline void slice_stats(const typename Row<DT>::Bits* row, int64_t lo, int64_t hi,
                                   C c, float* sh_m, double* sh_s, RowPart* out) {
  LseState st = thread_stats<DT, kOpThreads>(row, lo, hi, c);
  block_lse<kOpWaves>(st.m, st.s, c, sh_m, sh_s);
  if (threadIdx.x == 0) *out = {st.m, 0, st.s};
}

// First maximum of row[lo, hi) into *out, for greedy rows; s marks a NaN or +inf.
template <int DT>
__device__ inline void slice_argmax(const typename Row<DT>::Bits* row, int64_t lo, int64_t hi,
                                    float* sh_m, double* sh_s, int32_t* sh_at, RowPart* out) {
  float m = -__builtin_inff();
  int32_t at = INT32_MAX;
  bool bad = false;
  for (int64_t p = lo + (int64_t)threadIdx.x * 8; p < hi; p += (int64_t)kOpThreads * 8) {
    float x[8];
    load8<DT>(row, p, hi, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      bad |= !(x[e] < __builtin_inff());
      if (x[e] > m) m = x[e], at = (int32_t)(p + e);
    }
  }
  const float wm = wave_max(m);
  const int32_t wat = wave_reduce(m == wm ? at : INT32_MAX, MinOp());
  const bool wbad = __ballot(bad) != 0;
  const uint32_t w = threadIdx.x / kWaveSize;
  if ((threadIdx.x & (kWaveSize - 1)) == 0)
    sh_m[w] = wm, sh_at[w] = wat, sh_s[w] = wbad ? __builtin_nan("") : 0.0;
  lds_barrier();
  if (threadIdx.x == 0) {
    RowPart r{sh_m[0], sh_at[0], sh_s[0]};
    for (int i = 1; i < kOpWaves; ++i) {
      if (sh_m[i] > r.m || (sh_m[i] == r.m && sh_at[i] < r.at)) r.m = sh_m[i], r.at = sh_at[i];
      r.s += sh_s[i];
    }
    r.s += 1.0;
    *out = r;
  }
}

// A row's state from its slices' (n <= 64, one per lane), the same for every lane.
template <class C>
__device__ inline RowPart merge_slices(RowPart v, C c) {
  const float M = wave_max(v.m);
  const int32_t at = wave_reduce(v.m == M ? v.at : INT32_MAX, MinOp());
  return {M, at, wave_reduce(rescaled(v.s, v.m, M, c), SumOp())};
}

}  // namespace tsc
