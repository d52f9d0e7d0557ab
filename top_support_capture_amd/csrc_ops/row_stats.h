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
  __device__ static inline void unpack(const Chunk& c, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(c.v[i] << 16);
      x[2 * i + 1] = __uint_as_float(c.v[i] & 0xFFFF0000u);
    }
  }
  __device__ static inline float get(const Bits* p) { return __uint_as_float((uint32_t)*p << 16); }
  // Results are rounded once, to nearest even, from the 32-bit value.
  __device__ static inline void put(Bits* p, float x) { *p = __builtin_bit_cast(uint16_t, (__bf16)x); }
  __device__ static inline void store(Bits* p, const float (&x)[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16;
    *reinterpret_cast<u32x4_by2*>(p) = v;
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
    q[0] = a, q[1] = b;
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

__device__ inline float get_any(const void* row, int64_t at, int dtype) {
  return dtype == TSC_DTYPE_F32 ? Row<TSC_DTYPE_F32>::get((const float*)row + at)
                                : Row<TSC_DTYPE_BF16>::get((const uint16_t*)row + at);
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
  template <int N>
  __device__ inline void add(const float (&x)[N], Scale c) {
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
__device__ inline double rescaled(double s, float m, float M, Scale c) {
  return m == M ? s : s * (double)exp2_scaled(m - M, c);
}

// The workgroup's state from its threads', the same for every thread.
template <int kW>
__device__ inline void block_lse(float& m, double& s, Scale c, float* sh_m, double* sh_s) {
  const uint32_t w = threadIdx.x / kWaveSize, lane = threadIdx.x & (kWaveSize - 1);
  const float wm = wave_reduce(m, [](float a, float b) { return __builtin_fmaxf(a, b); });
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

// Statistics of row[lo, hi) into *out (threads of one workgroup of kOpThreads).
template <int DT>
__device__ inline void slice_stats(const typename Row<DT>::Bits* row, int64_t lo, int64_t hi,
                                   Scale c, float* sh_m, double* sh_s, RowPart* out) {
  constexpr int kU = 4;  // chunks in flight per thread
  LseState st;
  for (int64_t at = lo + (int64_t)threadIdx.x * 8; at < hi; at += (int64_t)kOpThreads * 8 * kU) {
    float x[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u) load8<DT>(row, at + (int64_t)u * kOpThreads * 8, hi, x[u]);
    float f[kU * 8];
#pragma unroll
    for (int i = 0; i < kU * 8; ++i) f[i] = x[i >> 3][i & 7];
    st.add(f, c);
  }
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
  const float wm = wave_reduce(m, [](float a, float b) { return __builtin_fmaxf(a, b); });
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
__device__ inline RowPart merge_slices(RowPart v, Scale c) {
  const float M = wave_reduce(v.m, [](float a, float b) { return __builtin_fmaxf(a, b); });
  const int32_t at = wave_reduce(v.m == M ? v.at : INT32_MAX, MinOp());
  return {M, at, wave_reduce(rescaled(v.s, v.m, M, c), SumOp())};
}

}  // namespace tsc
