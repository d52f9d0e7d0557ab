// Log probabilities of given tokens under the whole softmax, with entropy and the most likely
// alternatives, and their gradient. With z = (x - m) / T, m the row's maximum, s = sum e^z and
// M = sum e^z z / s (the mean of z under p = e^z / s):
//     ln p_i = z_i - ln s,   H = -sum p_i ln p_i = ln s - M,
// and, with upstream gradients a of the token's logprob, b of H and u_j of the alternatives',
//     dx_i = (a [i = t] + sum_j u_j [i = id_j] - p_i (a + sum_j u_j) - b p_i (z_i - M)) / T
// (ln p_i + H = z_i - M). One pass over the row gives m, s and M; the gradient is one more, an
// affine function of z times e^z.
#pragma once

#include "replay_grad.h"
#include "top_ids.h"

namespace tsc {

constexpr int kTopThreads = 1024, kTopWaves = kTopThreads / kWaveSize;

// State of a row or a part of it: the maximum, the sum of the numerators e = 2^t, t = (x - m) log2(e) / T,
// and (kEnt) the sum of e t.
struct LogprobPart {
  float m;
  double s, a;
};

struct LogprobArgs {
  const void* logits;  // [N, V]
  int64_t N, V, ld;
  const float* temperature;  // [N] or null
  const int32_t* tokens;     // [N]
  int32_t top;
  float* logprobs;      // [N]
  float* entropy;       // [N] or null
  int32_t* top_ids;     // [N, top]
  float* top_logprobs;  // [N, top]
  int8_t* row_status;   // [N]
  float* stats;         // [N, 4] or null: m, s, M, whether the row has a gradient
  LogprobPart* parts;   // workspace [N, slices], when slices > 1
  uint64_t* keys;       // workspace [N, slices, top], when slices > 1
  int32_t slices;
  int64_t slice_len;
  const float* grad_logprobs;  // [N] or null
  const float* grad_entropy;   // [N] or null
  const float* grad_top;       // [N, top] or null
  void* grad;                  // [N, V], contiguous
  int32_t segments;
  int64_t seg_len;
  int32_t held;  // pieces a thread of the fused kernel keeps in LDS
  __device__ inline float T(int64_t n) const { return temperature ? temperature[n] : 1.0f; }
};

// Exponents below this have numerator 0; as a factor it keeps 0 * -inf out.
constexpr float kLeastExponent = -200.0f;

// The exponent t = (x - m) log2(e) / T as (half x - half m) c. From a temperature of 2^64 on half is 1/2,
// so that the difference of any two finite logits stays finite: at 1e38 some that are 5e38 apart count.
// Below, what is so far behind has numerator 0. Of a row, the same for the workgroup.
struct ExponentScale {
  float half, c;
  __device__ inline float operator()(float x, float half_m) const { return __builtin_fmaf(x, half, -half_m) * c; }
};
constexpr float kFarFrom = 0x1p64f;
__device__ inline ExponentScale exponent_scale(float T) {
  const float half = T >= kFarFrom ? 0.5f : 1.0f;
  return {half, plain_scale(half * T)};  // one division
}

// A thread's running state: sums of up to 32 terms in float32, all else in float64. `at` is the
// first piece (kTop only) that reached the maximum, -1 before the first one.
template <bool kEnt, bool kTop>
struct LogprobState {
  float m = -__builtin_inff();
  int32_t at = -1;
  double s = 0.0, a = 0.0;
  // kU pieces of kE elements, the first piece's index and the distance from one to the next. kFar: c.half
  // is 1/2.
  template <bool kFar, int kU, int kE>
  __device__ inline void add(const float (&x)[kU][kE], ExponentScale c, int32_t piece, int32_t step) {
    float b = m;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float most = x[u][0];
#pragma unroll
      for (int e = 1; e < kE; ++e) most = __builtin_fmaxf(most, x[u][e]);
      if constexpr (kTop) {
        if (most > b) at = piece + u * step;
      }
      b = __builtin_fmaxf(b, most);
    }
    if constexpr (kTop) at = at < 0 ? piece : at;
    const float base = b == -__builtin_inff() ? 0.0f : kFar ? 0.5f * b : b;
    float t4[4] = {}, a4[4] = {};
#pragma unroll
    for (int i = 0; i < kU * kE; ++i) {
      const float v = x[i / kE][i % kE], t = (kFar ? __builtin_fmaf(v, 0.5f, -base) : v - base) * c.c;
      const float e = __builtin_amdgcn_exp2f(t);
      t4[i & 3] += e;
      if constexpr (kEnt) a4[i & 3] = __builtin_fmaf(e, __builtin_fmaxf(t, kLeastExponent), a4[i & 3]);
    }
    if (b != m) rescale(b, c);
    s += (double)((t4[0] + t4[1]) + (t4[2] + t4[3]));
    if constexpr (kEnt) a += (double)((a4[0] + a4[1]) + (a4[2] + a4[3]));
  }
  // Relative to M >= m; s and a of m = -inf are 0 (or NaN). With d the exponent of m, e t becomes
  // 2^d e (t + d).
  __device__ inline void rescale(float M, ExponentScale c) {
    if (m == M) return;
    const float d = c(m, M * c.half);
    const double by = (double)__builtin_amdgcn_exp2f(d);
    if constexpr (kEnt) a = by * __builtin_fma((double)__builtin_fmaxf(d, kLeastExponent), s, a);
    s *= by;
    m = M;
  }
};

template <int kW>
struct LogprobShared {
  float m[kW];
  double s[kW], a[kW];
};

// The workgroup's state from its threads', the same for every thread.
template <int kW, bool kEnt, bool kTop>
__device__ inline LogprobPart block_part(LogprobState<kEnt, kTop> st, ExponentScale c, LogprobShared<kW>& sh) {
  const uint32_t w = threadIdx.x / kWaveSize, lane = threadIdx.x & (kWaveSize - 1);
  st.rescale(wave_max(st.m), c);
  const double ws = wave_reduce(st.s, SumOp()), wa = kEnt ? wave_reduce(st.a, SumOp()) : 0.0;
  if (lane == 0) sh.m[w] = st.m, sh.s[w] = ws, sh.a[w] = wa;
  lds_barrier();
  LogprobState<kEnt, kTop> v;
  const uint32_t from = lane & 15u;
  static_assert(kW <= 16, "a partial for each lane of a row of 16");
  if (from < kW) v.m = sh.m[from], v.s = sh.s[from], v.a = sh.a[from];
  v.rescale(row16_reduce(v.m, [](float p, float q) { return __builtin_fmaxf(p, q); }), c);
  return {v.m, row16_reduce(v.s, SumOp()), kEnt ? row16_reduce(v.a, SumOp()) : 0.0};
}

// The first pieces of a row, kept in LDS from one pass over it to the next: `pieces` a thread.
template <int kThr>
struct HeldPieces {
  u32x4* at;
  int32_t pieces;
  __device__ inline void put(int64_t k, const u32x4& v) const {
    if (k < pieces) at[k * kThr + threadIdx.x] = v;  // uniform
  }
};
struct NothingHeld {
  __device__ inline void put(int64_t, const u32x4&) const {}
};

// A thread's state of row[lo, hi), lo a multiple of 8, in a workgroup of kThr threads. (32 float32
// elements in flight per thread instead of 16 spill where alternatives are kept, and gain nothing.)
template <int DT, int kThr, bool kEnt, bool kTop, bool kOnce, bool kFar, int kU, class Held>
__device__ inline LogprobState<kEnt, kTop> logprob_pass_of(const typename Row<DT>::Bits* row, int64_t lo, int64_t hi,
                                                           ExponentScale c, Held held) {
  constexpr int kE = Piece<DT>::kSize;  // kU of them in flight per thread
  constexpr int64_t kStep = kThr * kE;
  LogprobState<kEnt, kTop> st;
  int64_t at = lo + (int64_t)threadIdx.x * kE;
  for (int64_t base = lo; base < hi; base += kU * kStep, at += kU * kStep) {
    Piece<DT> v[kU];
    float x[kU][kE];
    const bool last = base + kU * kStep > hi;  // uniform
    if (!last) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
        v[u] = kOnce ? Piece<DT>::load_once(row + at + u * kStep) : Piece<DT>::load(row + at + u * kStep);
    } else {  // all at once too; -inf behind the end
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        v[u] = Piece<DT>::lowest();
        if (at + u * kStep + kE <= hi) v[u] = Piece<DT>::load(row + at + u * kStep);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      v[u].unpack(x[u]);
      held.put((base - lo) / kStep + u, v[u].v);
    }
    if (last) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (at + u * kStep < hi && at + u * kStep + kE > hi) load_part<DT>(row, at + u * kStep, hi, x[u]);
    }
    st.template add<kFar>(x, c, (int32_t)(at / kE), (int32_t)(kStep / kE));
  }
  if (lo + (int64_t)threadIdx.x * kE >= hi) st.at = -1;  // nothing of the row
  return st;
}

// Rows whose logits may be far apart are passed over again, by a function that is called: so the usual loop
// keeps a subtraction and its registers, and its loads do not wait for the temperature. (With both ways in
// the loop 256 rows of 151936 with 5 alternatives take 49 us instead of 24.2, with this one inlined 25.4.)
template <int DT, int kThr, bool kEnt, bool kTop, class Held>
__device__ __attribute__((noinline)) LogprobState<kEnt, kTop> logprob_far_pass(const typename Row<DT>::Bits* row,
                                                                               int64_t lo, int64_t hi, ExponentScale c,
                                                                               Held held) {
  return logprob_pass_of<DT, kThr, kEnt, kTop, false, true, 1>(row, lo, hi, c, held);
}
template <int DT, int kThr, bool kEnt, bool kTop, bool kOnce = false, class Held = NothingHeld>
__device__ inline LogprobState<kEnt, kTop> logprob_pass(const typename Row<DT>::Bits* row, int64_t lo, int64_t hi,
                                                        ExponentScale c, Held held = Held()) {
  auto st = logprob_pass_of<DT, kThr, kEnt, kTop, kOnce, false, 4>(row, lo, hi, c, held);
  if (__builtin_expect(__builtin_amdgcn_readfirstlane(c.half != 1.0f), 0))
    st = logprob_far_pass<DT, kThr, kEnt, kTop>(row, lo, hi, c, held);
  return st;
}

template <bool kEnt>
__device__ inline uint64_t state_key(const LogprobState<kEnt, true>& st) {
  return st.at < 0 ? 0 : top_key(st.m, (uint32_t)st.at);
}

// What a row's gradient is computed from; nothing when it has none.
struct LogprobRow {
  float m, s, M;
  bool ok;
};

// Status of row n before its logits are read; TSC_ROW_OK if they are to be read.
__device__ inline int32_t logprob_early_status(const LogprobArgs& a, int64_t n) {
  const int32_t t = a.tokens[n];
  if (t == -1) return TSC_ROW_NO_SUPPORT;
  return t < -1 || t >= a.V || !temperature_ok(a.T(n)) ? TSC_ROW_INVALID_PARAM : TSC_ROW_OK;
}

__device__ inline int32_t logprob_status(int32_t early, const LogprobPart& p) {
  if (early != TSC_ROW_OK) return early;
  if (!(p.s < __builtin_inf()) || !(p.m < __builtin_inff())) return TSC_ROW_NONFINITE;
  return p.m == -__builtin_inff() ? TSC_ROW_NO_SUPPORT : TSC_ROW_OK;
}

// Row n's outputs: `x` is the token's logit (thread 0), top the a.top first keys of a row that is OK.
// The first waves write, each thread one alternative; every thread gets the row.
__device__ inline LogprobRow logprob_finish(const LogprobArgs& a, int64_t n, int32_t status, const LogprobPart& p,
                                            float x, const uint64_t* top) {
  const bool ok = status == TSC_ROW_OK;
  const int32_t tid = (int32_t)threadIdx.x, last_wave = a.top > 0 ? (a.top - 1) / kWaveSize : 0;
  const double M = ok ? p.a / p.s * 0.69314718055994530942 : 0.0;
  if (tid / kWaveSize <= last_wave) {
    const double ln_s = ok ? log(p.s) : 0.0, inv_T = 1.0 / (double)a.T(n);
    if (tid < a.top) {
      const uint64_t key = ok ? top[tid] : 0;
      a.top_ids[n * a.top + tid] = ok ? key_id(key) : -1;
      a.top_logprobs[n * a.top + tid] =
          ok ? (float)(((double)key_value(key) - (double)p.m) * inv_T - ln_s) : __builtin_nanf("");
    }
    if (tid == 0) {
      const float none = a.tokens[n] == -1 ? 0.0f : __builtin_nanf("");
      a.logprobs[n] = ok ? (float)(((double)x - (double)p.m) * inv_T - ln_s) : none;
      if (a.entropy) a.entropy[n] = ok ? (float)(ln_s - M) : none;
      a.row_status[n] = (int8_t)status;
      if (a.stats) {
        float* st = a.stats + n * 4;
        st[0] = ok ? p.m : 0.0f, st[1] = ok ? (float)p.s : 1.0f;
        st[2] = a.entropy ? (float)M : __builtin_nanf("");  // asked for without the entropy: shows
        st[3] = ok ? 1.0f : 0.0f;
      }
    }
  }
  return {p.m, (float)p.s, (float)M, ok};
}

// A row per workgroup, read once. kOnce: nontemporally. 4096 rows of 151936 bfloat16 logits take 194 us,
// 6.4 TB/s, with the first alternative 194 to 204; 1024 of them with the entropy 58 us, 5.4 TB/s, and 66 in
// front of a backward pass, where they are not read nontemporally. What keeps it from a bare read's rate
// are its vector instructions: 8 an element, of which the exponential takes four times as long, fill about
// two thirds of the time. 256 rows, one to a CU: 18.8 us from memory (17.0 from the last-level cache), with
// the entropy 20.2 (18.2), which has too few waves a CU to hide the first and the last steps' latency.
template <int DT, int kThr, bool kEnt, bool kTop, bool kOnce>
__global__ void __launch_bounds__(kThr, 8) logprob_kernel(LogprobArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint64_t dyn_top[];
  __shared__ LogprobShared<kThr / kWaveSize> sh;
  __shared__ TopShared<kThr> top;
  const int64_t n = blockIdx.x;
  const int32_t early = logprob_early_status(a, n);
  LogprobPart p{-__builtin_inff(), 0.0, 0.0};
  const auto* row = (const typename Row<DT>::Bits*)a.logits + n * a.ld;
  float x = 0.0f;
  uint64_t key = 0;
  if (early == TSC_ROW_OK) {
    if (threadIdx.x == 0) x = Row<DT>::get(row + a.tokens[n]);
    const ExponentScale c = exponent_scale(a.T(n));
    const auto st = logprob_pass<DT, kThr, kEnt, kTop, kOnce>(row, 0, a.V, c);
    if constexpr (kTop) key = state_key(st);
    p = block_part<kThr / kWaveSize>(st, c, sh);
  }
  const int32_t status = logprob_status(early, p);
  const uint64_t* first = nullptr;
  if constexpr (kTop) {
    if (status == TSC_ROW_OK) {
      const TopLists<kThr> lists(dyn_top);
      top_collect<DT>(row, 0, a.V, key, a.top, lists, top);
      first = top_sort(lists.cand, a.top, top);
    }
  }
  logprob_finish(a, n, status, p, x, first);
}

// Few rows: a slice of a row per workgroup, then the rows from their slices. One row of 151936 bfloat16
// logits 7.0 us for both, 13.3 with 20 alternatives: two launches' latency and the selection's steps. (Joins
// by 256 threads instead of 1024 take 6.0 us against 5.0 with 20 alternatives, 16 against 7.6 with 128.)
template <int DT, bool kEnt, bool kTop>
__global__ void __launch_bounds__(kTopThreads, 8) logprob_slice_kernel(LogprobArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint64_t dyn_top[];
  __shared__ LogprobShared<kTopWaves> sh;
  __shared__ TopShared<kTopThreads> top;
  const int64_t item = blockIdx.x, n = item / a.slices, sl = item - n * a.slices;
  const int64_t lo = sl * a.slice_len, hi = lo + a.slice_len < a.V ? lo + a.slice_len : a.V;
  const auto* row = (const typename Row<DT>::Bits*)a.logits + n * a.ld;
  const ExponentScale c = exponent_scale(a.T(n));
  const auto st = logprob_pass<DT, kTopThreads, kEnt, kTop>(row, lo, hi, c);
  if (logprob_early_status(a, n) != TSC_ROW_OK) return;  // not looked at earlier: the row is on its way by now
  const LogprobPart p = block_part<kTopWaves>(st, c, sh);
  if (threadIdx.x == 0) a.parts[item] = p;
  if constexpr (kTop) {
    const TopLists<kTopThreads> lists(dyn_top);
    top_collect<DT>(row, lo, hi, state_key(st), a.top, lists, top);
    const uint64_t* first = top_sort(lists.cand, a.top, top);
    if ((int32_t)threadIdx.x < a.top) a.keys[item * a.top + threadIdx.x] = first[threadIdx.x];
  }
}

template <int DT, bool kEnt, bool kTop>
__global__ void __launch_bounds__(kTop ? kTopThreads : kWaveSize) logprob_join_kernel(LogprobArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint64_t dyn_top[];
  __shared__ TopShared<kTopThreads> top;
  const int64_t n = blockIdx.x;
  const int32_t early = logprob_early_status(a, n), lane = (int32_t)threadIdx.x & (kWaveSize - 1);
  LogprobPart p{-__builtin_inff(), 0.0, 0.0};
  float x = 0.0f;
  if (early == TSC_ROW_OK) {
    if (threadIdx.x == 0) x = Row<DT>::get((const typename Row<DT>::Bits*)a.logits + n * a.ld + a.tokens[n]);
    const ExponentScale c = exponent_scale(a.T(n));
    LogprobState<kEnt, kTop> st;
    if (lane < a.slices) {
      const LogprobPart q = a.parts[n * a.slices + lane];
      st.m = q.m, st.s = q.s, st.a = q.a;
    }
    st.rescale(wave_max(st.m), c);
    p = {st.m, wave_reduce(st.s, SumOp()), kEnt ? wave_reduce(st.a, SumOp()) : 0.0};
  }
  const int32_t status = logprob_status(early, p);
  const uint64_t* first = nullptr;
  if constexpr (kTop) {
    if (status == TSC_ROW_OK) {
      const TopLists<kTopThreads> lists(dyn_top);
      top_collect_keys(a.keys + n * a.slices * a.top, a.slices, a.top, lists, top);
      first = top_sort(lists.cand, a.top, top);
    }
  }
  logprob_finish(a, n, status, p, x, first);
}

// ---- the gradient ----------------------------------------------------------------------------------

// dx_i = again (2^t (alpha + beta t) + hits) with t the exponent of x_i; the hits are a / T at the token and
// u_j / T at the alternatives, of this T. T again is the row's temperature, `again` a power of two: 1
// from 2^-80 to 2^80. Past that the coefficients would leave float32, or lose digits, for temperatures
// whose gradients do not (an element of numerator 0 would get 0 * inf). With again at most 2^40 the sums
// stay below 2^127 for upstream gradients up to 2^32; up to 2^20 what the roundings of a hit and of the
// stream leave where they cancel, 2^-22 of the hit, is finite too.
struct LogprobCoef {
  float half_m;
  ExponentScale c;
  float alpha, beta, T, again;
};

__device__ inline LogprobCoef logprob_coef(const LogprobRow& r, float T, float total, float b) {
  const float again = T < 0x1p-80f ? 0x1p40f : T > 0x1p80f ? 0x1p-40f : 1.0f;
  const float scaled = T * again, g = 1.0f / (r.s * scaled);
  const ExponentScale c = exponent_scale(T);
  return {r.m * c.half, c, (b == 0.0f ? -total : __builtin_fmaf(b, r.M, -total)) * g,
          -b * 0.69314718055994531f * g, scaled, again};
}

template <int kE>
__device__ inline void logprob_grad_of(float (&x)[kE], const LogprobCoef& k) {
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const float t = __builtin_fmaxf(k.c(x[e], k.half_m), kLeastExponent);
    x[e] = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(k.beta, t, k.alpha);
  }
}

// The piece's gradient. beside(at, x) adds the hits among the elements from `at` on.
template <int kE, class Beside>
__device__ inline void logprob_grad_piece(float (&x)[kE], int64_t at, const LogprobCoef& k, Beside& beside) {
  logprob_grad_of(x, k);
  beside(at, x);
#pragma unroll
  for (int e = 0; e < kE; ++e) x[e] *= k.again;
}

// Writes the gradient of row[lo, hi), kU pieces in flight per thread.
template <int DT, int kThr, int kU, class Beside>
__device__ inline void logprob_grad_pass(const typename Row<DT>::Bits* row, typename Row<DT>::Bits* out, int64_t lo,
                                         int64_t hi, const LogprobCoef& k, Beside beside) {
  constexpr int kE = Piece<DT>::kSize;
  constexpr int64_t kStep = kThr * kE;
  int64_t at = lo + (int64_t)threadIdx.x * kE;
  int64_t base = lo;
  for (; base + kU * kStep <= hi; base += kU * kStep, at += kU * kStep) {
    Piece<DT> v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) v[u] = Piece<DT>::load_once(row + at + u * kStep);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float x[kE];
      v[u].unpack(x);
      logprob_grad_piece(x, at + u * kStep, k, beside);
      Piece<DT>::store(out + at + u * kStep, x);
    }
  }
  for (; at < hi; at += kStep) {
    float x[kE];
    load_piece<DT>(row, at, hi, x);
    logprob_grad_piece(x, at, k, beside);
    store_piece<DT>(out, at, hi, x);
  }
}

// x[i] += v: without an index into registers.
template <int kE>
__device__ inline void add_at(float (&x)[kE], uint32_t i, float v) {
#pragma unroll
  for (uint32_t e = 0; e < kE; ++e) x[e] += e == i ? v : 0.0f;
}

constexpr int kLogprobGradThreads = 256, kLogprobGradPieces = 4;  // in flight per thread
constexpr int64_t kLogprobGradSegment = 8192;  // elements, or more to bound the grid

// A segment of a row per workgroup: 83 us for 1024 rows of 151936 bfloat16 logits, a tenth of them padding,
// 7.1 TB/s behind the L2; 93 us without padding.
// (Segments of 16384 elements 88, of 4096 with two pieces in flight 92; reversing the rows' order, so
// that those read last come first, 84.) Pieces that the entries of a list join are looked for, so that
// each result is rounded and written once. With alternatives (kTop), a bit for each 8 elements of the segment
// that hold one says where the list is looked through.
template <int DT, bool kTop>
__global__ void __launch_bounds__(kLogprobGradThreads, 8) logprob_grad_kernel(LogprobArgs a) {
  constexpr int kThr = kLogprobGradThreads, kE = Piece<DT>::kSize;
  using B = typename Row<DT>::Bits;
  __shared__ uint32_t bits[kTop ? kMaxSegment / 8 / 32 : 1];
  __shared__ int32_t ids[kTop ? kTopMost : 1];
  __shared__ float ups[kTop ? kTopMost : 1];
  const int64_t item = blockIdx.x, n = item / a.segments;
  const int64_t lo = (item - n * a.segments) * a.seg_len;
  const int64_t hi = lo + a.seg_len < a.V ? lo + a.seg_len : a.V;
  B* out = (B*)a.grad + n * a.V;
  const float* st = a.stats + n * 4;
  const LogprobRow r{st[0], st[1], a.grad_entropy ? st[2] : 0.0f, st[3] != 0.0f};
  if (!r.ok) {
    fill_zero<DT, kThr>(out, lo, hi);
    return;
  }
  const B* row = (const B*)a.logits + n * a.ld;
  const float T = a.T(n), up = a.grad_logprobs ? a.grad_logprobs[n] : 0.0f;
  const int64_t token = a.tokens[n];
  float total = up;
  if constexpr (kTop) {
    const int words = (int)((hi - lo + 255) / 256);
    for (int i = (int)threadIdx.x; i < words; i += kThr) bits[i] = 0;
    const int i = (int)threadIdx.x;
    if (i < a.top) ids[i] = a.top_ids[n * a.top + i], ups[i] = a.grad_top[n * a.top + i];
    __syncthreads();
    for (int j = 0; j < a.top; ++j) total += ups[j];
    if (i < a.top && ids[i] >= lo && ids[i] < hi) {
      const uint32_t chunk = (uint32_t)(ids[i] - lo) >> 3;
      atomicOr(&bits[chunk >> 5], 1u << (chunk & 31));
    }
    __syncthreads();
  }
  const LogprobCoef k = logprob_coef(r, T, total, a.grad_entropy ? a.grad_entropy[n] : 0.0f);
  const float hit = up / k.T;
  logprob_grad_pass<DT, kThr, kLogprobGradPieces>(row, out, lo, hi, k, [&](int64_t at, float(&x)[kE]) {
    if ((uint64_t)(token - at) < (unsigned)kE) add_at(x, (uint32_t)(token - at), hit);
    if constexpr (kTop) {
      const uint32_t chunk = (uint32_t)(at - lo) >> 3;
      if ((bits[chunk >> 5] >> (chunk & 31)) & 1u) {
        for (int j = 0; j < a.top; ++j)
          if ((uint64_t)(ids[j] - at) < (unsigned)kE) add_at(x, (uint32_t)(ids[j] - at), ups[j] / k.T);
      }
    }
  });
}

// Values and gradient, a row per workgroup: the second reading of the row comes from LDS as far as
// that goes, and from the last-level cache while the rows in flight fit there. 512 rows of 262144
// bfloat16 logits, a twentieth of them padding, 120 to 128 us, 724 MB behind the L2 at 5.7 to 6.0 TB/s; in one
// run 122, and without the LDS 126. (With it, one workgroup to
// a CU no longer pays where the rows exceed the cache: 1024 such rows 270 us, in pairs 253.)
template <int DT, int kThr, bool kEnt>
__global__ void __launch_bounds__(kThr, 8) logprob_fused_kernel(LogprobArgs a) {
  using B = typename Row<DT>::Bits;
  extern __shared__ __attribute__((aligned(16))) uint64_t dyn_top[];
  __shared__ LogprobShared<kThr / kWaveSize> sh;
  constexpr int kE = Piece<DT>::kSize;
  const HeldPieces<kThr> held{reinterpret_cast<u32x4*>(dyn_top), a.held};
  const int64_t n = blockIdx.x;
  const int32_t early = logprob_early_status(a, n);
  LogprobPart p{-__builtin_inff(), 0.0, 0.0};
  const B* row = (const B*)a.logits + n * a.ld;
  B* out = (B*)a.grad + n * a.V;
  float x = 0.0f;
  const float T = a.T(n);
  const ExponentScale c = exponent_scale(T);
  if (early == TSC_ROW_OK) {
    if (threadIdx.x == 0) x = Row<DT>::get(row + a.tokens[n]);
    p = block_part<kThr / kWaveSize>(logprob_pass<DT, kThr, kEnt, false>(row, 0, a.V, c, held), c, sh);
  }
  const LogprobRow r = logprob_finish(a, n, logprob_status(early, p), p, x, nullptr);
  if (!r.ok) {
    fill_zero<DT, kThr>(out, 0, a.V);
    return;
  }
  const float up = a.grad_logprobs[n];
  const int64_t token = a.tokens[n];
  const LogprobCoef k = logprob_coef(r, T, up, a.grad_entropy ? a.grad_entropy[n] : 0.0f);
  const float hit = up / k.T;
  auto beside = [&](int64_t at, float(&v)[kE]) {
    if ((uint64_t)(token - at) < (unsigned)kE) add_at(v, (uint32_t)(token - at), hit);
  };
  // Whole steps of the workgroup that every thread holds.
  int64_t lo = 0;
  for (int32_t i = 0; i < a.held && lo + kThr * kE <= a.V; ++i, lo += kThr * kE) {
    float v[kE];
    Piece<DT>{held.at[i * kThr + threadIdx.x]}.unpack(v);
    const int64_t at = lo + (int64_t)threadIdx.x * kE;
    logprob_grad_piece(v, at, k, beside);
    Piece<DT>::store(out + at, v);
  }
  logprob_grad_pass<DT, kThr, 4>(row, out, lo, a.V, k, beside);
}

}  // namespace tsc
