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

// State of a row or a part of it: the maximum, the sum of the numerators e = 2^t, t = (x - m) c,
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
  __device__ inline float T(int64_t n) const { return temperature ? temperature[n] : 1.0f; }
};

// Exponents below this have numerator 0; as a factor it keeps 0 * -inf out.
constexpr float kLeastExponent = -200.0f;

// A thread's running state: sums of up to 32 terms in float32, all else in float64. `at` is the
// first chunk (kTop only) that reached the maximum, -1 before the first one.
template <bool kEnt, bool kTop>
struct LogprobState {
  float m = -__builtin_inff();
  int32_t at = -1;
  double s = 0.0, a = 0.0;
  // U chunks of 8 elements, the first chunk's index and the distance from one to the next.
  template <int U>
  __device__ inline void add(const float (&x)[U * 8], float c, int32_t chunk, int32_t step) {
    float b = m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* v = x + u * 8;
      const float most = __builtin_fmaxf(
          __builtin_fmaxf(__builtin_fmaxf(v[0], v[1]), __builtin_fmaxf(v[2], v[3])),
          __builtin_fmaxf(__builtin_fmaxf(v[4], v[5]), __builtin_fmaxf(v[6], v[7])));
      if constexpr (kTop) {
        if (most > b) at = chunk + u * step;
      }
      b = __builtin_fmaxf(b, most);
    }
    if constexpr (kTop) at = at < 0 ? chunk : at;
    const float base = b == -__builtin_inff() ? 0.0f : b;
    float t4[4] = {}, a4[4] = {};
#pragma unroll
    for (int i = 0; i < U * 8; ++i) {
      const float t = (x[i] - base) * c, e = __builtin_amdgcn_exp2f(t);
      t4[i & 3] += e;
      if constexpr (kEnt) a4[i & 3] = __builtin_fmaf(e, __builtin_fmaxf(t, kLeastExponent), a4[i & 3]);
    }
    if (b != m) rescale(b, c);
    s += (double)((t4[0] + t4[1]) + (t4[2] + t4[3]));
    if constexpr (kEnt) a += (double)((a4[0] + a4[1]) + (a4[2] + a4[3]));
  }
  // Relative to M >= m; s and a of m = -inf are 0 (or NaN). With d = (m - M) c, e t becomes
  // 2^d e (t + d).
  __device__ inline void rescale(float M, float c) {
    if (m == M) return;
    const float d = (m - M) * c;
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
__device__ inline LogprobPart block_part(LogprobState<kEnt, kTop> st, float c, LogprobShared<kW>& sh) {
  const uint32_t w = threadIdx.x / kWaveSize, lane = threadIdx.x & (kWaveSize - 1);
  st.rescale(wave_max(st.m), c);
  const double ws = wave_reduce(st.s, SumOp()), wa = kEnt ? wave_reduce(st.a, SumOp()) : 0.0;
  if (lane == 0) sh.m[w] = st.m, sh.s[w] = ws, sh.a[w] = wa;
  lds_barrier();
  LogprobState<kEnt, kTop> v;
  const uint32_t from = lane & (kW - 1);
  v.m = sh.m[from], v.s = sh.s[from], v.a = sh.a[from];
  static_assert(kW == 16, "one partial for each lane of a row of 16");
  v.rescale(row16_reduce(v.m, [](float p, float q) { return __builtin_fmaxf(p, q); }), c);
  return {v.m, row16_reduce(v.s, SumOp()), kEnt ? row16_reduce(v.a, SumOp()) : 0.0};
}

// A thread's state of row[lo, hi), lo a multiple of 8, in a workgroup of kTopThreads threads.
template <int DT, bool kEnt, bool kTop>
__device__ inline LogprobState<kEnt, kTop> logprob_pass(const typename Row<DT>::Bits* row, int64_t lo, int64_t hi,
                                                        float c) {
  constexpr int kU = 4;  // chunks in flight per thread
  constexpr int64_t kStep = kTopRound;
  LogprobState<kEnt, kTop> st;
  const int64_t first = (int64_t)threadIdx.x * 8;
  int64_t base = lo;
  for (; base + kU * kStep <= hi; base += kU * kStep) {
    typename Row<DT>::Chunk v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) v[u] = Row<DT>::load(row + base + u * kStep + first);
    float f[kU * 8];
#pragma unroll
    for (int u = 0; u < kU; ++u) Row<DT>::unpack(v[u], reinterpret_cast<float(&)[8]>(f[u * 8]));
    st.template add<kU>(f, c, (int32_t)((base + first) >> 3), (int32_t)(kStep >> 3));
  }
  for (int64_t at = base + first; at < hi; at += kStep) {
    float x[8];
    load8<DT>(row, at, hi, x);
    st.template add<1>(x, c, (int32_t)(at >> 3), 0);
  }
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

// Row n's outputs but the alternatives: thread 0 writes, every thread gets the row. `x` is the
// token's logit.
__device__ inline LogprobRow logprob_finish(const LogprobArgs& a, int64_t n, int32_t status, const LogprobPart& p,
                                            float x) {
  if (status == TSC_ROW_OK) {
    if (!(p.s < __builtin_inf()) || !(p.m < __builtin_inff())) status = TSC_ROW_NONFINITE;
    else if (p.m == -__builtin_inff()) status = TSC_ROW_NO_SUPPORT;
  }
  const bool ok = status == TSC_ROW_OK;
  const double M = ok ? p.a / p.s * 0.69314718055994530942 : 0.0;
  if (threadIdx.x == 0) {
    const bool padding = a.tokens[n] == -1;
    const double ln_s = ok ? log(p.s) : 0.0;
    const float none = padding ? 0.0f : __builtin_nanf("");
    a.logprobs[n] = ok ? (float)(((double)x - (double)p.m) / (double)a.T(n) - ln_s) : none;
    if (a.entropy) a.entropy[n] = ok ? (float)(ln_s - M) : none;
    a.row_status[n] = (int8_t)status;
    if (a.stats) {
      float* st = a.stats + n * 4;
      st[0] = ok ? p.m : 0.0f, st[1] = ok ? (float)p.s : 1.0f;
      st[2] = a.entropy ? (float)M : __builtin_nanf("");  // asked for without the entropy: shows
      st[3] = ok ? 1.0f : 0.0f;
    }
  }
  return {p.m, (float)p.s, (float)M, ok};
}

// The alternatives of a row that is not OK.
__device__ inline void logprob_no_top(const LogprobArgs& a, int64_t n) {
  for (int32_t i = (int32_t)threadIdx.x; i < a.top; i += kTopThreads)
    a.top_ids[n * a.top + i] = -1, a.top_logprobs[n * a.top + i] = __builtin_nanf("");
}

// Place r of row n's alternatives.
__device__ inline void logprob_put_top(const LogprobArgs& a, int64_t n, const LogprobPart& p, int r, uint64_t key) {
  a.top_ids[n * a.top + r] = key_id(key);
  a.top_logprobs[n * a.top + r] =
      (float)(((double)key_value(key) - (double)p.m) / (double)a.T(n) - log(p.s));
}

// A row per workgroup, read once.
template <int DT, bool kEnt, bool kTop>
__global__ void __launch_bounds__(kTopThreads, 8) logprob_kernel(LogprobArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint64_t dyn_top[];
  __shared__ LogprobShared<kTopWaves> sh;
  __shared__ TopShared top;
  const int64_t n = blockIdx.x;
  const int32_t status = logprob_early_status(a, n);
  LogprobPart p{-__builtin_inff(), 0.0, 0.0};
  const auto* row = (const typename Row<DT>::Bits*)a.logits + n * a.ld;
  float x = 0.0f;
  uint64_t key = 0;
  if (status == TSC_ROW_OK) {
    if (threadIdx.x == 0) x = Row<DT>::get(row + a.tokens[n]);
    const float c = plain_scale(a.T(n));
    const auto st = logprob_pass<DT, kEnt, kTop>(row, 0, a.V, c);
    if constexpr (kTop) key = state_key(st);
    p = block_part<kTopWaves>(st, c, sh);
  }
  const LogprobRow r = logprob_finish(a, n, status, p, x);
  if constexpr (kTop) {
    if (!r.ok) {
      logprob_no_top(a, n);
      return;
    }
    const TopLists lists(dyn_top);
    top_collect<DT>(row, 0, a.V, key, a.top, lists, top);
    top_emit(lists.cand, a.top, top, [&](int at, uint64_t k) { logprob_put_top(a, n, p, at, k); });
  }
}

// Few rows: a slice of a row per workgroup, then the rows from their slices.
template <int DT, bool kEnt, bool kTop>
__global__ void __launch_bounds__(kTopThreads, 8) logprob_slice_kernel(LogprobArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint64_t dyn_top[];
  __shared__ LogprobShared<kTopWaves> sh;
  __shared__ TopShared top;
  const int64_t item = blockIdx.x, n = item / a.slices, sl = item - n * a.slices;
  if (logprob_early_status(a, n) != TSC_ROW_OK) return;
  const int64_t lo = sl * a.slice_len, hi = lo + a.slice_len < a.V ? lo + a.slice_len : a.V;
  const auto* row = (const typename Row<DT>::Bits*)a.logits + n * a.ld;
  const float c = plain_scale(a.T(n));
  const auto st = logprob_pass<DT, kEnt, kTop>(row, lo, hi, c);
  const LogprobPart p = block_part<kTopWaves>(st, c, sh);
  if (threadIdx.x == 0) a.parts[item] = p;
  if constexpr (kTop) {
    const TopLists lists(dyn_top);
    top_collect<DT>(row, lo, hi, state_key(st), a.top, lists, top);
    top_emit(lists.cand, a.top, top, [&](int at, uint64_t k) { a.keys[item * a.top + at] = k; });
  }
}

template <int DT, bool kEnt, bool kTop>
__global__ void __launch_bounds__(kTop ? kTopThreads : kWaveSize) logprob_join_kernel(LogprobArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint64_t dyn_top[];
  __shared__ TopShared top;
  const int64_t n = blockIdx.x;
  const int32_t status = logprob_early_status(a, n), lane = (int32_t)threadIdx.x & (kWaveSize - 1);
  LogprobPart p{-__builtin_inff(), 0.0, 0.0};
  float x = 0.0f;
  if (status == TSC_ROW_OK) {
    if (threadIdx.x == 0) x = Row<DT>::get((const typename Row<DT>::Bits*)a.logits + n * a.ld + a.tokens[n]);
    const float c = plain_scale(a.T(n));
    LogprobState<kEnt, kTop> st;
    if (lane < a.slices) {
      const LogprobPart q = a.parts[n * a.slices + lane];
      st.m = q.m, st.s = q.s, st.a = q.a;
    }
    st.rescale(wave_max(st.m), c);
    p = {st.m, wave_reduce(st.s, SumOp()), kEnt ? wave_reduce(st.a, SumOp()) : 0.0};
  }
  const LogprobRow r = logprob_finish(a, n, status, p, x);
  if constexpr (kTop) {
    if (!r.ok) {
      logprob_no_top(a, n);
      return;
    }
    const TopLists lists(dyn_top);
    top_collect_keys(a.keys + n * a.slices * a.top, a.slices * a.top, a.top, lists, top);
    top_emit(lists.cand, a.top, top, [&](int at, uint64_t k) { logprob_put_top(a, n, p, at, k); });
  }
}

// ---- the gradient ----------------------------------------------------------------------------------

// dx_i = 2^t (alpha + beta t) with t = (x_i - m) c, plus `hit` at the token and u_j / T at the
// alternatives.
struct LogprobCoef {
  float m, c, alpha, beta;
};

__device__ inline LogprobCoef logprob_coef(const LogprobRow& r, float T, float total, float b) {
  const float g = 1.0f / (r.s * T);
  return {r.m, plain_scale(T), (b == 0.0f ? -total : __builtin_fmaf(b, r.M, -total)) * g, -b * 0.69314718055994531f * g};
}

__device__ inline void logprob_grad8(float (&x)[8], const LogprobCoef& k) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = __builtin_fmaxf((x[e] - k.m) * k.c, kLeastExponent);
    x[e] = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(k.beta, t, k.alpha);
  }
}

// Writes the gradient of row[lo, hi). at_chunk(at, x) adds what stands beside the stream to the
// chunk from `at` on.
template <int DT, int kThr, class AtChunk>
__device__ inline void logprob_grad_pass(const typename Row<DT>::Bits* row, typename Row<DT>::Bits* out, int64_t lo,
                                         int64_t hi, const LogprobCoef& k, AtChunk at_chunk) {
  constexpr int kU = DT == TSC_DTYPE_BF16 ? 4 : 2;  // chunks in flight per thread
  constexpr int64_t kStep = (int64_t)kThr * 8;
  const int64_t first = (int64_t)threadIdx.x * 8;
  int64_t base = lo;
  for (; base + kU * kStep <= hi; base += kU * kStep) {
    typename Row<DT>::Chunk v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) v[u] = Row<DT>::load_once(row + base + u * kStep + first);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float x[8];
      Row<DT>::unpack(v[u], x);
      logprob_grad8(x, k);
      at_chunk(base + u * kStep + first, x);
      Row<DT>::store(out + base + u * kStep + first, x);
    }
  }
  for (int64_t at = base + first; at < hi; at += kStep) {
    float x[8];
    load8<DT>(row, at, hi, x);
    logprob_grad8(x, k);
    at_chunk(at, x);
    store8<DT>(out, at, hi, x);
  }
}

// x[i] += v, i in [0, 8): without an index into registers.
__device__ inline void add_at(float (&x)[8], uint32_t i, float v) {
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e) x[e] += e == i ? v : 0.0f;
}

constexpr int kLogprobGradThreads = 256;

// A segment of a row per workgroup. With alternatives (kTop), a bit for each chunk of the segment
// that holds one says where the list is looked through.
template <int DT, bool kTop>
__global__ void __launch_bounds__(kLogprobGradThreads, 8) logprob_grad_kernel(LogprobArgs a) {
  constexpr int kThr = kLogprobGradThreads;
  using B = typename Row<DT>::Bits;
  __shared__ uint32_t bits[kTop ? kMaxSegment / 8 / 32 : 1];
  __shared__ int32_t ids[kTop ? kTopMost : 1];
  __shared__ float ups[kTop ? kTopMost : 1];
  const int64_t n = blockIdx.x / a.segments;
  const int64_t lo = (blockIdx.x - n * a.segments) * a.seg_len;
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
  const float hit = up / T;
  logprob_grad_pass<DT, kThr>(row, out, lo, hi, k, [&](int64_t at, float(&x)[8]) {
    if ((uint64_t)(token - at) < 8u) add_at(x, (uint32_t)(token - at), hit);
    if constexpr (kTop) {
      const uint32_t chunk = (uint32_t)(at - lo) >> 3;
      if ((bits[chunk >> 5] >> (chunk & 31)) & 1u) {
        for (int j = 0; j < a.top; ++j)
          if ((uint64_t)(ids[j] - at) < 8u) add_at(x, (uint32_t)(ids[j] - at), ups[j] / T);
      }
    }
  });
}

// Values and gradient, a row per workgroup: the second reading of the row comes from the last-level
// cache while the rows in flight fit there.
template <int DT, bool kEnt>
__global__ void __launch_bounds__(kTopThreads, 8) logprob_fused_kernel(LogprobArgs a) {
  using B = typename Row<DT>::Bits;
  __shared__ LogprobShared<kTopWaves> sh;
  const int64_t n = blockIdx.x;
  const int32_t status = logprob_early_status(a, n);
  LogprobPart p{-__builtin_inff(), 0.0, 0.0};
  const B* row = (const B*)a.logits + n * a.ld;
  B* out = (B*)a.grad + n * a.V;
  float x = 0.0f;
  const float T = a.T(n), c = plain_scale(T);
  if (status == TSC_ROW_OK) {
    if (threadIdx.x == 0) x = Row<DT>::get(row + a.tokens[n]);
    p = block_part<kTopWaves>(logprob_pass<DT, kEnt, false>(row, 0, a.V, c), c, sh);
  }
  const LogprobRow r = logprob_finish(a, n, status, p, x);
  if (!r.ok) {
    fill_zero<DT, kTopThreads>(out, 0, a.V);
    return;
  }
  const float up = a.grad_logprobs[n], hit = up / T;
  const int64_t token = a.tokens[n];
  const LogprobCoef k = logprob_coef(r, T, up, a.grad_entropy ? a.grad_entropy[n] : 0.0f);
  logprob_grad_pass<DT, kTopThreads>(row, out, 0, a.V, k, [&](int64_t at, float(&v)[8]) {
    if ((uint64_t)(token - at) < 8u) add_at(v, (uint32_t)(token - at), hit);
  });
}

}  // namespace tsc
