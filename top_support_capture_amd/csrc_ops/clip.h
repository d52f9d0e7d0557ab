// The norm of many tensors taken together, and tensors scaled down to a norm.
//
// A launch covers up to a table of tensors, which travels in the kernel's arguments: nothing is
// copied to the device beforehand, and a captured launch keeps its table. The tensors' elements,
// cut into units of kClipUnit, are dealt to the workgroups in one contiguous span each, whatever
// the tensors' sizes.
#pragma once

#include "row_stats.h"

namespace tsc {

constexpr int kClipThreads = 512;
constexpr int kClipWaves = kClipThreads / kWaveSize;
constexpr int64_t kClipUnit = kClipThreads * 8;  // elements
constexpr int kClipGroups = 1024;                // at most, of one launch
constexpr int kClipInFlight = 4;                 // chunks of 8 elements a thread

// kN tensors, the table's size bounded by the 4 KB that a kernel's arguments may take.
template <int kN>
struct ClipTable {
  static constexpr int kSize = kN;
  const void* src[kN];
  int64_t numel[kN];
  uint32_t first[kN + 1];  // units before each tensor; the last: all
  uint32_t f32[(kN + 31) / 32];
  int32_t n;
  __device__ inline bool is_f32(int t) const { return (f32[t >> 5] >> (t & 31)) & 1u; }
};

template <int kN>
struct ClipOutTable : ClipTable<kN> {
  void* dst[kN];
  uint32_t dst_f32[(kN + 31) / 32];
  __device__ inline bool to_f32(int t) const { return (dst_f32[t >> 5] >> (t & 31)) & 1u; }
};

using NormTable = ClipTable<184>;
using ScaleTable = ClipOutTable<136>;

// visit(t, lo, hi) for the parts of tensors in this workgroup's span of units, in order or from
// the last to the first.
template <bool kBackwards, class Table, class Visit>
__device__ inline void visit_span(const Table& a, Visit visit) {
  const uint32_t units = a.first[a.n];
  uint32_t u0 = (uint32_t)((uint64_t)blockIdx.x * units / gridDim.x);
  uint32_t u1 = (uint32_t)((uint64_t)(blockIdx.x + 1) * units / gridDim.x);
  if (u0 == u1) return;
  const uint32_t at = kBackwards ? u1 - 1 : u0;
  int t = 0;  // the last tensor that begins at or before unit `at`
  for (int below = a.n; below - t > 1;) {
    const int mid = (t + below) >> 1;
    if (a.first[mid] <= at) t = mid;
    else below = mid;
  }
  while (u0 < u1) {
    const uint32_t b = a.first[t], e = a.first[t + 1];
    const uint32_t lo = u0 > b ? u0 : b, hi = u1 < e ? u1 : e;
    if (lo < hi) {
      const int64_t end = (int64_t)(hi - b) * kClipUnit;
      visit(t, (int64_t)(lo - b) * kClipUnit, end < a.numel[t] ? end : a.numel[t]);
    }
    if (kBackwards) u1 = lo < u1 ? lo : u1, --t;
    else u0 = hi > u0 ? hi : u0, ++t;
  }
}

// Squares in float64: exact for float32 values, and without overflow or underflow. (One float64
// multiply-add an element keeps up with the loads.)
template <int DT>
__device__ inline double sum_squares(const void* tensor, int64_t lo, int64_t hi) {
  const auto* x = (const typename Row<DT>::Bits*)tensor;
  double s[2] = {0.0, 0.0};
  auto add = [&](const float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e & 1] = __builtin_fma((double)v[e], (double)v[e], s[e & 1]);
  };
  const int64_t first = (int64_t)threadIdx.x * 8;
  int64_t at = lo;
  for (; at + kClipInFlight * kClipUnit <= hi; at += kClipInFlight * kClipUnit) {
    typename Row<DT>::Chunk c[kClipInFlight];
#pragma unroll
    for (int u = 0; u < kClipInFlight; ++u) c[u] = Row<DT>::load(x + at + u * kClipUnit + first);
#pragma unroll
    for (int u = 0; u < kClipInFlight; ++u) {
      float v[8];
      Row<DT>::unpack(c[u], v);
      add(v);
    }
  }
  for (at += first; at < hi; at += kClipUnit) {
    if (at + 8 <= hi) {
      float v[8];
      Row<DT>::unpack(Row<DT>::load(x + at), v);
      add(v);
    } else {
      for (int64_t i = at; i < hi; ++i) {
        const double v = (double)Row<DT>::get(x + i);
        s[0] = __builtin_fma(v, v, s[0]);
      }
    }
  }
  return s[0] + s[1];
}

// The sum over the workgroup, the same for every thread.
__device__ inline double clip_block_sum(double s, double* sh) {
  s = wave_reduce(s, SumOp());
  if ((threadIdx.x & (kWaveSize - 1)) == 0) sh[threadIdx.x / kWaveSize] = s;
  lds_barrier();
  s = sh[0];
#pragma unroll
  for (int i = 1; i < kClipWaves; ++i) s += sh[i];
  return s;
}

// A partial sum for each workgroup: a fixed order of additions, whatever order they run in.
__global__ void __launch_bounds__(kClipThreads, 8) clip_norm_kernel(NormTable a, double* partials) {
  __shared__ double sh[kClipWaves];
  double s = 0.0;
  visit_span<false>(a, [&](int t, int64_t lo, int64_t hi) {
    s += a.is_f32(t) ? sum_squares<TSC_DTYPE_F32>(a.src[t], lo, hi) : sum_squares<TSC_DTYPE_BF16>(a.src[t], lo, hi);
  });
  s = clip_block_sum(s, sh);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

__device__ inline float norm_of(const double* partials, int32_t n, double* sh) {
  double s = 0.0;
  for (int32_t i = (int32_t)threadIdx.x; i < n; i += kClipThreads) s += partials[i];
  return (float)sqrt(clip_block_sum(s, sh));
}

__global__ void __launch_bounds__(kClipThreads, 8) clip_join_kernel(const double* partials, int32_t n, float* norm) {
  __shared__ double sh[kClipWaves];
  const float v = norm_of(partials, n, sh);
  if (threadIdx.x == 0) *norm = v;
}

template <int DT, int OT>
__device__ inline void scale_span(const void* tensor, void* out, int64_t lo, int64_t hi, float by) {
  const auto* x = (const typename Row<DT>::Bits*)tensor;
  auto* y = (typename Row<OT>::Bits*)out;
  const int64_t first = (int64_t)threadIdx.x * 8;
  // From the end: what the norm's pass has read last is still in the last-level cache.
  int64_t end = lo + (hi - lo) / (kClipInFlight * kClipUnit) * (kClipInFlight * kClipUnit);
  for (int64_t at = end + first; at < hi; at += kClipUnit) {
    if (at + 8 <= hi) {
      float v[8];
      Row<DT>::unpack(Row<DT>::load(x + at), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= by;
      Row<OT>::store(y + at, v);
    } else {
      for (int64_t i = at; i < hi; ++i) Row<OT>::put(y + i, Row<DT>::get(x + i) * by);
    }
  }
  while (end > lo) {
    end -= kClipInFlight * kClipUnit;
    typename Row<DT>::Chunk c[kClipInFlight];
#pragma unroll
    for (int u = 0; u < kClipInFlight; ++u) c[u] = Row<DT>::load(x + end + u * kClipUnit + first);
#pragma unroll
    for (int u = 0; u < kClipInFlight; ++u) {
      float v[8];
      Row<DT>::unpack(c[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= by;
      Row<OT>::store(y + end + u * kClipUnit + first, v);
    }
  }
}

// The factor of a norm; values stay as they are below max_norm and where the norm is no number.
__device__ inline float clip_factor(float norm, float max_norm) {
  return norm > max_norm && norm < __builtin_inff() ? max_norm / norm : 1.0f;
}

// Scales by the norm of `n` partial sums, which workgroup 0 writes to `norm_out` (if not null), or
// by *norm_in.
struct ClipNorm {
  const double* partials;
  int32_t n;
  float* norm_out;
  const float* norm_in;
  float max_norm;
  int32_t in_place;  // nothing to do where the factor is 1
};

__global__ void __launch_bounds__(kClipThreads, 8) clip_scale_kernel(ScaleTable a, ClipNorm c) {
  __shared__ double sh[kClipWaves];
  const float norm = c.norm_in ? *c.norm_in : norm_of(c.partials, c.n, sh);
  if (c.norm_out && blockIdx.x == 0 && threadIdx.x == 0) *c.norm_out = norm;
  const float by = clip_factor(norm, c.max_norm);
  if (by == 1.0f && c.in_place) return;
  visit_span<true>(a, [&](int t, int64_t lo, int64_t hi) {
    const void* x = a.src[t];
    void* y = a.dst[t];
    if (a.is_f32(t))
      a.to_f32(t) ? scale_span<TSC_DTYPE_F32, TSC_DTYPE_F32>(x, y, lo, hi, by)
                  : scale_span<TSC_DTYPE_F32, TSC_DTYPE_BF16>(x, y, lo, hi, by);
    else
      a.to_f32(t) ? scale_span<TSC_DTYPE_BF16, TSC_DTYPE_F32>(x, y, lo, hi, by)
                  : scale_span<TSC_DTYPE_BF16, TSC_DTYPE_BF16>(x, y, lo, hi, by);
  });
}

}  // namespace tsc
