// Distillation of a student's logits from a teacher's top logits. With S a row's teacher ids,
// p = softmax over S of the teacher's values and q the student's softmax over the vocabulary,
//     loss = sum_{i in S} p_i (ln p_i - ln q_i),   dloss/dx_j = (q_j - [j in S] p_j) / T.
// The student's statistics come from row_stats.h, slice by slice; one workgroup per row joins
// them and sums over S. The gradient reads the row once more and writes it.
#pragma once

#include "row_stats.h"

namespace tsc {

struct DistillArgs {
  const void* logits;  // [N, V]
  int64_t N, V, ld;
  const float* temperature;  // [N]
  const int32_t* ids;        // [N, W]
  const float* values;       // [N, W]
  const int32_t* lengths;    // [N]
  int32_t W;
  const float* teacher_temperature;  // [N] or null: the values as they are
  float* loss;                       // [N]
  int8_t* row_status;                // [N]
  float* stats;                      // [N, 4]: student maximum and sum, teacher maximum and sum
  RowPart* parts;                    // workspace [N, slices]
  int32_t slices;
  int64_t slice_len;
  const float* grad_loss;  // [N]
  void* grad;              // [N, V], contiguous
};

template <int DT>
__global__ void __launch_bounds__(kOpThreads) distill_stats_kernel(DistillArgs a) {
  __shared__ float sh_m[kOpWaves];
  __shared__ double sh_s[kOpWaves];
  for (int64_t item = blockIdx.x; item < a.N * a.slices; item += gridDim.x) {
    const int64_t n = item / a.slices, sl = item - n * a.slices;
    if (a.lengths[n] <= 0) continue;  // the row has no loss: it is not read
    const int64_t lo = sl * a.slice_len, hi = lo + a.slice_len < a.V ? lo + a.slice_len : a.V;
    slice_stats<DT>((const typename Row<DT>::Bits*)a.logits + n * a.ld, lo, hi,
                    make_scale(a.temperature[n]), sh_m, sh_s, a.parts + item);
    lds_barrier();
  }
}

__device__ inline float teacher_value(const DistillArgs& a, int64_t n, int32_t i, float inv_T) {
  return a.values[n * a.W + i] * inv_T;
}

template <int DT>
__global__ void __launch_bounds__(kOpThreads) distill_loss_kernel(DistillArgs a) {
  __shared__ uint64_t scratch[kOpWaves];
  const int64_t n = blockIdx.x;
  const uint32_t tid = threadIdx.x, lane = tid & (kWaveSize - 1), w = tid / kWaveSize;
  const int32_t len = a.lengths[n];
  const float T = a.temperature[n];
  const float Tt = a.teacher_temperature ? a.teacher_temperature[n] : 1.0f;
  float* stats = a.stats + n * 4;
  auto end = [&](int32_t status, float loss) {  // a row without a gradient: teacher sum 0
    if (tid != 0) return;
    a.loss[n] = loss;
    a.row_status[n] = (int8_t)status;
    stats[0] = stats[1] = stats[2] = stats[3] = 0.0f;
  };
  if (len == 0) return end(TSC_ROW_NO_SUPPORT, 0.0f);
  if (len < 0 || len > a.W || !temperature_ok(T) || !temperature_ok(Tt))
    return end(TSC_ROW_INVALID_PARAM, __builtin_nanf(""));
  // Sums over the workgroup; every thread gets the result.
  auto block = [&](auto v, auto op) {
    using U = decltype(v);
    v = wave_reduce(v, op);
    U* s = reinterpret_cast<U*>(scratch);
    lds_barrier();
    if (lane == 0) s[w] = v;
    lds_barrier();
    v = s[0];
#pragma unroll
    for (int i = 1; i < kOpWaves; ++i) v = op(v, s[i]);
    return v;
  };
  const int32_t* ids = a.ids + n * a.W;
  const float* values = a.values + n * a.W;
  float vm = -__builtin_inff();
  uint32_t flags = 0;  // 1: an id out of range, 2: a value NaN or +inf
  for (int32_t i = (int32_t)tid; i < len; i += kOpThreads) {
    const float v = values[i];
    const int32_t id = ids[i];
    flags |= (id < 0 || id >= a.V ? 1u : 0u) | (v < __builtin_inff() ? 0u : 2u);
    vm = __builtin_fmaxf(vm, v);
  }
  vm = block(vm, [](float p, float q) { return __builtin_fmaxf(p, q); });
  flags = block(flags, [](uint32_t p, uint32_t q) { return p | q; });
  if (flags & 1u) return end(TSC_ROW_INVALID_PARAM, __builtin_nanf(""));
  if (flags & 2u) return end(TSC_ROW_NONFINITE, __builtin_nanf(""));
  if (vm == -__builtin_inff()) return end(TSC_ROW_NO_SUPPORT, 0.0f);
  const Scale c = make_scale(T), ct = make_scale(Tt);
  const RowPart none{-__builtin_inff(), 0, 0.0};
  const RowPart st = merge_slices((int32_t)lane < a.slices ? a.parts[n * a.slices + lane] : none, c);
  if (!(st.s < __builtin_inf()) || !(__builtin_fabsf(st.m) < __builtin_inff()))
    return end(TSC_ROW_NONFINITE, __builtin_nanf(""));
  // With e_i the teacher's numerators and A their sum, the loss is
  //     sum_i e_i ((v_i - vm) / Tt - (x_i - m) / T) / A - ln A + ln s.
  double A = 0.0, D = 0.0;
  const auto* row = (const typename Row<DT>::Bits*)a.logits + n * a.ld;
  for (int32_t i = (int32_t)tid; i < len; i += kOpThreads) {
    const float d = values[i] - vm, e = exp2_scaled(d, ct);
    const double x = (double)Row<DT>::get(row + ids[i]);
    if (e > 0.0f) {  // a teacher probability of 0 takes no part, whatever the student's logit
      A += (double)e;
      D += (double)e * ((double)d / (double)Tt - (x - (double)st.m) / (double)T);
    }
  }
  A = block(A, SumOp());
  D = block(D, SumOp());
  if (tid == 0) {
    a.loss[n] = (float)(D / A - log(A) + log(st.s));
    a.row_status[n] = TSC_ROW_OK;
    stats[0] = st.m, stats[1] = (float)st.s, stats[2] = vm, stats[3] = (float)A;
  }
}

// The gradient, a tile of a row per workgroup. The teacher's part is gathered into a float32
// tile in LDS first (ids come in any order), so that each result is rounded once and the row is
// written in whole chunks.
constexpr int kGradThreads = 512;
constexpr int kTile = 16384;  // elements: 64 KB of float32, two workgroups to a CU

__device__ inline void clear_tile(float* tile) {
  for (int i = threadIdx.x * 4; i < kTile; i += kGradThreads * 4)
    *reinterpret_cast<float4*>(tile + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}

template <int DT>
__global__ void __launch_bounds__(kGradThreads) distill_grad_kernel(DistillArgs a) {
  __shared__ __attribute__((aligned(16))) float tile[kTile];
  using B = typename Row<DT>::Bits;
  const int64_t tiles = (a.V + kTile - 1) / kTile;
  for (int64_t item = blockIdx.x; item < a.N * tiles; item += gridDim.x) {
    const int64_t n = item / tiles, lo = (item - n * tiles) * kTile;
    const int64_t hi = lo + kTile < a.V ? lo + kTile : a.V;
    const float m = a.stats[n * 4], s = a.stats[n * 4 + 1];
    const float vm = a.stats[n * 4 + 2], A = a.stats[n * 4 + 3];
    B* out = (B*)a.grad + n * a.V;
    constexpr int kU = kTile / (kGradThreads * 8);
    if (A == 0.0f) {
      const float zero[8] = {};
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t at = lo + (int64_t)(u * kGradThreads + threadIdx.x) * 8;
        if (at < hi) store8<DT>(out, at, hi, zero);
      }
      continue;
    }
    const B* row = (const B*)a.logits + n * a.ld;
    float x[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u) load8<DT>(row, lo + (int64_t)(u * kGradThreads + threadIdx.x) * 8, hi, x[u]);
    const float T = a.temperature[n];
    const float Tt = a.teacher_temperature ? a.teacher_temperature[n] : 1.0f;
    const Scale c = make_scale(T), ct = make_scale(Tt);
    const float inv_A = 1.0f / A, inv_s = 1.0f / s, g = a.grad_loss[n] / T;
    clear_tile(tile);
    lds_barrier();
    const int32_t len = a.lengths[n] < a.W ? a.lengths[n] : a.W;
    for (int32_t i = (int32_t)threadIdx.x; i < len; i += kGradThreads) {
      const int64_t id = a.ids[n * a.W + i];
      if (id >= lo && id < hi)
        atomicAdd(&tile[id - lo], exp2_scaled(a.values[n * a.W + i] - vm, ct) * inv_A);
    }
    lds_barrier();
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t at = lo + (int64_t)(u * kGradThreads + threadIdx.x) * 8;
      if (at < hi) {
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          r[e] = (exp2_scaled(x[u][e] - m, c) * inv_s - tile[at - lo + e]) * g;
        store8<DT>(out, at, hi, r);
      }
    }
    lds_barrier();  // the tile is cleared again by the next item
  }
}

}  // namespace tsc
