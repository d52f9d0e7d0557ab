// The gradient of the replayed logprobs of a captured support. With S a row's support,
// pi the softmax of x / T over S and lp_i = ln pi_i, upstream gradients G_i of the lp_i (the
// selected logprob's joins its token's) give
//     dx_j = (G_j - pi_j sum_{i in S} G_i) / T for j in S, and 0 elsewhere.
// One workgroup per row takes the support's maximum, sum and sum of G; then the rows are written
// tile by tile.
#pragma once

#include "distill.h"

namespace tsc {

struct ReplayGradArgs {
  const void* logits;  // [N, V]
  int64_t N, V, ld;
  const float* temperature;      // [N]
  const int32_t* ids;            // [N, W]
  const int32_t* lengths;        // [N]
  int32_t W;
  const int8_t* capture_status;  // [N] or null
  const uint8_t* bits;           // [N, bits_ld] or null
  int64_t bits_ld;
  const int32_t* tokens;         // [N]
  const float* grad_selected;    // [N] or null
  const float* grad_logprobs;    // [N, W] or null
  void* grad;                    // [N, V], contiguous
  float* stats;                  // workspace [N, 4]: maximum, sum, sum of G, kind of the row
};

// Kinds of rows: no gradient, support in the packed ids, support in the bitmask.
constexpr float kRowZero = 0.0f, kRowPacked = 1.0f, kRowBits = 2.0f;

template <int DT>
__global__ void __launch_bounds__(kOpThreads) replay_grad_stats_kernel(ReplayGradArgs a) {
  __shared__ float sh_m[kOpWaves];
  __shared__ double sh_s[kOpWaves], sh_g[kOpWaves];
  __shared__ uint32_t sh_f[kOpWaves];
  const int64_t n = blockIdx.x;
  const uint32_t tid = threadIdx.x, lane = tid & (kWaveSize - 1), w = tid / kWaveSize;
  const float T = a.temperature[n];
  const int32_t len = a.lengths[n], tok = a.tokens[n];
  const int32_t cs = a.capture_status ? (int32_t)a.capture_status[n] : TSC_ROW_OK;
  const bool from_bits = cs == TSC_ROW_OVERFLOW;
  const bool len_ok = len >= 1 && len <= a.W;
  float* stats = a.stats + n * 4;
  if (cs >= TSC_ROW_NO_SUPPORT || !temperature_ok(T) || tok < 0 || tok >= a.V ||
      !(from_bits ? a.bits != nullptr : len_ok)) {
    if (tid == 0) stats[0] = stats[1] = stats[2] = 0.0f, stats[3] = kRowZero;
    return;
  }
  const Scale c = make_scale(T);
  const auto* row = (const typename Row<DT>::Bits*)a.logits + n * a.ld;
  const uint8_t* bits = from_bits ? a.bits + n * a.bits_ld : nullptr;
  LseState st;
  double G = 0.0;
  uint32_t flags = 0;  // 1: an id out of range, 2: an element of the support, 4: the token is one
  if (len_ok) {
    for (int32_t i = (int32_t)tid; i < len; i += kOpThreads) {
      const int32_t id = a.ids[n * a.W + i];
      if (id < 0 || id >= a.V) {
        flags |= from_bits ? 0u : 1u;
        continue;
      }
      if (from_bits && !((bits[id >> 3] >> (id & 7)) & 1u)) continue;
      if (!from_bits) {
        const float x[1] = {Row<DT>::get(row + id)};
        st.add(x, c);
        flags |= 2u | (id == tok ? 4u : 0u);
      }
      if (a.grad_logprobs) G += (double)a.grad_logprobs[n * a.W + i];
    }
  }
  if (from_bits) {
    const int64_t chunks = (a.V + 7) / 8;
    for (int64_t ch = tid; ch < chunks; ch += kOpThreads) {
      uint32_t b = bits[ch];
      if (ch == chunks - 1 && (a.V & 7)) b &= (1u << (a.V & 7)) - 1u;
      if (b == 0u) continue;
      float x[8];
      load8<DT>(row, ch * 8, a.V, x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!((b >> e) & 1u)) x[e] = -__builtin_inff();
      st.add(x, c);
      flags |= 2u | (ch == tok >> 3 && ((b >> (tok & 7)) & 1u) ? 4u : 0u);
    }
  }
  block_lse<kOpWaves>(st.m, st.s, c, sh_m, sh_s);
  G = wave_reduce(G, SumOp());
  flags = wave_reduce(flags, [](uint32_t p, uint32_t q) { return p | q; });
  if (lane == 0) sh_g[w] = G, sh_f[w] = flags;
  lds_barrier();
  if (tid == 0) {
    G = 0.0;
    for (int i = 0; i < kOpWaves; ++i) G += sh_g[i], flags |= sh_f[i];
    if (a.grad_selected && (flags & 4u)) G += (double)a.grad_selected[n];
    const bool ok = (flags & 3u) == 2u && st.s < __builtin_inf() && __builtin_fabsf(st.m) < __builtin_inff();
    stats[0] = st.m, stats[1] = (float)st.s, stats[2] = (float)G;
    stats[3] = !ok ? kRowZero : from_bits ? kRowBits : kRowPacked;
  }
}

template <int DT>
__global__ void __launch_bounds__(kGradThreads) replay_grad_kernel(ReplayGradArgs a) {
  __shared__ __attribute__((aligned(16))) float tile[kTile];
  using B = typename Row<DT>::Bits;
  const int64_t tiles = (a.V + kTile - 1) / kTile;
  for (int64_t item = blockIdx.x; item < a.N * tiles; item += gridDim.x) {
    const int64_t n = item / tiles, lo = (item - n * tiles) * kTile;
    const int64_t hi = lo + kTile < a.V ? lo + kTile : a.V;
    const float m = a.stats[n * 4], s = a.stats[n * 4 + 1], G = a.stats[n * 4 + 2];
    const float kind = a.stats[n * 4 + 3];
    const B* row = (const B*)a.logits + n * a.ld;
    B* out = (B*)a.grad + n * a.V;
    clear_tile(tile);
    lds_barrier();
    const uint8_t* bits = kind == kRowBits ? a.bits + n * a.bits_ld : nullptr;
    float inv_T = 0.0f, share = 0.0f;  // share: sum of G over T s
    Scale c{0.0f, 0.0f};
    if (kind != kRowZero) {
      const float T = a.temperature[n];
      c = make_scale(T);
      inv_T = 1.0f / T;
      share = G / (T * s);
      const int32_t len = a.lengths[n], tok = a.tokens[n];
      const float gs = a.grad_selected ? a.grad_selected[n] : 0.0f;
      if (len >= 1 && len <= a.W) {
        for (int32_t i = (int32_t)threadIdx.x; i < len; i += kGradThreads) {
          const int64_t id = a.ids[n * a.W + i];
          if (id < lo || id >= hi) continue;
          float v = a.grad_logprobs ? a.grad_logprobs[n * a.W + i] * inv_T : 0.0f;
          if (kind == kRowPacked) {
            if (id == tok) v += gs * inv_T;
            v -= exp2_scaled(Row<DT>::get(row + id) - m, c) * share;
          }
          atomicAdd(&tile[id - lo], v);
        }
      }
      if (kind == kRowBits && threadIdx.x == 0 && tok >= lo && tok < hi) atomicAdd(&tile[tok - lo], gs * inv_T);
    }
    lds_barrier();
    for (int64_t at = lo + (int64_t)threadIdx.x * 8; at < hi; at += kGradThreads * 8) {
      float r[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = tile[at - lo + e];
      if (kind == kRowBits) {
        const uint32_t b = bits[at >> 3];
        if (b != 0u) {
          float x[8];
          load8<DT>(row, at, hi, x);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            r[e] = (b >> e) & 1u ? r[e] - exp2_scaled(x[e] - m, c) * share : 0.0f;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) r[e] = 0.0f;
        }
      }
      store8<DT>(out, at, hi, r);
    }
    lds_barrier();  // the tile is cleared again by the next item
  }
}

}  // namespace tsc
