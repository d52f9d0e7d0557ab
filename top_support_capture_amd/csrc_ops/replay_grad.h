// The gradient of the replayed logprobs of a captured support. With S a row's support,
// pi the softmax of x / T over S and lp_i = ln pi_i, upstream gradients G_i of the lp_i (the
// selected logprob's joins its token's) give
//     dx_j = (G_j - pi_j sum_{i in S} G_i) / T for j in S, and 0 elsewhere.
// A workgroup writes a segment of a row (the whole row when there are rows enough). It takes the
// support's statistics itself, which costs a gather of S (or a pass over a bitmask row) per
// segment but no second launch; then it writes its segment once, window by window.
#pragma once

#include "row_stats.h"

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
  int32_t segments;
  int64_t seg_len;
};

constexpr int kGradThreads = 1024;
constexpr int kGradWaves = kGradThreads / kWaveSize;
// Elements of the longest segment: its windows' offsets fit kMaxWindows.
constexpr int64_t kMaxSegment = (int64_t)kMaxWindows * Window<kGradThreads>::kSize;

template <int DT, int kThr>
__device__ inline void fill_zero(typename Row<DT>::Bits* out, int64_t lo, int64_t hi) {
  const float zero[8] = {};
  for (int64_t at = lo + (int64_t)threadIdx.x * 8; at < hi; at += kThr * 8)
    store8<DT>(out, at, hi, zero);
}

template <int DT>
__global__ void __launch_bounds__(kGradThreads, 8) replay_grad_kernel(ReplayGradArgs a) {
  using B = typename Row<DT>::Bits;
  extern __shared__ __attribute__((aligned(16))) float dyn_lds[];
  __shared__ float sh_m[kGradWaves];
  __shared__ double sh_s[kGradWaves], sh_g[kGradWaves];
  __shared__ uint32_t sh_f[kGradWaves];
  const Entries<kGradThreads> ent(dyn_lds, a.W);
  const int64_t n = blockIdx.x / a.segments;
  const int64_t lo = (blockIdx.x - n * a.segments) * a.seg_len;
  const int64_t hi = lo + a.seg_len < a.V ? lo + a.seg_len : a.V;
  const int32_t tid = (int32_t)threadIdx.x;
  const float T = a.temperature[n];
  const int32_t len = a.lengths[n], tok = a.tokens[n];
  const int32_t cs = a.capture_status ? (int32_t)a.capture_status[n] : TSC_ROW_OK;
  const bool from_bits = cs == TSC_ROW_OVERFLOW;
  const bool len_ok = len >= 1 && len <= a.W;
  const B* row = (const B*)a.logits + n * a.ld;
  B* out = (B*)a.grad + n * a.V;
  if (cs >= TSC_ROW_NO_SUPPORT || !temperature_ok(T) || tok < 0 || tok >= a.V ||
      !(from_bits ? a.bits != nullptr : len_ok)) {
    fill_zero<DT, kGradThreads>(out, lo, hi);
    return;
  }
  const float c = plain_scale(T);
  const uint8_t* bits = from_bits ? a.bits + n * a.bits_ld : nullptr;
  const int32_t* ids = a.ids + n * a.W;
  const float* gl = a.grad_logprobs ? a.grad_logprobs + n * a.W : nullptr;
  const bool entries = !from_bits || (gl != nullptr && len_ok);  // the packed ids take part

  // Entries of the packed row, kE per thread at a time: the first batch stays in registers.
  constexpr int kE = 4;
  constexpr int kBatch = kGradThreads * kE;
  int32_t id[kE];
  float x[kE], up[kE];
  auto load_entries = [&](int32_t i0) {
#pragma unroll
    for (int u = 0; u < kE; ++u) id[u] = i0 + u * kGradThreads < len ? ids[i0 + u * kGradThreads] : -1;
#pragma unroll
    for (int u = 0; u < kE; ++u) {
      up[u] = gl && i0 + u * kGradThreads < len ? gl[i0 + u * kGradThreads] : 0.0f;
      x[u] = id[u] >= 0 && id[u] < a.V ? Row<DT>::get(row + id[u]) : -__builtin_inff();
    }
  };
  LseState st;
  double G = 0.0;
  uint32_t flags = 0;  // 1: an id out of range, 2: an element of the support, 4: the token is one
  if (entries) load_entries(tid);
  ent.begin();
  lds_barrier();
  if (entries) {
    for (int32_t i0 = tid;; i0 += kBatch) {
      if (!from_bits) st.add(x, c);
#pragma unroll
      for (int u = 0; u < kE; ++u) {
        const bool in = id[u] >= 0 && id[u] < a.V;
        if (!from_bits && i0 + u * kGradThreads < len) flags |= !in ? 1u : id[u] == tok ? 6u : 2u;
        if (!in || (from_bits && !((bits[id[u] >> 3] >> (id[u] & 7)) & 1u))) continue;
        G += (double)up[u];
        if (id[u] >= lo && id[u] < hi) ent.count((uint32_t)(id[u] - lo));
      }
      if (i0 - tid + kBatch >= len) break;
      load_entries(i0 + kBatch);
    }
  }
  if (from_bits) {
    // The whole row and its mask are streamed: where members are so many that they did not fit
    // the packed width, hardly a line of the row is without one.
    constexpr int kU = 4;
    const int64_t full = a.V / 8;
    auto add_chunk = [&](uint32_t b, float (&v)[8], int64_t ch) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!((b >> e) & 1u)) v[e] = -__builtin_inff();
      st.add(v, c);
      flags |= (b != 0u ? 2u : 0u) | (ch == tok >> 3 && ((b >> (tok & 7)) & 1u) ? 4u : 0u);
    };
    int64_t ch0 = 0;
    for (; ch0 + kU * kGradThreads <= full; ch0 += kU * kGradThreads) {
      uint32_t b[kU];
      typename Row<DT>::Chunk v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) b[u] = bits[ch0 + u * kGradThreads + tid];
#pragma unroll
      for (int u = 0; u < kU; ++u) v[u] = Row<DT>::load(row + (ch0 + u * kGradThreads) * 8 + tid * 8);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float f[8];
        Row<DT>::unpack(v[u], f);
        add_chunk(b[u], f, ch0 + u * kGradThreads + tid);
      }
    }
    for (int64_t ch = ch0 + tid; ch * 8 < a.V; ch += kGradThreads) {
      float f[8];
      load8<DT>(row, ch * 8, a.V, f);
      add_chunk(ch < full ? bits[ch] : bits[ch] & ((1u << (a.V & 7)) - 1u), f, ch);
    }
  }
  block_lse<kGradWaves>(st.m, st.s, c, sh_m, sh_s);
  G = block_all<kGradWaves>(G, SumOp(), sh_g);
  flags = block_all<kGradWaves>(flags, [](uint32_t p, uint32_t q) { return p | q; }, sh_f);
  if (!((flags & 3u) == 2u && st.s < __builtin_inf() && __builtin_fabsf(st.m) < __builtin_inff())) {
    fill_zero<DT, kGradThreads>(out, lo, hi);
    return;
  }
  const float gs = a.grad_selected && (flags & 4u) ? a.grad_selected[n] : 0.0f;
  G += (double)gs;
  const float inv_T = 1.0f / T, m = st.m;
  const float share = (float)(G / ((double)T * st.s));  // sum of G over T s
  // What a packed id adds: all of a packed row's gradient, the upstream gradient alone of a
  // bitmask row's, whose other term comes with the stream.
  ent.offsets();
  lds_barrier();
  if (entries) {
    for (int32_t i0 = tid; i0 - tid < len; i0 += kBatch) {
      if (len > kBatch) load_entries(i0);
#pragma unroll
      for (int u = 0; u < kE; ++u) {
        if (id[u] < lo || id[u] >= hi || (from_bits && !((bits[id[u] >> 3] >> (id[u] & 7)) & 1u))) continue;
        const float own = from_bits ? 0.0f : exp2_scaled(x[u] - m, c) * share;
        ent.place((uint32_t)(id[u] - lo), up[u] * inv_T - own);
      }
    }
  }
  lds_barrier();
  constexpr int kSize = Window<kGradThreads>::kSize;
  auto add = [&](int k) {
    ent.add(k, [](float v) { return v; });
    if (tid == 0 && tok >= lo && tok < hi && (tok - lo) / kSize == k)
      ent.at_window(k).add((uint32_t)((tok - lo) % kSize), gs * inv_T);
  };
  add(0);
  lds_barrier();
  for (int k = 0; lo + (int64_t)k * kSize < hi; ++k) {
    const int64_t at = lo + (int64_t)k * kSize + tid * 8;
    uint32_t b = 0u;
    float v[8];
    if (from_bits && at < hi) {
      b = bits[at >> 3];
      load8<DT>(row, at, hi, v);
    }
    ent.turn(k, add, [&] {
      if (at >= hi) return;
      float r[8];
      ent.at_window(k).take(tid, r);
      if (from_bits) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = (b >> e) & 1u ? r[e] - exp2_scaled(v[e] - m, c) * share : 0.0f;
      }
      store8<DT>(out, at, hi, r);
    });
  }
}

}  // namespace tsc
