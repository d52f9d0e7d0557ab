// The gradient of the replayed logprobs of a captured support. With S a row's support,
// pi the softmax of x / T over S and lp_i = ln pi_i, upstream gradients G_i of the lp_i (the
// selected logprob's joins its token's) give
//     dx_j = (G_j - pi_j sum_{i in S} G_i) / T for j in S, and 0 elsewhere.
// A workgroup writes a segment of a row (the whole row when there are rows enough). It takes the
// support's statistics itself, which costs a gather of S per segment (or a pass over the row, where
// it is streamed under a bitmask) but no second launch; then it writes its segment once.
//
// Measured for bfloat16: 256 rows of 151936 with supports of up to 2048 take 23 us, 78 MB written
// and 27 MB of gathered lines; 256 rows of 129280, three in four of them bitmask rows of about 10000
// members, 35 us (195 MB: two readings and a write). 1024 rows of 151936 with 2048 entries 110 us.
#pragma once

#include <type_traits>

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
  int32_t dense;       // packed rows longer than this are streamed under a bitmask in LDS
  int32_t mask_bytes;  // of that bitmask, for V bits; 0 where no row is that long
  int32_t lds_bytes;   // of dynamic LDS, where rows are streamed
  int32_t hold;        // whether streamed rows are kept in it as far as it goes
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

struct ReplayShared {
  float m[kGradWaves];
  uint32_t f[kGradWaves];
  double s[kGradWaves], g[kGradWaves];
};

// Entries i0, i0 + kGradThreads, ... of a packed row: ids (-1 past the length), upstream gradients
// and, unless the row is streamed, logits.
template <int DT, int N>
struct PackedEntries {
  static constexpr int kE = N;
  int32_t id[N];
  float up[N], x[N];
  __device__ inline void load(const int32_t* ids, const float* gl, const typename Row<DT>::Bits* row, bool streamed,
                              int64_t V, int32_t len, int32_t i0) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      id[u] = i0 + u * kGradThreads < len ? ids[i0 + u * kGradThreads] : -1;
      up[u] = gl && i0 + u * kGradThreads < len ? gl[i0 + u * kGradThreads] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
      x[u] = !streamed && id[u] >= 0 && id[u] < V ? Row<DT>::get(row + id[u]) : -__builtin_inff();
  }
};

// The first chunks of a streamed row, kept in LDS from the first pass over it to the second where
// no entries need the room: `steps` of a chunk a thread.
template <int DT>
struct HeldChunks {
  using Chunk = typename Row<DT>::Chunk;
  static constexpr int kParts = sizeof(Chunk) / 16;
  u32x4* at;
  int32_t steps;
  __device__ inline HeldChunks(void* lds, int32_t bytes)
      : at(reinterpret_cast<u32x4*>(lds)), steps(bytes / (int32_t)(kGradThreads * sizeof(Chunk))) {}
  __device__ inline void put(int64_t step, const Chunk& c) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      at[(step * kParts + i) * kGradThreads + threadIdx.x] = reinterpret_cast<const u32x4*>(&c)[i];
  }
  __device__ inline Chunk get(int64_t step) const {
    Chunk c;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      reinterpret_cast<u32x4*>(&c)[i] = at[(step * kParts + i) * kGradThreads + threadIdx.x];
    return c;
  }
};

struct NoneHeld {
  static constexpr int32_t steps = 0;
};

// Mask bytes and logits of a bitmask row, kAhead windows before their turn. Lanes past the last
// whole chunk of [lo, hi) ask for the first one, and use nothing of it.
template <int DT, class Mask, class Held>
struct MaskedStream {
  static constexpr int kSize = Window<kGradThreads>::kSize;
  static constexpr int kAhead = DT == TSC_DTYPE_BF16 ? 4 : 2;
  const typename Row<DT>::Bits* row;
  Mask bits;
  int64_t lo, hi;
  Held held;
  typename Row<DT>::Chunk v[kAhead];
  uint32_t b[kAhead];
  __device__ inline int64_t place(int k) const { return lo + (int64_t)k * kSize + (int64_t)threadIdx.x * 8; }
  __device__ inline void ask(int j, int k) {
    if (lo + 8 > hi) return;
    const int64_t at = place(k) + 8 <= hi ? place(k) : lo;
    b[j] = bits[at >> 3];
    if constexpr (!std::is_same<Held, NoneHeld>::value) {
      if (k < held.steps) {  // uniform
        v[j] = held.get(k);
        return;
      }
    }
    v[j] = Row<DT>::load(row + at);
  }
  // use(k, at, x, mask) for every window k of the segment, the logits of non-members as they are.
  template <class Use>
  __device__ inline void run(Use use) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) ask(j, j);
    for (int k0 = 0; lo + (int64_t)k0 * kSize < hi; k0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int k = k0 + j;
        if (lo + (int64_t)k * kSize < hi) {  // uniform
          const int64_t at = place(k);
          float x[8];
          uint32_t mask = b[j];
          if (at + 8 <= hi) {
            Row<DT>::unpack(v[j], x);
          } else {
            load8<DT>(row, at, hi, x);
            mask = at < hi ? bits[at >> 3] & ((1u << (hi - at)) - 1u) : 0u;
          }
          ask(j, k + kAhead);
          use(k, at, x, mask);
        }
      }
    }
  }
};

// All ones where bit e of b is set: members are kept by masks, not by branches.
__device__ inline uint32_t member_mask(uint32_t b, int e) { return (uint32_t)((int32_t)(b << (31 - e)) >> 31); }

// kStreams: rows may be streamed under a bitmask. Calls without bitmasks or rows that long take the
// kernel without that code, which fits two workgroups to a CU (1024 rows of 32000 32 us against 44,
// 300 of 151936 37 against 47; with the code in, the registers of two workgroups spill).
template <int DT, bool kStreams>
__global__ void __launch_bounds__(kGradThreads, kStreams ? 4 : 8) replay_grad_kernel(ReplayGradArgs a) {
  using B = typename Row<DT>::Bits;
  extern __shared__ __attribute__((aligned(16))) float dyn_lds[];
  __shared__ ReplayShared sh;
  const Entries<kGradThreads> ent(dyn_lds, a.W, a.mask_bytes);
  const int64_t n = blockIdx.x / a.segments;
  const int64_t lo = (blockIdx.x - n * a.segments) * a.seg_len;
  const int64_t hi = lo + a.seg_len < a.V ? lo + a.seg_len : a.V;
  const int32_t tid = (int32_t)threadIdx.x, lane = tid & (kWaveSize - 1), w = tid / kWaveSize;
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

  uint32_t flags = 0;  // 1: an id out of range, 2: an element of the support, 4: the token is one
  // A long packed row is turned into a bitmask in LDS and treated as a bitmask row, unless an id
  // occurs twice.
  uint32_t* own = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(dyn_lds) + (a.lds_bytes - a.mask_bytes));
  bool streamed = kStreams && from_bits;
  if (kStreams && !from_bits && len > a.dense) {
    for (int32_t i = tid; i < a.mask_bytes / 4; i += kGradThreads) own[i] = 0u;
    lds_barrier();
    uint32_t again = 0u;
    constexpr int kU = 8;
    for (int32_t i0 = tid; i0 - tid < len; i0 += kU * kGradThreads) {
      int32_t id[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) id[u] = i0 + u * kGradThreads < len ? ids[i0 + u * kGradThreads] : INT32_MIN;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t bit = 1u << (id[u] & 31);
        if (id[u] >= 0 && id[u] < a.V)
          again |= atomicOr(own + (id[u] >> 5), bit) & bit;
        else if (id[u] != INT32_MIN || i0 + u * kGradThreads < len)
          flags |= 1u;
      }
    }
    streamed = block_all(again, [](uint32_t p, uint32_t q) { return p | q; }, sh.f) == 0u;
  }
  const bool entries = !streamed || (gl != nullptr && len_ok);  // the packed ids take part

  // Entries of the packed row: a thread's first kKept stay in registers (longer rows' second half
  // of them is skipped as a whole where there is none), the rest come kMore at a time, all of their
  // loads together, and are read again when they are placed.
  constexpr int kFirst = 2, kKept = 4, kMore = 4;
  PackedEntries<DT, kFirst> first;
  PackedEntries<DT, kKept - kFirst> second;
  const bool longer = entries && len > kFirst * kGradThreads;
  // Whether entry u is of the support and, if so, of this segment.
  auto of_support = [&](int32_t id) {
    return id >= 0 && id < a.V && (!from_bits || ((bits[id >> 3] >> (id & 7)) & 1u));
  };
  auto here = [&](int32_t id) { return id >= lo && id < hi && of_support(id); };
  LseState st;
  double G = 0.0;
  if (entries) first.load(ids, gl, row, streamed, a.V, len, tid);
  if (longer) second.load(ids, gl, row, streamed, a.V, len, tid + kFirst * kGradThreads);
  if (entries) ent.begin();
  lds_barrier();
  HeldChunks<DT> held(dyn_lds, streamed && !entries && a.hold ? a.lds_bytes - a.mask_bytes : 0);
  auto look = [&](auto& t, int32_t i0) {
    if (!streamed) st.add(t.x, c);
#pragma unroll
    for (int u = 0; u < t.kE; ++u) {
      const int32_t id = t.id[u];
      if (!streamed && i0 + u * kGradThreads < len) flags |= id < 0 || id >= a.V ? 1u : id == tok ? 6u : 2u;
      if (of_support(id)) G += (double)t.up[u];
      if (here(id)) ent.count((uint32_t)(id - lo));
    }
  };
  if (entries) {
    look(first, tid);
    if (longer) look(second, tid + kFirst * kGradThreads);
    for (int32_t i0 = tid + kKept * kGradThreads; i0 - tid < len; i0 += kMore * kGradThreads) {
      PackedEntries<DT, kMore> t;
      t.load(ids, gl, row, streamed, a.V, len, i0);
      look(t, i0);
    }
  }
  // The whole row and its mask are streamed: where members are so many, hardly a line of the row is
  // without one.
  auto stream_stats = [&](auto mask) {
    constexpr int kU = DT == TSC_DTYPE_BF16 ? 4 : 2;  // chunks of a thread at a time, and as many ahead
    constexpr int64_t kStep = kGradThreads * 8;
    const int64_t whole = a.V & ~int64_t{7}, start = (int64_t)tid * 8;
    typename Row<DT>::Chunk v[kU];
    uint32_t b[kU], any = 0;
    auto ask = [&](int u, int64_t at) {  // past the last whole chunk: the first one, without members
      const bool in = at < whole;
      b[u] = mask[in ? at >> 3 : 0];
      v[u] = Row<DT>::load(row + (in ? at : 0));
      if (!in) b[u] = 0u;
    };
    if (whole > 0) {
#pragma unroll
      for (int u = 0; u < kU; ++u) ask(u, start + u * kStep);
    }
    for (int64_t base = 0; base < whole; base += kU * kStep) {
      float f[kU * 8];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        Row<DT>::unpack(v[u], reinterpret_cast<float(&)[8]>(f[u * 8]));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t keep = member_mask(b[u], e);
          f[u * 8 + e] = __uint_as_float((__float_as_uint(f[u * 8 + e]) & keep) | (0xFF800000u & ~keep));
        }
        any |= b[u];
        if (base / kStep + u < held.steps) held.put(base / kStep + u, v[u]);
        ask(u, base + start + (kU + u) * kStep);
      }
      st.add(f, c);
    }
    if (whole < a.V && tid == 0) {  // the ragged last chunk
      const uint32_t last = mask[whole >> 3] & ((1u << (a.V & 7)) - 1u);
      float f[8];
      load8<DT>(row, whole, a.V, f);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!((last >> e) & 1u)) f[e] = -__builtin_inff();
      st.add(f, c);
      any |= last;
    }
    flags |= (any != 0u ? 2u : 0u) | ((mask[tok >> 3] >> (tok & 7)) & 1u ? 4u : 0u);
  };
  if constexpr (kStreams) {
    if (from_bits)
      stream_stats(bits);
    else if (streamed)
      stream_stats(reinterpret_cast<const uint8_t*>(own));
  }
  // The workgroup's maximum and flags, then its sums; between the two barriers the first wave
  // also turns the windows' counts into offsets.
  const float wm = wave_max(st.m);
  flags = wave_reduce(flags, [](uint32_t p, uint32_t q) { return p | q; });
  if (lane == 0) sh.m[w] = wm, sh.f[w] = flags;
  lds_barrier();
  float m = sh.m[0];
  flags = sh.f[0];
#pragma unroll
  for (int i = 1; i < kGradWaves; ++i) m = __builtin_fmaxf(m, sh.m[i]), flags |= sh.f[i];
  const double ws = wave_reduce(rescaled(st.s, st.m, m, c), SumOp());
  G = wave_reduce(G, SumOp());
  if (lane == 0) sh.s[w] = ws, sh.g[w] = G;
  if (entries) ent.offsets();
  lds_barrier();
  double S = sh.s[0];
  G = sh.g[0];
#pragma unroll
  for (int i = 1; i < kGradWaves; ++i) S += sh.s[i], G += sh.g[i];
  if (!((flags & 3u) == 2u && S < __builtin_inf() && __builtin_fabsf(m) < __builtin_inff())) {
    fill_zero<DT, kGradThreads>(out, lo, hi);
    return;
  }
  const float gs = a.grad_selected && (flags & 4u) ? a.grad_selected[n] : 0.0f;
  G += (double)gs;
  const float inv_T = 1.0f / T;
  const float share = (float)(G / ((double)T * S));  // sum of G over T s
  // What a packed id adds: all of the gradient, or the upstream gradient alone where the other term
  // comes with the stream.
  auto place = [&](const auto& t) {
#pragma unroll
    for (int u = 0; u < t.kE; ++u)
      if (here(t.id[u]))
        ent.place((uint32_t)(t.id[u] - lo),
                  t.up[u] * inv_T - (streamed ? 0.0f : exp2_scaled(t.x[u] - m, c) * share));
  };
  if (entries) {
    place(first);
    if (longer) place(second);
    for (int32_t i0 = tid + kKept * kGradThreads; i0 - tid < len; i0 += kMore * kGradThreads) {
      PackedEntries<DT, kMore> t;
      t.load(ids, gl, row, streamed, a.V, len, i0);
      place(t);
    }
  }
  lds_barrier();
  constexpr int kSize = Window<kGradThreads>::kSize;
  auto add = [&](int k) {
    ent.add(k);
    if (tid == 0 && tok >= lo && tok < hi && (tok - lo) / kSize == k)
      ent.at_window(k).add((uint32_t)((tok - lo) % kSize), gs * inv_T);
  };
  if (entries) {
    add(0);
    lds_barrier();
  }
  if (!kStreams || !streamed) {
    for (int k = 0; lo + (int64_t)k * kSize < hi; ++k) {
      ent.turn(k, add, [&] {
        const int64_t at = lo + (int64_t)k * kSize + tid * 8;
        if (at >= hi) return;
        float r[8];
        ent.at_window(k).take(tid, r);
        store8<DT>(out, at, hi, r);
      });
    }
    return;
  }
  // Of a member the stream gives -pi sum of G / T; `r` holds what the entries add to it.
  auto write = [&](int64_t at, const float (&v)[8], uint32_t b, float (&r)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      r[e] = __uint_as_float(__float_as_uint(__builtin_fmaf(exp2_scaled(v[e] - m, c), -share, r[e])) &
                             member_mask(b, e));
    store8<DT>(out, at, hi, r);
  };
  auto write_row = [&](auto mask) {
    if (entries) {
      MaskedStream<DT, decltype(mask), NoneHeld>{row, mask, lo, hi, {}}.run([&](int k, int64_t at, float (&v)[8], uint32_t b) {
        ent.turn(k, add, [&] {
          if (at >= hi) return;
          float r[8];
          ent.at_window(k).take(tid, r);
          write(at, v, b, r);
        });
      });
    } else {  // the token alone has an upstream gradient: no windows, no barriers
      MaskedStream<DT, decltype(mask), HeldChunks<DT>>{row, mask, lo, hi, held}.run([&](int, int64_t at, float (&v)[8], uint32_t b) {
        if (at >= hi) return;
        float r[8] = {};
        if (at >> 3 == tok >> 3) {
#pragma unroll
          for (int e = 0; e < 8; ++e) r[e] = e == (tok & 7) ? gs * inv_T : 0.0f;
        }
        write(at, v, b, r);
      });
    }
  };
  if constexpr (kStreams) {
    if (from_bits)
      write_row(bits);
    else
      write_row(reinterpret_cast<const uint8_t*>(own));
  }
}

}  // namespace tsc
