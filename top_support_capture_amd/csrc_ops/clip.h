// The norm of many tensors taken together, and tensors scaled down to a norm.
//
// A launch covers up to a table of tensors, which travels in the kernel's arguments: nothing is
// copied to the device beforehand, and a captured launch keeps its table. The tensors' elements are
// cut into units, numbered through the table, and dealt to the workgroups in turn, so that what is
// in flight lies close together in memory.
#pragma once

#include "piece.h"

namespace tsc {

constexpr int kClipThreads = 256;
constexpr int kClipWaves = kClipThreads / kWaveSize;
constexpr int kClipGroups = 2048;  // of a norm's launch, at most: 8 workgroups on each CU

// Up to kN tensors in units of kUnit elements. kN is bounded by the 4 KB that a kernel's arguments
// may take: a tensor's address, type and the size of its last unit share a word.
enum class ClipOut {
  kSelf,  // results in place
  kEach,  // an address each
  kFlat,  // one type each for tensors and results, and all results as far from each other as the tensors
};

template <int kN, int kUnit, ClipOut kOut>
struct ClipTable {
  static constexpr int kSize = kN;
  static constexpr int64_t kUnitSize = kUnit;
  static constexpr int kHints = 32;
  static_assert(kUnit <= 8192, "13 bits of the word");
  uint64_t src[kN];
  uint64_t dst[kOut == ClipOut::kEach ? kN : 1];  // the address and the type; kFlat: their distance
  uint32_t first[kN + 1];                         // units before each tensor; the last: all
  uint32_t hint[kHints];  // the tensor of unit i << hint_shift (whole words: scalar loads)
  uint32_t units, hint_shift;
  int32_t n;

  struct Part {
    const void* src;
    void* dst;
    int64_t lo, hi;  // elements
    bool f32, to_f32;
  };
  static constexpr uint64_t kAddress = (uint64_t{1} << 48) - 1, kF32 = uint64_t{1} << 61;
  // Of global memory: without the address space the accesses would be flat ones.
  __device__ static inline void* address(uint64_t word) {
    return (void*)(__attribute__((address_space(1))) void*)(word & kAddress);
  }
  __device__ inline Part part(uint32_t unit) const {
    uint32_t t = hint[unit >> hint_shift];
    while (first[t + 1] <= unit) ++t;
    const uint64_t s = src[t];
    uint64_t d = s;
    if constexpr (kOut == ClipOut::kEach) d = dst[t];
    if constexpr (kOut == ClipOut::kFlat) {
      const uint64_t at = s & kAddress, to = dst[0] & kF32;
      d = (((s & kF32) ? at >> 2 : at >> 1) << (to ? 2 : 1)) + (dst[0] & kAddress);
      d = (d & kAddress) | to;
    }
    const int64_t lo = (int64_t)(unit - first[t]) * kUnit;
    const int64_t size = unit + 1 == first[t + 1] ? (int64_t)(s >> 48 & 0x1FFF) + 1 : kUnit;
    return {address(s), address(d), lo, lo + size, (s & kF32) != 0, (d & kF32) != 0};
  }

  // What a result's address has over its tensor's, counted in elements from 0 and in the result's size.
  static uint64_t distance(const void* tensor, bool f32, const void* out, bool to_f32) {
    return reinterpret_cast<uint64_t>(out) - (reinterpret_cast<uint64_t>(tensor) >> (f32 ? 2 : 1) << (to_f32 ? 2 : 1));
  }

  // The host's side: an empty table, a tensor of `numel` > 0 more (false: it is full), the end.
  void begin() { n = 0, first[0] = 0; }
  bool add(const void* tensor, int64_t numel, bool f32, void* out, bool to_f32) {
    if (n == kN) return false;
    const uint64_t last = (uint64_t)((numel - 1) % kUnit);
    src[n] = reinterpret_cast<uint64_t>(tensor) | last << 48 | (f32 ? kF32 : 0);
    if constexpr (kOut == ClipOut::kEach) dst[n] = reinterpret_cast<uint64_t>(out) | (to_f32 ? kF32 : 0);
    if constexpr (kOut == ClipOut::kFlat) dst[0] = (distance(tensor, f32, out, to_f32) & kAddress) | (to_f32 ? kF32 : 0);
    first[n + 1] = first[n] + (uint32_t)((numel + kUnit - 1) / kUnit);
    ++n;
    return true;
  }
  void end() {
    units = first[n], hint_shift = 0;
    while ((units - 1) >> hint_shift >= (uint32_t)kHints) ++hint_shift;
    int t = 0;
    for (int i = 0; i < kHints; ++i) {
      const uint64_t unit = (uint64_t)i << hint_shift;
      while (t + 1 < n && first[t + 1] <= unit) ++t;
      hint[i] = (uint32_t)t;
    }
  }
};

using NormTable = ClipTable<304, 8192, ClipOut::kSelf>;
// Two loads a thread of kE elements each.
template <int kE, ClipOut kOut>
using ScaleTable = ClipTable<kOut == ClipOut::kFlat ? 300 : 184, 2 * kClipThreads * kE, kOut>;

// Pieces of a thread in a unit of the norm's table.
template <int DT>
constexpr int unit_pieces() { return (int)NormTable::kUnitSize / (kClipThreads * Piece<DT>::kSize); }

// Squares in float64: exact for float32 values, and without overflow or underflow; one float64
// multiply-add an element costs nothing beside the loads (2.1 GB 345 us, in float32 348).
template <int DT>
__device__ inline double sum_squares(const NormTable::Part& p) {
  using P = Piece<DT>;
  constexpr int kU = unit_pieces<DT>();
  const auto* x = (const typename P::Bits*)p.src;
  const int64_t first = p.lo + (int64_t)threadIdx.x * P::kSize;
  constexpr int kStep = kClipThreads * P::kSize;
  double s[2] = {0.0, 0.0};
  auto add = [&](const P& c) {
    float v[P::kSize];
    c.unpack(v);
#pragma unroll
    for (int e = 0; e < P::kSize; ++e) s[e & 1] = __builtin_fma((double)v[e], (double)v[e], s[e & 1]);
  };
  if (p.hi - p.lo == NormTable::kUnitSize) {
    P c[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) c[u] = P::load_once(x + first + u * kStep);
#pragma unroll
    for (int u = 0; u < kU; ++u) add(c[u]);
  } else {
    for (int64_t at = first; at < p.hi; at += kStep) {
      if (at + P::kSize <= p.hi) {
        add(P::load_once(x + at));
      } else {
        for (int64_t i = at; i < p.hi; ++i) {
          const double v = (double)Row<DT>::get(x + i);
          s[0] = __builtin_fma(v, v, s[0]);
        }
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
  for (uint32_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const auto p = a.part(unit);
    s += p.f32 ? sum_squares<TSC_DTYPE_F32>(p) : sum_squares<TSC_DTYPE_BF16>(p);
  }
  s = clip_block_sum(s, sh);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// The norm from its partial sums.
__device__ inline float norm_of(const double* partials, int32_t n, double* sh) {
  double s = 0.0;
  for (int32_t i = (int32_t)threadIdx.x; i < n; i += kClipThreads * 8) {
    double v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i + u * kClipThreads < n ? partials[i + u * kClipThreads] : 0.0;
    s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
  }
  return (float)sqrt(clip_block_sum(s, sh));
}

__global__ void __launch_bounds__(kClipThreads) clip_join_kernel(const double* partials, int32_t n, float* norm) {
  __shared__ double sh[kClipWaves];
  const float v = norm_of(partials, n, sh);
  if (threadIdx.x == 0) *norm = v;
}

// Where a scaling has its norm from: `n` partial sums, which workgroup 0 writes to `norm_out` (if
// not null), or *norm_in.
struct ClipNorm {
  const double* partials;
  int32_t n;
  float max_norm;
  float* norm_out;
  const float* norm_in;
};

// The factor; values stay as they are up to max_norm and where the norm is no number.
__device__ inline float clip_factor(const ClipNorm& c, double* sh) {
  const float norm = c.norm_in ? *c.norm_in : norm_of(c.partials, c.n, sh);
  if (c.norm_out && blockIdx.x == 0 && threadIdx.x == 0) *c.norm_out = norm;
  return norm > c.max_norm && norm < __builtin_inff() ? c.max_norm / norm : 1.0f;
}

// In place: nothing to do where the factor is 1. A workgroup takes several units, as many as leave
// a grid that is soon through when there is nothing to do: for 357 million elements an empty grid with a unit
// of 2048 elements each takes 76 us, this one 5. Scaled, 357 million float32 elements take 524 us, 5.4 TB/s,
// bfloat16 ones 235 to 247, 5.8 to 6.1. (374 million float32 ones took 540 us, and 515 with a unit for each
// workgroup.)
template <int DT>
__device__ inline void scale_unit(const NormTable::Part& p, float by) {
  using P = Piece<DT>;
  constexpr int kU = unit_pieces<DT>();
  auto* x = (typename P::Bits*)p.dst;
  const int64_t first = p.lo + (int64_t)threadIdx.x * P::kSize;
  constexpr int kStep = kClipThreads * P::kSize;
  auto put = [&](const P& c, int64_t at) {
    float v[P::kSize];
    c.unpack(v);
#pragma unroll
    for (int e = 0; e < P::kSize; ++e) v[e] *= by;
    P::store(x + at, v);
  };
  if (p.hi - p.lo == NormTable::kUnitSize) {
    P c[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) c[u] = P::load_once(x + first + u * kStep);
#pragma unroll
    for (int u = 0; u < kU; ++u) put(c[u], first + u * kStep);
  } else {
    for (int64_t at = first; at < p.hi; at += kStep) {
      if (at + P::kSize <= p.hi) put(P::load_once(x + at), at);
      else
        for (int64_t i = at; i < p.hi; ++i) Row<DT>::put(x + i, Row<DT>::get(x + i) * by);
    }
  }
}

constexpr int64_t kInPlaceGroups = 16384;

__global__ void __launch_bounds__(kClipThreads, 8) clip_in_place_kernel(NormTable a, ClipNorm c) {
  __shared__ double sh[kClipWaves];
  const float by = clip_factor(c, sh);
  if (by == 1.0f) return;
  for (uint32_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const auto p = a.part(unit);
    p.f32 ? scale_unit<TSC_DTYPE_F32>(p, by) : scale_unit<TSC_DTYPE_BF16>(p, by);
  }
}

// Into other tensors: a unit per workgroup and two loads a thread, near what the memory does fastest.
// 1.12 billion elements from bfloat16 to float32 (6.7 GB) take 1060 us, 6.3 TB/s; one load a thread 1440
// (it waits for the table's), four 1140; a contiguous span for each of 1024 workgroups and 16-byte
// stores 32 bytes apart 1850. 128 million from bfloat16 to bfloat16 84 us, 6.4 TB/s, with one load 89.
// Tensors allocated one by one, with addresses for the results: 109 of 357 million elements from bfloat16
// to float32 340 us, 6.3 TB/s, as from flat buffers; 224 of 12 million, in two launches, 16.6 against 14.6.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_by2 __attribute__((aligned(2)));

// kE elements of a thread: a piece, or half of one where the other side's piece has 4.
template <int DT, int kE>
__device__ inline void load_few(const typename Row<DT>::Bits* p, float (&v)[kE]) {
  if constexpr (kE == Piece<DT>::kSize) {
    Piece<DT>::load_once(p).unpack(v);
  } else {
    static_assert(DT == TSC_DTYPE_BF16 && kE == 4, "half a piece");
    const u32x2 c = __builtin_nontemporal_load(reinterpret_cast<const u32x2_by2*>(p));
#pragma unroll
    for (int i = 0; i < 2; ++i) v[2 * i] = __uint_as_float(c[i] << 16), v[2 * i + 1] = __uint_as_float(c[i] & 0xFFFF0000u);
  }
}
template <int OT, int kE>
__device__ inline void store_few(typename Row<OT>::Bits* p, const float (&v)[kE]) {
  if constexpr (kE == Piece<OT>::kSize) {
    Piece<OT>::store(p, v);
  } else {
    u32x2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i + 1]) << 16;
    __builtin_nontemporal_store((u32x2_by2)r, reinterpret_cast<u32x2_by2*>(p));
  }
}

// The values are asked for before the factor is, which comes from memory too.
template <int DT, int OT, int kE, class Part, class Factor>
__device__ inline void copy_unit(const Part& p, Factor factor) {
  constexpr int kStep = kClipThreads * kE, kU = 2;
  const auto* x = (const typename Row<DT>::Bits*)p.src;
  auto* y = (typename Row<OT>::Bits*)p.dst;
  const int64_t at = p.lo + (int64_t)threadIdx.x * kE;
  float v[kU][kE];
  if (p.hi - p.lo == kU * kStep) {
#pragma unroll
    for (int u = 0; u < kU; ++u) load_few<DT, kE>(x + at + u * kStep, v[u]);
    const float by = factor();
#pragma unroll
    for (int u = 0; u < kU; ++u) {
#pragma unroll
      for (int e = 0; e < kE; ++e) v[u][e] *= by;
      store_few<OT, kE>(y + at + u * kStep, v[u]);
    }
  } else {
    const float by = factor();
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t here = at + u * kStep;
      if (here + kE <= p.hi) {
        load_few<DT, kE>(x + here, v[u]);
#pragma unroll
        for (int e = 0; e < kE; ++e) v[u][e] *= by;
        store_few<OT, kE>(y + here, v[u]);
      } else {
        for (int64_t i = here; i < p.hi; ++i) Row<OT>::put(y + i, Row<DT>::get(x + i) * by);
      }
    }
  }
}

// kE 8: bfloat16 tensors with bfloat16 results; 4: any.
template <int kE, ClipOut kOut>
__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(ScaleTable<kE, kOut> a, ClipNorm c) {
  constexpr int F = TSC_DTYPE_F32, B = TSC_DTYPE_BF16;
  __shared__ double sh[kClipWaves];
  float by = 0.0f;
  for (uint32_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const auto p = a.part(unit);
    auto factor = [&] { return unit == blockIdx.x ? by = clip_factor(c, sh) : by; };
    if constexpr (kE == 8) copy_unit<B, B, 8>(p, factor);
    else if (p.f32) p.to_f32 ? copy_unit<F, F, 4>(p, factor) : copy_unit<F, B, 4>(p, factor);
    else p.to_f32 ? copy_unit<B, F, 4>(p, factor) : copy_unit<B, B, 4>(p, factor);
  }
}

}  // namespace tsc
