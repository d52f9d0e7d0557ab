// Rows and tensors read and written once, 16 bytes a lane: neighbouring lanes' pieces lie next to
// each other for either type. Nontemporal: a float32 tensor read as 8 elements a lane (two pieces,
// each 32 bytes from the next lane's) reaches 6.2 TB/s, pieces 6.0, nontemporal pieces 6.8 to 7.0;
// nontemporal stores 32 bytes apart reach 3.4 where neighbouring ones reach 6.5.
#pragma once

#include <type_traits>

#include "row_stats.h"

namespace tsc {

template <int DT>
struct Piece {
  using Bits = typename Row<DT>::Bits;
  static constexpr int kSize = 16 / (int)sizeof(Bits);  // elements
  using Vec = typename std::conditional<DT == TSC_DTYPE_BF16, u32x4_by2, u32x4_by4>::type;
  u32x4 v;
  __device__ static inline Piece load(const Bits* p) { return {*reinterpret_cast<const Vec*>(p)}; }
  __device__ static inline Piece load_once(const Bits* p) {
    return {__builtin_nontemporal_load(reinterpret_cast<const Vec*>(p))};
  }
  __device__ static inline Piece lowest() {  // -inf throughout
    const uint32_t w = DT == TSC_DTYPE_BF16 ? 0xFF80FF80u : 0xFF800000u;
    return {{w, w, w, w}};
  }
  __device__ inline void unpack(float (&x)[kSize]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == TSC_DTYPE_BF16)
        x[2 * i] = __uint_as_float(v[i] << 16), x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
      else
        x[i] = __uint_as_float(v[i]);
    }
  }
  __device__ static inline void store(Bits* p, const float (&x)[kSize]) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == TSC_DTYPE_BF16)
        r[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16;
      else
        r[i] = __float_as_uint(x[i]);
    }
    __builtin_nontemporal_store((Vec)r, reinterpret_cast<Vec*>(p));
  }
};

// The elements of a piece from `at` on that lie before `end`, one by one; -inf behind it.
template <int DT>
__device__ inline void load_part(const typename Row<DT>::Bits* row, int64_t at, int64_t end,
                                 float (&x)[Piece<DT>::kSize]) {
#pragma unroll
  for (int e = 0; e < Piece<DT>::kSize; ++e) x[e] = at + e < end ? Row<DT>::get(row + at + e) : -__builtin_inff();
}
template <int DT>
__device__ inline void load_piece(const typename Row<DT>::Bits* row, int64_t at, int64_t end,
                                  float (&x)[Piece<DT>::kSize]) {
  if (at + Piece<DT>::kSize <= end) Piece<DT>::load(row + at).unpack(x);
  else load_part<DT>(row, at, end, x);
}
template <int DT>
__device__ inline void store_piece(typename Row<DT>::Bits* row, int64_t at, int64_t end,
                                   const float (&x)[Piece<DT>::kSize]) {
  if (at + Piece<DT>::kSize <= end) {
    Piece<DT>::store(row + at, x);
  } else {
#pragma unroll
    for (int e = 0; e < Piece<DT>::kSize; ++e)
      if (at + e < end) Row<DT>::put(row + at + e, x[e]);
  }
}

}  // namespace tsc
