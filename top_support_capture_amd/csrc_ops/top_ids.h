// The n first elements of a row in (value desc, id asc) order, n small, beside a pass over the row
// that is made anyway.
//
// While a thread reads its pieces it keeps the maximum and the first piece that holds it: its key,
// (value, earlier piece first). Any element among the row's n first lies in a thread whose key is
// among the n best keys: each better key stands for an element that precedes every element of the
// thread. So a bound below the n-th best key leaves few threads, whose pieces are read once more and
// compared with the bound; what reaches it is ranked.
//
// All of it is a chain of short steps between barriers. For 256 rows of 151936 bfloat16 logits it adds
// 4.4 us to a pass of 18.8 for one alternative, 5.5 for 20, 8.2 for 64 and 13.5 for 128 (waves' best, ranks
// and pieces all grow with n); with rows enough other workgroups' loads cover most of it.
#pragma once

#include "piece.h"

namespace tsc {

// Order-preserving bits of a float; -0 ties +0.
__device__ inline uint32_t order_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ inline float from_order_bits(uint32_t o) {
  return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// Keys in 64 bits, greater ones first; 0 stands for none. Of an element, or of a piece.
__device__ inline uint64_t top_key(float x, uint32_t id) { return (uint64_t)order_bits(x) << 32 | (uint32_t)~id; }
__device__ inline float key_value(uint64_t k) { return from_order_bits((uint32_t)(k >> 32)); }
__device__ inline int32_t key_id(uint64_t k) { return (int32_t)~(uint32_t)k; }
// The least key that an element of the pieces up to this one's can have at its value.
template <int kPiece>
__device__ inline uint64_t piece_bound(uint64_t k) {
  return k == 0 ? 0 : (k >> 32 << 32) | (uint32_t)~(~(uint32_t)k * kPiece + (kPiece - 1));
}

constexpr int kTopMost = 128;  // n
constexpr int kTopFew = 512;   // candidates that are ranked by counting

// The LDS of a selection by kThr threads: kBytes of dynamic LDS, and TopShared.
template <int kThr>
struct TopLists {
  static constexpr int kWaves = kThr / kWaveSize, kGroups = kThr / 16;
  static constexpr int kCap = kTopFew + kThr * 8;  // those, and a round of pieces of 8
  static constexpr size_t kBytes = kCap * 8 + kThr * 2;
  uint64_t* cand;    // [kCap]
  uint16_t* thread;  // [kThr]
  __device__ inline explicit TopLists(void* lds)
      : cand(reinterpret_cast<uint64_t*>(lds)), thread(reinterpret_cast<uint16_t*>(cand + kCap)) {}
};
template <int kThr>
struct TopShared {
  static constexpr int kPerWave = kTopMost / TopLists<kThr>::kWaves + 1;
  uint64_t wave[TopLists<kThr>::kWaves * kPerWave];
  uint64_t bound;
  uint32_t hist[256];
  uint32_t count, threads, digit, left;
};

// How many of list[0, c) are greater than `mine`, which 16 neighbouring lanes ask for together: each
// takes every 16th. (One thread to a key, reading the list by itself, took the largest part of the
// selection: every read is waited for.)
__device__ inline int count_above(const uint64_t* list, int c, uint64_t mine) {
  int above = 0;
#pragma unroll 4
  for (int i = (int)threadIdx.x & 15; i < c; i += 16) above += list[i] > mine;
  above += dpp_mov<dpp::kQuadSwap1>(above, above);
  above += dpp_mov<dpp::kQuadSwap2>(above, above);
  above += dpp_mov<dpp::kRowRor4>(above, above);
  return above + dpp_mov<dpp::kRowRor8>(above, above);
}

// The n-th greatest of list[0, c), 0 if there are fewer (keys other than 0 are distinct). Needs
// sh.bound == 0 and a barrier before, and a barrier behind it.
template <int kThr>
__device__ inline void top_nth(const uint64_t* list, int c, int n, TopShared<kThr>& sh) {
  for (int g = 0; g < c; g += TopLists<kThr>::kGroups) {
    const int i = g + ((int)threadIdx.x >> 4);
    const uint64_t mine = i < c ? list[i] : 0;
    if (count_above(list, c, mine) == n - 1 && mine != 0) sh.bound = mine;
  }
}

// The greatest of the wave's keys: by the values, and by the rest only where values tie.
__device__ inline uint64_t wave_best(uint64_t key) {
  const uint32_t hi = (uint32_t)(key >> 32), most = wave_reduce(hi, MaxOp());
  const uint64_t at = __ballot(hi == most);
  if ((at & (at - 1)) == 0) return read_lane(key, __builtin_ctzll(at));
  return (uint64_t)most << 32 | wave_reduce(hi == most ? (uint32_t)key : 0u, MaxOp());
}

// A key that at least n of the threads' keys reach, near the n-th best: the n-th best among each
// wave's best few; 0 if those are fewer than n. Where only the first threads have a key (`some`),
// they are dealt out to all waves first.
template <int kThr>
__device__ inline uint64_t top_bound(uint64_t key, int n, bool some, const TopLists<kThr>& lists,
                                     TopShared<kThr>& sh) {
  constexpr int kWaves = TopLists<kThr>::kWaves;
  const uint32_t tid = threadIdx.x, w = tid / kWaveSize;
  const int per = (n + kWaves - 1) / kWaves + (n > 1 ? 1 : 0);  // at most kPerWave
  lds_barrier();  // sh may still be read by an earlier call
  if (some) {
    lists.cand[tid] = key;
    lds_barrier();
    key = lists.cand[(tid % kWaves) * kWaveSize + tid / kWaves];
  }
  for (int i = 0; i < per; ++i) {
    const uint64_t best = wave_best(key);
    if (key == best) key = 0;
    if ((tid & (kWaveSize - 1)) == 0) sh.wave[w * per + i] = best;
  }
  if (tid == 0) sh.bound = 0;
  lds_barrier();
  top_nth(sh.wave, kWaves * per, n, sh);
  lds_barrier();
  return sh.bound;
}

// Leaves the n greatest of cand[0, c) there, in any order, and sh.count = n (n < c <= kCap,
// all distinct). Digit by digit from the top: a histogram of the keys that share the n-th one's
// upper digits gives its next digit. Returns the n-th greatest.
template <int kThr>
__device__ inline uint64_t top_narrow(uint64_t* cand, int c, int n, TopShared<kThr>& sh) {
  constexpr int kE = (TopLists<kThr>::kCap + kThr - 1) / kThr;
  static_assert(kThr >= 256, "a thread for each digit");
  const int tid = (int)threadIdx.x;
  uint64_t k[kE], prefix = 0;
  lds_barrier();
#pragma unroll
  for (int i = 0; i < kE; ++i) k[i] = tid + i * kThr < c ? cand[tid + i * kThr] : 0;
  uint32_t left = (uint32_t)n;
  for (int shift = 56; shift >= 0; shift -= 8) {
    if (tid < 256) sh.hist[tid] = 0;
    lds_barrier();
    const uint64_t above = shift == 56 ? 0 : ~uint64_t{0} << (shift + 8);
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (k[i] != 0 && (k[i] & above) == prefix) atomicAdd(&sh.hist[(uint32_t)(k[i] >> shift) & 255u], 1u);
    lds_barrier();
    if (tid < kWaveSize) {  // lane l: digits 255 - 4 l and the three below
      uint32_t h[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += h[i] = sh.hist[255 - 4 * tid - i];
      uint32_t before = wave_incl_scan(sum, SumOp(), 0u) - sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (before < left && left <= before + h[i]) sh.digit = (uint32_t)(255 - 4 * tid - i), sh.left = left - before;
        before += h[i];
      }
    }
    lds_barrier();
    prefix |= (uint64_t)sh.digit << shift;
    left = sh.left;
  }
  if (tid == 0) sh.count = 0;
  lds_barrier();
#pragma unroll
  for (int i = 0; i < kE; ++i)
    if (k[i] >= prefix && k[i] != 0) cand[atomicAdd(&sh.count, 1u)] = k[i];
  lds_barrier();
  return prefix;
}

// The n first of the sh.count candidates in order, and 0 behind them if they are fewer: sh.wave[0, n),
// once all threads are through.
template <int kThr>
__device__ inline const uint64_t* top_sort(uint64_t* cand, int n, TopShared<kThr>& sh) {
  static_assert(sizeof(sh.wave) >= kTopMost * 8 && kThr >= kTopMost, "room for the result");
  lds_barrier();
  if ((int)sh.count > kTopFew) top_narrow(cand, (int)sh.count, n, sh);
  const int c = (int)sh.count, tid = (int)threadIdx.x;
  for (int g = 0; g < c; g += TopLists<kThr>::kGroups) {
    const int i = g + (tid >> 4);
    const uint64_t mine = i < c ? cand[i] : 0;
    const int above = count_above(cand, c, mine);
    if ((tid & 15) == 0 && i < c && above < n) sh.wave[above] = mine;
  }
  if (tid >= c && tid < n) sh.wave[tid] = 0;
  lds_barrier();
  return sh.wave;
}

// The candidates among row[lo, hi), lo a multiple of 8, from the threads' keys (0 of a thread that
// has read nothing), into lists.cand and sh.count: all of the n first (as many as there are) and
// few others. Thread t has read the pieces from lo + t pieces on in steps of kThr.
template <int DT, int kThr>
__device__ inline void top_collect(const typename Row<DT>::Bits* row, int64_t lo, int64_t hi, uint64_t key, int n,
                                   const TopLists<kThr>& lists, TopShared<kThr>& sh) {
  constexpr int kSize = Piece<DT>::kSize, kStep = kThr * kSize, kCap = TopLists<kThr>::kCap;
  const uint32_t tid = threadIdx.x;
  const uint64_t threads_bound = top_bound(key, n, hi - lo < kStep, lists, sh);
  uint64_t bound = piece_bound<kSize>(threads_bound);
  if (tid == 0) sh.count = 0, sh.threads = 0;
  lds_barrier();
  if (key != 0 && key >= threads_bound) lists.thread[atomicAdd(&sh.threads, 1u)] = (uint16_t)tid;
  lds_barrier();
  const uint32_t steps = (uint32_t)((hi - lo + kStep - 1) / kStep);
  const uint32_t items = sh.threads * steps;  // pieces to read: at most 2^10 * 2^19
  // Item j is piece j % steps of the thread j / steps of the list; from round to round by addition.
  const uint32_t di = kThr / steps, dr = kThr - di * steps;
  uint32_t i = tid / steps, r = tid - i * steps;
  // kB rounds of pieces from item j0 on, all in flight together; what does not fit is counted.
  auto rounds = [&](uint32_t j0, auto blocks) {
    constexpr int kB = decltype(blocks)::value;
    float x[kB][kSize];
    int64_t at[kB];
    const uint32_t wave_first = j0 + (tid & ~(uint32_t)(kWaveSize - 1));
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      at[b] = hi;
      if (wave_first + b * kThr < items) {  // the same for the wave
        if (j0 + b * kThr + tid < items) at[b] = lo + (int64_t)r * kStep + (int64_t)lists.thread[i] * kSize;
        Piece<DT> v = Piece<DT>::lowest();
        if (at[b] + kSize <= hi) v = Piece<DT>::load(row + at[b]);
        v.unpack(x[b]);
      }
      i += di, r += dr;
      if (r >= steps) r -= steps, ++i;
    }
    const float least = bound == 0 ? -__builtin_inff() : key_value(bound);
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      if (wave_first + b * kThr >= items) continue;
      if (at[b] < hi && at[b] + kSize > hi) load_part<DT>(row, at[b], hi, x[b]);
      uint32_t reach = 0;  // elements that reach the bound's value: few
#pragma unroll
      for (int e = 0; e < kSize; ++e) reach |= x[b][e] >= least && at[b] + e < hi ? 1u << e : 0u;
      for (; reach != 0; reach &= reach - 1) {
        const int e = __builtin_ctz(reach);
        float v = x[b][0];
#pragma unroll
        for (int f = 1; f < kSize; ++f) v = e == f ? x[b][f] : v;
        const uint64_t k = top_key(v, (uint32_t)(at[b] + e));
        if (k >= bound) {
          const uint32_t to = atomicAdd(&sh.count, 1u);
          if (to < (uint32_t)kCap) lists.cand[to] = k;
        }
      }
    }
    lds_barrier();
    const uint32_t have = sh.count;
    lds_barrier();  // every thread has the same count: the next rounds add to it
    return have;
  };
  constexpr uint32_t kBatch = 2;
  bool fits = true;
  for (uint32_t j0 = 0; j0 < items && fits; j0 += kBatch * kThr) {
    const uint32_t have = rounds(j0, std::integral_constant<int, kBatch>());
    fits = have <= (uint32_t)kCap;
    if (fits && j0 + kBatch * kThr < items && have > (uint32_t)kTopFew)
      bound = top_narrow(lists.cand, (int)have, n, sh);
  }
  if (fits) return;
  // Rows in an order that piles their first elements up: from the start, a round that always fits
  // at a time.
  if (tid == 0) sh.count = 0;
  lds_barrier();
  i = tid / steps, r = tid - i * steps;
  for (uint32_t j0 = 0; j0 < items; j0 += kThr) {
    const uint32_t have = rounds(j0, std::integral_constant<int, 1>());
    if (j0 + kThr < items && have > (uint32_t)kTopFew) bound = top_narrow(lists.cand, (int)have, n, sh);
  }
}

// The candidates among the keys of `slices` (at most kMaxSlices) slices in memory, n of each, in
// order: as above. The n-th best among each slice's first few bounds them.
template <int kThr>
__device__ inline void top_collect_keys(const uint64_t* keys, int slices, int n, const TopLists<kThr>& lists,
                                        TopShared<kThr>& sh) {
  static_assert(TopLists<kThr>::kCap >= kMaxSlices * kTopMost, "every key may be a candidate");
  const int tid = (int)threadIdx.x, count = slices * n;
  const int some = (n + slices - 1) / slices + 2, per = some < n ? some : n;  // slices * per < n + 3 slices
  for (int i = tid; i < slices * per; i += kThr) lists.cand[i] = keys[i / per * n + i % per];
  if (tid == 0) sh.bound = 0, sh.count = 0;
  lds_barrier();
  top_nth(lists.cand, slices * per, n, sh);
  lds_barrier();
  const uint64_t bound = sh.bound;
  for (int i = tid; i < count; i += kThr)
    if (keys[i] != 0 && keys[i] >= bound) lists.cand[atomicAdd(&sh.count, 1u)] = keys[i];
  lds_barrier();
}

}  // namespace tsc
