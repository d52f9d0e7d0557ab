// The n first elements of a row in (value desc, id asc) order, n small, beside a pass over the row
// that is made anyway.
//
// While a thread reads its chunks of 8 elements it keeps the maximum and the first chunk that holds
// it: its key, (value, earlier chunk first). Any element among the row's n first lies in a thread
// whose key is among the n best keys: each better key stands for an element that precedes every
// element of the thread. So a bound below the n-th best key leaves few threads, whose chunks are
// read once more and compared with the bound; what reaches it is ranked.
#pragma once

#include "row_stats.h"

namespace tsc {

// Order-preserving bits of a float; -0 ties +0.
__device__ inline uint32_t order_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ inline float from_order_bits(uint32_t o) {
  return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// Keys in 64 bits, greater ones first; 0 stands for none. Of an element, or of a chunk.
__device__ inline uint64_t top_key(float x, uint32_t id) { return (uint64_t)order_bits(x) << 32 | (uint32_t)~id; }
__device__ inline float key_value(uint64_t k) { return from_order_bits((uint32_t)(k >> 32)); }
__device__ inline int32_t key_id(uint64_t k) { return (int32_t)~(uint32_t)k; }
// The least key that an element of the chunks up to this one's can have at its value.
__device__ inline uint64_t chunk_bound(uint64_t k) {
  return k == 0 ? 0 : (k >> 32 << 32) | (uint32_t)~(~(uint32_t)k * 8u + 7u);
}

constexpr int kTopThreads = 1024;
constexpr int kTopWaves = kTopThreads / kWaveSize;
constexpr int kTopMost = 128;          // n
constexpr int kTopFew = 512;           // candidates that are ranked by counting
constexpr int kTopRound = kTopThreads * 8;
constexpr int kTopCap = kTopFew + kTopRound;
constexpr int kTopPerWave = kTopMost / kTopWaves + 1;

// A workgroup's LDS for the selection: kTopLds bytes of dynamic LDS, and this.
struct TopShared {
  uint64_t wave[kTopWaves * kTopPerWave];
  uint64_t bound;
  uint32_t hist[256];
  uint32_t count, threads, digit, left;
};
struct TopLists {
  uint64_t* cand;   // [kTopCap]
  uint16_t* thread; // [kTopThreads]
  __device__ inline explicit TopLists(void* lds)
      : cand(reinterpret_cast<uint64_t*>(lds)), thread(reinterpret_cast<uint16_t*>(cand + kTopCap)) {}
};
constexpr size_t kTopLds = kTopCap * 8 + kTopThreads * 2;

// A key that at least n of the threads' keys reach, near the n-th best: the n-th best among each
// wave's best few; 0 if those are fewer than n.
__device__ inline uint64_t top_bound(uint64_t key, int n, TopShared& sh) {
  const uint32_t tid = threadIdx.x, w = tid / kWaveSize;
  const int per = (n + kTopWaves - 1) / kTopWaves + (n > 1 ? 1 : 0);  // at most kTopPerWave
  lds_barrier();  // sh may still be read by an earlier call
  for (int i = 0; i < per; ++i) {
    const uint64_t best = wave_reduce(key, MaxOp());
    if (key == best) key = 0;
    if ((tid & (kWaveSize - 1)) == 0) sh.wave[w * per + i] = best;
  }
  if (tid == 0) sh.bound = 0;
  lds_barrier();
  const int all = kTopWaves * per;
  if ((int)tid < all) {
    const uint64_t mine = sh.wave[tid];
    int above = 0;
    for (int i = 0; i < all; ++i) above += sh.wave[i] > mine;
    if (above == n - 1 && mine != 0) sh.bound = mine;
  }
  lds_barrier();
  return sh.bound;
}

// Leaves the n greatest of cand[0, c) there, in any order, and sh.count = n (n < c <= kTopCap,
// all distinct). Digit by digit from the top: a histogram of the keys that share the n-th one's
// upper digits gives its next digit. Returns the n-th greatest.
__device__ inline uint64_t top_narrow(uint64_t* cand, int c, int n, TopShared& sh) {
  constexpr int kE = (kTopCap + kTopThreads - 1) / kTopThreads;
  const int tid = (int)threadIdx.x;
  uint64_t k[kE], prefix = 0;
  lds_barrier();
#pragma unroll
  for (int i = 0; i < kE; ++i) k[i] = tid + i * kTopThreads < c ? cand[tid + i * kTopThreads] : 0;
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

// emit(r, key) for the n first of the sh.count candidates, r their place; one thread each. Fewer
// than n candidates: emit(r, 0) for the places behind them.
template <class Emit>
__device__ inline void top_emit(uint64_t* cand, int n, TopShared& sh, Emit emit) {
  lds_barrier();
  if ((int)sh.count > kTopFew) top_narrow(cand, (int)sh.count, n, sh);
  const int c = (int)sh.count, tid = (int)threadIdx.x;
  if (tid < c) {
    const uint64_t mine = cand[tid];
    int above = 0;
    for (int i = 0; i < c; ++i) above += cand[i] > mine;
    if (above < n) emit(above, mine);
  }
  if (tid >= c && tid < n) emit(tid, uint64_t{0});
}

// The candidates among row[lo, hi), lo a multiple of 8, from the threads' keys (0 of a thread that
// has read nothing), into lists.cand and sh.count: all of the n first (as many as there are) and
// few others. Thread t has read the chunks from lo + 8 t on in steps of kTopRound elements.
template <int DT>
__device__ inline void top_collect(const typename Row<DT>::Bits* row, int64_t lo, int64_t hi, uint64_t key, int n,
                                   const TopLists& lists, TopShared& sh) {
  const uint32_t tid = threadIdx.x;
  const uint64_t threads_bound = top_bound(key, n, sh);
  uint64_t bound = chunk_bound(threads_bound);
  if (tid == 0) sh.count = 0, sh.threads = 0;
  lds_barrier();
  if (key != 0 && key >= threads_bound) lists.thread[atomicAdd(&sh.threads, 1u)] = (uint16_t)tid;
  lds_barrier();
  const uint32_t steps = (uint32_t)((hi - lo + kTopRound - 1) / kTopRound);
  const uint32_t items = sh.threads * steps;  // at most 2^10 * 2^18
  for (uint32_t j0 = 0; j0 < items; j0 += kTopThreads) {
    const uint32_t j = j0 + tid;
    if (j < items) {
      const uint32_t i = j / steps;
      const int64_t at = lo + (int64_t)(j - i * steps) * kTopRound + (int64_t)lists.thread[i] * 8;
      if (at < hi) {
        float x[8];
        load8<DT>(row, at, hi, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint64_t k = top_key(x[e], (uint32_t)(at + e));
          if (k >= bound && at + e < hi) lists.cand[atomicAdd(&sh.count, 1u)] = k;
        }
      }
    }
    lds_barrier();
    const uint32_t have = sh.count;
    lds_barrier();  // every thread has the same count: the next round adds to it
    // Room for another round. Rows in an order that piles their first elements up get here.
    if (j0 + kTopThreads < items && have > (uint32_t)kTopFew) bound = top_narrow(lists.cand, (int)have, n, sh);
  }
}

// The candidates among `count` keys (0: none) in memory: as above.
__device__ inline void top_collect_keys(const uint64_t* keys, int count, int n, const TopLists& lists, TopShared& sh) {
  const int tid = (int)threadIdx.x;
  uint64_t key = 0;
  for (int i = tid; i < count; i += kTopThreads) key = key > keys[i] ? key : keys[i];
  const uint64_t bound = top_bound(key, n, sh);
  if (tid == 0) sh.count = 0;
  lds_barrier();
  for (int i = tid; i < count; i += kTopThreads)  // at most kTopCap
    if (keys[i] != 0 && keys[i] >= bound) lists.cand[atomicAdd(&sh.count, 1u)] = keys[i];
  lds_barrier();
}

}  // namespace tsc
