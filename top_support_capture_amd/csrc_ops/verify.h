// Speculative verification of drafted tokens (exact acceptance and recovery): with p the target's
// distribution at a position and q the drafter's, draft d is accepted iff u q(d) < p(d), u a
// given uniform; at the first draft that is not, the token is drawn from max(p - q, 0), and after
// the last accepted one from the target's next position. What is emitted is then distributed as
// p alone would give it. The draws are exponential races, argmax w_i / E_i, as the sampler's.
//
// On logits, two launches: every slice of every row gives its softmax statistics (row_stats.h);
// then several workgroups per request merge them, decide where the request stops, and race over
// the vocabulary of that position alone, each over a share of it. The last one to finish a
// request joins the shares' winners.
#pragma once

#include "row_stats.h"
#include "tsc_verify.h"

namespace tsc {

struct VerifyArgs {
  const void* target;  // [N, K + 1, V]
  int64_t t_sn, t_sk;  // strides in elements
  const void* draft;   // [N, K, V] or null: drafts without a distribution (q is 1 at the draft)
  int64_t d_sn, d_sk;
  int32_t t_dtype, d_dtype;
  int64_t N, V;
  int32_t K;
  const float* temperature;        // [N]
  const float* draft_temperature;  // [N] or null: temperature
  const int32_t* draft_tokens;     // [N, K]
  const int32_t* draft_counts;     // [N] or null: K
  const float* uniforms;           // [N, K]
  const uint64_t* seeds;
  const uint64_t* positions;
  int32_t* tokens;    // [N, K + 1]
  int32_t* accepted;  // [N]
  float* logprobs;    // [N, K + 1]
  int8_t* row_status; // [N]
  // Workspace.
  RowPart* parts;     // [N, rows, slices]
  struct RacePart* best;  // [N, shares]
  uint32_t* arrived;  // [N]
  int32_t rows;       // K + 1 target rows, then K draft rows when there is a draft distribution
  int32_t slices, shares;
  int64_t slice_len, share_len;
};

// The best entry of a race: its score w / E (0 when nothing takes part) and its id.
struct RacePart {
  double score;
  int32_t id;
  int32_t pad;
};

__device__ inline RacePart better(RacePart a, RacePart b) {
  return b.score > a.score || (b.score == a.score && b.id < a.id) ? b : a;
}

// Softmax statistics of each row's slices; greedy requests take the maximum's place of each
// target row instead and read no draft row.
template <int TD, int DD>
__global__ void __launch_bounds__(kOpThreads) verify_stats_kernel(VerifyArgs a) {
  __shared__ float sh_m[kOpWaves];
  __shared__ double sh_s[kOpWaves];
  __shared__ int32_t sh_at[kOpWaves];
  const int64_t per = (int64_t)a.rows * a.slices;
  for (int64_t item = blockIdx.x; item < a.N * per; item += gridDim.x) {
    const int64_t n = item / per, rest = item - n * per;
    const int32_t r = (int32_t)(rest / a.slices), sl = (int32_t)(rest - (int64_t)r * a.slices);
    if (rest == 0 && threadIdx.x == 0) a.arrived[n] = 0u;
    const float T = a.temperature[n];
    const bool is_draft = r > a.K;
    const int32_t i = is_draft ? r - a.K - 1 : r;
    const int32_t count = a.draft_counts ? a.draft_counts[n] : a.K;
    if (i > count - (is_draft ? 1 : 0)) continue;  // uniform over the workgroup, as is all below
    const int64_t lo = sl * a.slice_len, hi = lo + a.slice_len < a.V ? lo + a.slice_len : a.V;
    RowPart* out = a.parts + item;
    if (T == 0.0f) {
      if (is_draft) continue;
      slice_argmax<TD>((const typename Row<TD>::Bits*)a.target + n * a.t_sn + i * a.t_sk, lo, hi,
                       sh_m, sh_s, sh_at, out);
    } else if (!is_draft) {
      slice_stats<TD>((const typename Row<TD>::Bits*)a.target + n * a.t_sn + i * a.t_sk, lo, hi,
                      make_scale(T), sh_m, sh_s, out);
    } else {
      const float Td = a.draft_temperature ? a.draft_temperature[n] : T;
      slice_stats<DD>((const typename Row<DD>::Bits*)a.draft + n * a.d_sn + i * a.d_sk, lo, hi,
                      make_scale(Td), sh_m, sh_s, out);
    }
    lds_barrier();  // the shared states are written again by the next item
  }
}

// t = 1 - u of a Philox word: u = (2 (word >> 9) + 1) / 2^24, both exact in float32.
__device__ inline float race_t(uint32_t word) {
  return (float)(0x1000000u - (2u * (word >> 9) + 1u)) * 0x1p-24f;
}

// E = -ln u = -ln(1 - t) to about 1e-6 relative: the series for small t (t^6 / 7 below 2^-26),
// where the logarithm of a u near 1 would keep few digits.
__device__ inline float race_exponential(float t) {
  const float series =
      t * (1.0f + t * (0.5f + t * (1.0f / 3 + t * (0.25f + t * (0.2f + t * (1.0f / 6))))));
  return t < 0.0625f ? series : -0.69314718f * __builtin_amdgcn_logf(1.0f - t);
}

// A race is run in float32 and decided in float64: each thread keeps its best entry by the
// float32 score, and the threads whose score is within kRaceClose of the best one evaluate
// theirs again in float64. (Two entries that close within one thread of the many are the
// float32 score's to order.) float32 holds p and q to about 2e-6, exponents down to -40 rounded.
// A difference p - q below p / 64 would keep too little of that: such a weight is evaluated in
// float64 at once, but only if its upper bound, (p - q) + p kRaceSlack, can still win.
constexpr float kRaceClose = 1e-3f, kRaceSlack = 1e-4f, kRaceNear = 1.0f / 64;

struct RaceEntry {
  float score = 0.0f, t = 0.5f;
  float a = 0.0f, b = 0.0f;  // what the exact weight is computed from
  int32_t id = INT32_MAX;
  // E >= t: an entry whose w / t is no better than `bound` cannot win, and is spared the rest.
  __device__ inline void offer(float w, float tt, int32_t i, float a_, float b_, float bound) {
    if (w > bound * tt) {
      const float sc = w / race_exponential(tt);
      if (sc > score || (sc == score && i < id)) score = sc, t = tt, a = a_, b = b_, id = i;
    }
  }
  // The same for a weight p - q of close terms; exact() is its float64 value.
  template <class Exact>
  __device__ inline void offer_near(float p, float w, float tt, int32_t i, float a_, float b_,
                                    float bound, Exact exact) {
    if (race_near(p, w) && w + p * kRaceSlack > bound * tt) {
      const float we = (float)exact(a_, b_);
      if (we > 0.0f) offer(we, tt, i, a_, b_, bound);
    }
  }
  __device__ static inline bool race_near(float p, float w) { return __builtin_fabsf(w) < p * kRaceNear; }
};

// The winner among the workgroup's entries; weight(a, b) is the exact weight.
template <int kW, class Weight>
__device__ inline RacePart race_winner(const RaceEntry& e, Weight weight, float* sh_score,
                                       RacePart* sh_best) {
  const uint32_t w = threadIdx.x / kWaveSize, lane = threadIdx.x & (kWaveSize - 1);
  const float wave = wave_max(e.score);
  if (lane == 0) sh_score[w] = wave;
  lds_barrier();
  float top = sh_score[0];
#pragma unroll
  for (int i = 1; i < kW; ++i) top = __builtin_fmaxf(top, sh_score[i]);
  RacePart b{0.0, INT32_MAX, 0};
  if (wave > 0.0f && wave >= top * (1.0f - kRaceClose)) {  // wave-uniform
    if (e.score > 0.0f && e.score >= top * (1.0f - kRaceClose)) {
      const double sc = weight(e.a, e.b) / -log1p(-(double)e.t);
      if (sc > 0.0) b = {sc, e.id, 0};
    }
    const double best = wave_reduce(b.score, MaxOp());
    b.id = wave_reduce(b.score == best ? b.id : INT32_MAX, MinOp());
    b.score = best;
  }
  if (lane == 0) sh_best[w] = b;
  lds_barrier();
  b = sh_best[0];
#pragma unroll
  for (int i = 1; i < kW; ++i) b = better(b, sh_best[i]);
  return b;
}

// Where a request stops, and why: filled in by decide().
struct Decision {
  int32_t stop;    // index of the first draft that is not accepted; the count when all are
  int32_t code;    // kRejected, kBonus, or kStatus + a row status
};
enum { kAccepted = 0, kRejected = 1, kBonus = 2, kStatus = 16 };

constexpr int kMaxDrafts = TSC_MAX_DRAFTS;

__device__ inline int32_t part_status(const RowPart& p) {
  if (!(p.s < __builtin_inf()) || p.m == __builtin_inff()) return TSC_ROW_NONFINITE;
  return p.m == -__builtin_inff() ? TSC_ROW_NO_SUPPORT : TSC_ROW_OK;
}

// The first position whose code is not kAccepted among 0..count (its code is never kAccepted).
__device__ inline Decision first_stop(const int32_t* code, int32_t count, int32_t* sh_stop) {
  if (threadIdx.x == 0) *sh_stop = count;
  lds_barrier();
  for (int32_t i = threadIdx.x; i <= count; i += blockDim.x)
    if (code[i] != kAccepted) atomicMin(sh_stop, i);
  lds_barrier();
  const int32_t stop = *sh_stop;
  return {stop, code[stop]};
}

template <int TD, int DD>
__global__ void __launch_bounds__(kOpThreads) verify_race_kernel(VerifyArgs a) {
  __shared__ RowPart tp[kMaxDrafts + 1], dp[kMaxDrafts];
  __shared__ int32_t code[kMaxDrafts + 1];
  __shared__ float xt[kMaxDrafts];
  __shared__ int32_t sh_stop;
  __shared__ float sh_score[kOpWaves];
  __shared__ RacePart sh_best[kOpWaves];
  __shared__ uint32_t sh_last;
  using TB = typename Row<TD>::Bits;
  using DB = typename Row<DD>::Bits;
  const int64_t n = blockIdx.x / a.shares;
  const int32_t share = (int32_t)(blockIdx.x - n * a.shares);
  const uint32_t tid = threadIdx.x, lane = tid & (kWaveSize - 1), w = tid / kWaveSize;
  const int32_t K = a.K;
  const int32_t count = a.draft_counts ? a.draft_counts[n] : K;
  const float T = a.temperature[n];
  const bool greedy = T == 0.0f;
  const bool has_draft = a.draft != nullptr && !greedy;
  const float Td = has_draft ? (a.draft_temperature ? a.draft_temperature[n] : T) : 1.0f;
  const TB* trow = (const TB*)a.target + n * a.t_sn;
  const DB* drow = (const DB*)a.draft + n * a.d_sn;
  int32_t* out_tok = a.tokens + n * (K + 1);
  float* out_lp = a.logprobs + n * (K + 1);

  auto refuse = [&](int32_t status) {
    if (share != 0) return;
    for (int32_t j = tid; j <= K; j += kOpThreads) out_tok[j] = -1, out_lp[j] = __builtin_nanf("");
    if (tid == 0) a.accepted[n] = 0, a.row_status[n] = (int8_t)status;
  };
  if (count < 0 || count > K || !(greedy || temperature_ok(T)) || !temperature_ok(Td)) {
    refuse(TSC_ROW_INVALID_PARAM);
    return;
  }
  const Scale ct = make_scale(greedy ? 1.0f : T), cd = make_scale(Td);

  // Every row's state from its slices': a wave a row, a lane a slice.
  const RowPart none{-__builtin_inff(), INT32_MAX, 0.0};
  for (int32_t r = (int32_t)w; r < a.rows; r += kOpWaves) {
    const bool is_draft = r > K;
    const int32_t i = is_draft ? r - K - 1 : r;
    if (i > count - (is_draft ? 1 : 0) || (is_draft && !has_draft)) continue;  // wave-uniform
    const RowPart v = (int32_t)lane < a.slices ? a.parts[(n * a.rows + r) * a.slices + lane] : none;
    RowPart p = merge_slices(v, is_draft ? cd : ct);
    if (greedy && p.s == p.s) p.s = 1.0;
    if (lane == 0) (is_draft ? dp[i] : tp[i]) = p;
  }
  lds_barrier();
  for (int32_t i = (int32_t)tid; i <= count; i += kOpThreads) {
    const RowPart t = tp[i];
    int32_t st = part_status(t), c = kBonus;
    if (i < count) {
      const int32_t d = a.draft_tokens[n * K + i];
      const float u = a.uniforms[n * K + i];
      const bool valid = d >= 0 && d < a.V && u >= 0.0f && u < 1.0f;
      if (has_draft && st == TSC_ROW_OK) st = part_status(dp[i]);
      if (!valid) st = TSC_ROW_INVALID_PARAM;
      if (st == TSC_ROW_OK) {
        if (greedy) {
          c = d == t.at ? kAccepted : kRejected;
          xt[i] = t.m;
        } else {
          xt[i] = Row<TD>::get(trow + i * a.t_sk + d);
          const double p = exp(((double)xt[i] - (double)t.m) / (double)T) / t.s;
          double q = 1.0;
          if (has_draft) {
            const float xd = Row<DD>::get(drow + i * a.d_sk + d);
            q = exp(((double)xd - (double)dp[i].m) / (double)Td) / dp[i].s;
          }
          c = (double)u * q < p ? kAccepted : kRejected;
        }
      }
    }
    code[i] = st == TSC_ROW_OK ? c : kStatus + st;
  }
  const Decision dec = first_stop(code, count, &sh_stop);
  if (dec.code >= kStatus) {
    refuse(dec.code - kStatus);
    return;
  }
  const int32_t stop = dec.stop;
  const RowPart t = tp[stop];

  // The request's outputs, once its last token is known.
  auto finish = [&](int32_t token) {
    for (int32_t j = (int32_t)tid; j <= K; j += kOpThreads) {
      int32_t id = -1;
      float lp = __builtin_nanf("");
      if (j <= stop) {
        const float x = j < stop ? xt[j] : Row<TD>::get(trow + (int64_t)stop * a.t_sk + token);
        id = j < stop ? a.draft_tokens[n * K + j] : token;
        lp = greedy ? 0.0f : (float)(((double)x - (double)tp[j].m) / (double)T - log(tp[j].s));
      }
      out_tok[j] = id, out_lp[j] = lp;
    }
    if (tid == 0) a.accepted[n] = stop, a.row_status[n] = TSC_ROW_OK;
  };
  if (greedy) {
    if (share == 0) finish(t.at);
    return;
  }

  // The race over this workgroup's share of the vocabulary.
  const bool rejected = dec.code == kRejected;
  const int32_t drafted = rejected ? a.draft_tokens[n * K + stop] : -1;
  const bool subtract = rejected && has_draft;
  const RowPart d = subtract ? dp[stop] : RowPart{0.0f, 0, 1.0};
  const float inv_t = (float)(1.0 / t.s), inv_d = (float)(1.0 / d.s);
  const TB* tr = trow + (int64_t)stop * a.t_sk;
  const DB* dr = drow + (int64_t)stop * a.d_sk;
  const uint64_t seed = a.seeds[n], position = a.positions[n] + (uint64_t)stop;
  const int64_t lo = share * a.share_len, hi = lo + a.share_len < a.V ? lo + a.share_len : a.V;
  auto exact = [&](float xe, float ye) -> double {
    double p = exp(((double)xe - (double)t.m) / (double)T) / t.s;
    if (subtract) p -= exp(((double)ye - (double)d.m) / (double)Td) / d.s;
    return p;
  };
  RaceEntry best;
  float bound = 0.0f;  // the wave's best score so far, less the slack
  for (int64_t at = lo + (int64_t)tid * 8; at - (int64_t)lane * 8 < hi; at += (int64_t)kOpThreads * 8) {
    float x[8], y[8] = {}, p[8], wt[8];
    load8<TD>(tr, at, hi, x);
    if (subtract) load8<DD>(dr, at, hi, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = exp2_scaled(x[e] - t.m, ct) * inv_t;
      wt[e] = p[e];
      if (subtract) wt[e] -= exp2_scaled(y[e] - d.m, cd) * inv_d;
      if (!subtract && at + e == drafted) p[e] = wt[e] = 0.0f;
    }
    float tt[8];
    bool drawn[2];  // wave-uniform
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float most = 0.0f;
#pragma unroll
      for (int e = 4 * h; e < 4 * h + 4; ++e) most = __builtin_fmaxf(most, wt[e] + p[e] * kRaceSlack);
      // t is at least 2^-24: below that share of the bound no word wins, and none is drawn.
      drawn[h] = __ballot(most > bound * 0x1p-24f) != 0;
      if (!drawn[h]) continue;
      const uint32_t id0 = (uint32_t)at + 4u * h;
      const uint4 r = philox4x32_10(
          make_uint4(id0 >> 2, rejected ? 1u : 0u, (uint32_t)position, (uint32_t)(position >> 32)),
          (uint32_t)seed, (uint32_t)(seed >> 32));
      const uint32_t word[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int e = 4 * h; e < 4 * h + 4; ++e) {
        tt[e] = race_t(word[e & 3]);
        if (!(subtract && RaceEntry::race_near(p[e], wt[e])))
          best.offer(wt[e], tt[e], (int32_t)(at + e), x[e], y[e], bound);
      }
    }
    if (drawn[0] || drawn[1]) bound = wave_max(best.score) * (1.0f - kRaceClose);
    if (subtract) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (drawn[e >> 2])
          best.offer_near(p[e], wt[e], tt[e], (int32_t)(at + e), x[e], y[e], bound, exact);
    }
  }
  const RacePart won = race_winner<kOpWaves>(best, exact, sh_score, sh_best);
  if (tid == 0) {
    RacePart* slot = a.best + n * a.shares + share;
    __hip_atomic_store(&slot->id, won.id, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(reinterpret_cast<uint64_t*>(&slot->score), __builtin_bit_cast(uint64_t, won.score),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sh_last = __hip_atomic_fetch_add(&a.arrived[n], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
              (uint32_t)a.shares - 1u;
  }
  lds_barrier();
  if (sh_last == 0u) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  RacePart b{0.0, INT32_MAX, 0};
  if ((int32_t)lane < a.shares) {
    const RacePart* slot = a.best + n * a.shares + lane;
    b.id = __hip_atomic_load(&slot->id, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    b.score = __builtin_bit_cast(
        double, __hip_atomic_load(reinterpret_cast<const uint64_t*>(&slot->score), __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_AGENT));
  }
  const double top = wave_reduce(b.score, MaxOp());
  b.id = wave_reduce(b.score == top ? b.id : INT32_MAX, MinOp());
  b.score = top;
  // No token with p > q: the two distributions agree within rounding, and the draft is as good
  // a draw from p as any.
  finish(b.score > 0.0 ? b.id : drafted);
}

// ---- Over captured supports ---------------------------------------------------------------------
// A capture slot lists a position's support: its ids, their logprobs (normalised over the
// support) and their number. One workgroup per request: its waves look the drafts up in the
// lists, all positions at once; at the position where the request stops, the drafter's list goes
// into a hash table in LDS that the target's entries look themselves up in, and race.
struct SupportArgs {
  const int32_t* ids;      // slot i of request n at (n * sn + i * sk) * W
  const float* logprobs;   // likewise
  const int32_t* lengths;  // at n * sn + i * sk
  const int8_t* status;    // likewise, or null (every slot is complete)
  int64_t sn, sk;
  int32_t W;
};

struct CapturedArgs {
  SupportArgs target, draft;  // draft.ids null: drafts without a distribution
  int64_t N;
  int32_t K;
  const int32_t* draft_tokens;  // [N, K]
  const int32_t* draft_counts;  // [N] or null: K
  const float* uniforms;        // [N, K]
  const uint64_t* seeds;
  const uint64_t* positions;
  int32_t* tokens;     // [N, K + 1]
  int32_t* accepted;   // [N]
  float* logprobs;     // [N, K + 1]
  int8_t* row_status;  // [N]
};

constexpr int kCapThreads = 512;
constexpr int kCapWaves = kCapThreads / kWaveSize;

// The slot's status: a capture that is not whole cannot be verified against.
__device__ inline int32_t slot_status(const SupportArgs& s, int64_t slot) {
  const int32_t st = s.status ? (int32_t)s.status[slot] : TSC_ROW_OK;
  if (st != TSC_ROW_OK) return st;
  const int32_t n = s.lengths[slot];
  return n >= 1 && n <= s.W ? TSC_ROW_OK : TSC_ROW_INVALID_PARAM;
}

__device__ inline uint32_t id_hash(int32_t id) { return (uint32_t)id * 0x9E3779B1u; }

// 2^(lp log2 e) for the filter; lp is at most 0 and -inf gives 0.
__device__ inline float exp_fast(float lp) {
  return __builtin_amdgcn_exp2f(lp * 1.44269504f);
}

__global__ void __launch_bounds__(kCapThreads) verify_captured_kernel(CapturedArgs a) {
  // Index into the draft's list + 1, or 0; the launch gives it twice draft.W slots or more.
  extern __shared__ uint32_t table[];
  __shared__ float lp_t[kMaxDrafts], lp_d[kMaxDrafts];
  __shared__ int32_t code[kMaxDrafts + 1];
  __shared__ int32_t sh_stop;
  __shared__ float sh_score[kCapWaves];
  __shared__ RacePart sh_best[kCapWaves];
  __shared__ float sh_lp;
  const int64_t n = blockIdx.x;
  const uint32_t tid = threadIdx.x, lane = tid & (kWaveSize - 1);
  const int32_t w = __builtin_amdgcn_readfirstlane((int)(tid / kWaveSize));
  const int32_t K = a.K;
  const int32_t count = a.draft_counts ? a.draft_counts[n] : K;
  int32_t* out_tok = a.tokens + n * (K + 1);
  float* out_lp = a.logprobs + n * (K + 1);
  auto refuse = [&](int32_t status) {
    for (int32_t j = tid; j <= K; j += kCapThreads) out_tok[j] = -1, out_lp[j] = __builtin_nanf("");
    if (tid == 0) a.accepted[n] = 0, a.row_status[n] = (int8_t)status;
  };
  if (count < 0 || count > K) {
    refuse(TSC_ROW_INVALID_PARAM);
    return;
  }
  const bool has_draft = a.draft.ids != nullptr;
  for (int32_t i = (int32_t)tid; i < count; i += kCapThreads)
    lp_t[i] = -__builtin_inff(), lp_d[i] = has_draft ? -__builtin_inff() : 0.0f;
  lds_barrier();
  // The drafts' logprobs in both lists (-inf where they are not in them).
  for (int32_t j = w; j < (has_draft ? 2 : 1) * count; j += kCapWaves) {
    const bool is_draft = j >= count;
    const int32_t i = is_draft ? j - count : j;
    const SupportArgs& s = is_draft ? a.draft : a.target;
    const int64_t slot = n * s.sn + i * s.sk;
    if (slot_status(s, slot) != TSC_ROW_OK) continue;
    const int32_t len = s.lengths[slot], want = a.draft_tokens[n * K + i];
    const int32_t* ids = s.ids + slot * s.W;
    constexpr int kU = 8;
    for (int32_t e0 = (int32_t)lane; e0 < len; e0 += kWaveSize * kU) {
      int32_t id[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) id[u] = e0 + u * kWaveSize < len ? ids[e0 + u * kWaveSize] : ~want;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (id[u] == want) (is_draft ? lp_d : lp_t)[i] = s.logprobs[slot * s.W + e0 + u * kWaveSize];
    }
  }
  lds_barrier();
  for (int32_t i = (int32_t)tid; i <= count; i += kCapThreads) {
    int32_t st = slot_status(a.target, n * a.target.sn + i * a.target.sk), c = kBonus;
    if (i < count) {
      if (has_draft && st == TSC_ROW_OK) st = slot_status(a.draft, n * a.draft.sn + i * a.draft.sk);
      const float u = a.uniforms[n * K + i];
      if (!(u >= 0.0f && u < 1.0f) || a.draft_tokens[n * K + i] < 0) st = TSC_ROW_INVALID_PARAM;
      c = (double)u * exp((double)lp_d[i]) < exp((double)lp_t[i]) ? kAccepted : kRejected;
    }
    code[i] = st == TSC_ROW_OK ? c : kStatus + st;
  }
  const Decision dec = first_stop(code, count, &sh_stop);
  if (dec.code >= kStatus) {
    refuse(dec.code - kStatus);
    return;
  }
  const int32_t stop = dec.stop;
  const bool rejected = dec.code == kRejected;
  const int32_t drafted = rejected ? a.draft_tokens[n * K + stop] : -1;
  const bool subtract = rejected && has_draft;
  const int64_t t_slot = n * a.target.sn + stop * a.target.sk;
  const int32_t t_len = a.target.lengths[t_slot];
  const int32_t* t_ids = a.target.ids + t_slot * a.target.W;
  const float* t_lps = a.target.logprobs + t_slot * a.target.W;
  const int32_t* d_ids = nullptr;
  const float* d_lps = nullptr;
  uint32_t mask = 0;
  if (subtract) {
    const int64_t d_slot = n * a.draft.sn + stop * a.draft.sk;
    const int32_t d_len = a.draft.lengths[d_slot];
    d_ids = a.draft.ids + d_slot * a.draft.W;
    d_lps = a.draft.logprobs + d_slot * a.draft.W;
    uint32_t slots = 64;  // a power of two, at least twice the entries: every probe ends
    while (slots < 2u * (uint32_t)d_len) slots <<= 1;
    mask = slots - 1u;
    for (uint32_t i = tid; i < slots; i += kCapThreads) table[i] = 0u;
    lds_barrier();
    // A slot holds the entry's index + 1 (at most 16384) and 17 bits of the id's hash beside it, so
    // that an entry of another id rarely costs a read of its id.
    for (int32_t e = (int32_t)tid; e < d_len; e += kCapThreads) {
      const uint32_t h = id_hash(d_ids[e]);
      const uint32_t v = (h << 15) | (uint32_t)(e + 1);
      uint32_t at = (h >> 17) & mask;
      while (atomicCAS(&table[at], 0u, v) != 0u) at = (at + 1u) & mask;
    }
    lds_barrier();
  }
  const uint64_t seed = a.seeds[n], position = a.positions[n] + (uint64_t)stop;
  const uint32_t lo = (uint32_t)position, hi = (uint32_t)(position >> 32);
  auto exact = [](float lp, float lq) -> double { return exp((double)lp) - exp((double)lq); };
  RaceEntry best;
  for (int32_t e = (int32_t)tid; e < t_len; e += kCapThreads) {
    const int32_t id = t_ids[e];
    const float lp = t_lps[e];
    float lq = -__builtin_inff();
    if (subtract) {
      const uint32_t h = id_hash(id);
      for (uint32_t at = (h >> 17) & mask;; at = (at + 1u) & mask) {
        const uint32_t v = table[at];
        if (v == 0u) break;
        if ((v >> 15) == (h & 0x1FFFFu) && d_ids[(v & 0x7FFFu) - 1u] == id) {
          lq = d_lps[(v & 0x7FFFu) - 1u];
          break;
        }
      }
    } else if (id == drafted) {
      continue;
    }
    const float p = exp_fast(lp), wt = p - exp_fast(lq);
    const bool near = RaceEntry::race_near(p, wt);
    if (wt > 0.0f || near) {
      const uint4 r = philox4x32_10(make_uint4((uint32_t)id >> 2, rejected ? 1u : 0u, lo, hi),
                                    (uint32_t)seed, (uint32_t)(seed >> 32));
      const uint32_t j = (uint32_t)id & 3u;
      const float tt = race_t(j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w);
      const float bound = best.score * (1.0f - kRaceClose);
      if (near)
        best.offer_near(p, wt, tt, id, lp, lq, bound, exact);
      else
        best.offer(wt, tt, id, lp, lq, bound);
    }
  }
  const RacePart won = race_winner<kCapWaves>(best, exact, sh_score, sh_best);
  // No token with p > q: the two distributions agree within rounding, and the draft is as good a
  // draw from p as any. (The bonus draw has no such case, unless no logprob is a number.)
  if (won.score <= 0.0 && !rejected) {
    refuse(TSC_ROW_NONFINITE);
    return;
  }
  const int32_t token = won.score > 0.0 ? won.id : drafted;
  if (won.score > 0.0 ? best.id == token : false) sh_lp = best.a;
  if (tid == 0 && !(won.score > 0.0)) sh_lp = lp_t[stop];
  lds_barrier();
  for (int32_t j = (int32_t)tid; j <= K; j += kCapThreads) {
    out_tok[j] = j < stop ? a.draft_tokens[n * K + j] : j == stop ? token : -1;
    out_lp[j] = j < stop ? lp_t[j] : j == stop ? sh_lp : __builtin_nanf("");
  }
  if (tid == 0) a.accepted[n] = stop, a.row_status[n] = TSC_ROW_OK;
}

}  // namespace tsc
