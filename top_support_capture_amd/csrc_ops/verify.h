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
  uint64_t* score;    // [N, shares]: the score of each share's winner, the bits of a double
  uint32_t* winner;   // [N, shares]: its id
  uint32_t* arrived;  // [N]: shares that are done
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
// target row instead and read no draft row. Bound by reading: 64 requests of 4 drafts over 151936
// bfloat16 logits, 175 MB, take 36 us (4.8 TB/s; a bare read in workgroups of this size 34 us); 4 to
// 8 waves a SIMD, slices of 16384 to 100000 elements and fewer vector instructions all measure the
// same. (One request: 4.4 us.)
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
    if (T == 0.0f && is_draft) continue;
    const float Ti = is_draft && a.draft_temperature ? a.draft_temperature[n] : T;
    const int64_t start = is_draft ? n * a.d_sn + i * a.d_sk : n * a.t_sn + i * a.t_sk;
    const auto* row = (const typename Row<TD>::Bits*)(is_draft ? a.draft : a.target) + start;
    if (T == 0.0f) {
      slice_argmax<TD>(row, lo, hi, sh_m, sh_s, sh_at, out);
    } else if (TD == DD || !is_draft) {
      slice_stats<TD>(row, lo, hi, make_scale(Ti), sh_m, sh_s, out);
    } else {
      slice_stats<DD>((const typename Row<DD>::Bits*)a.draft + start, lo, hi, make_scale(Ti), sh_m, sh_s, out);
    }
    lds_barrier();  // the shared states are written again by the next item
  }
}

// Philox4x32-10 (Salmon et al., SC'11) of the sampler's race, several counters at once: a round's
// product and exclusive-ors depend on the last round's, so that independent counters side by side
// fill the pipeline, and gfx950 takes the exclusive-or of three words in one operation.
__device__ inline uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// Words of N groups of four ids (id / 4, in out[i][0] at first), under counter word 1 = `stream`.
template <int N>
__device__ inline void race_words(uint32_t stream, uint64_t seed, uint64_t position, uint32_t (&out)[N][4]) {
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < N; ++i)
    out[i][1] = stream, out[i][2] = (uint32_t)position, out[i][3] = (uint32_t)(position >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t a = (uint64_t)0xD2511F53u * out[i][0], b = (uint64_t)0xCD9E8D57u * out[i][2];
      out[i][0] = xor3((uint32_t)(b >> 32), out[i][1], k0), out[i][1] = (uint32_t)b;
      out[i][2] = xor3((uint32_t)(a >> 32), out[i][3], k1), out[i][3] = (uint32_t)a;
    }
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
}

__device__ inline uint32_t word_of(const uint32_t (&w)[4], uint32_t id) {
  const uint32_t j = id & 3u;
  return j == 0 ? w[0] : j == 1 ? w[1] : j == 2 ? w[2] : w[3];
}

__device__ inline uint32_t race_word(uint32_t id, uint32_t stream, uint64_t seed, uint64_t position) {
  uint32_t w[1][4] = {{id >> 2}};
  race_words(stream, seed, position, w);
  return word_of(w[0], id);
}

// t = 1 - u of a Philox word: u = (2 (word >> 9) + 1) / 2^24, all exact in float32.
__device__ inline float race_t(uint32_t word) {
  return __builtin_fmaf((float)(word >> 9), -0x1p-23f, 1.0f - 0x1p-24f);
}

// E = -ln u = -ln(1 - t) to about 1e-6 relative: the series for small t (t^6 / 7 below 2^-26),
// where the logarithm of a u near 1 would keep few digits.
__device__ inline float race_exponential(float t) {
  const float series =
      t * (1.0f + t * (0.5f + t * (1.0f / 3 + t * (0.25f + t * (0.2f + t * (1.0f / 6))))));
  return t < 0.0625f ? series : -0.69314718f * __builtin_amdgcn_logf(1.0f - t);
}

__device__ inline double race_exponential_64(float t) { return -log1p(-(double)t); }

// A race is run in float32 and decided in float64: each thread keeps its best entry, by the float32
// scores where they are kRaceClose apart and by float64 ones where they are not, and the threads
// whose score is within kRaceClose of the best one evaluate theirs in float64, as do the shares of
// a request. float32 holds p and q to about 2e-6, exponents down to -40 rounded.
// A difference p - q below p / 64 would keep too little of that: such a weight is evaluated in
// float64. An entry comes that far only if the upper bound of its weight, (p - q) + p kRaceSlack,
// can still win, which few entries' do.
constexpr float kRaceClose = 1e-3f, kRaceSlack = 1e-4f, kRaceNear = 1.0f / 64;

// The filter's probability of a logit: the logarithm of 1 / s is part of the exponent, and one
// float32 c does (its error is within the margins).
__device__ inline float weight_of(float x, float m, float c, float minus_lg_s) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(x - m, c, minus_lg_s));
}

struct RaceEntry {
  float score = 0.0f, t = 0.5f;
  float a = 0.0f, b = 0.0f;  // what the exact weight is computed from
  int32_t id = INT32_MAX;
  // An entry of weight p - q; exact() is the float64 value.
  template <class Exact>
  __device__ inline void offer(float p, float q, int32_t i, float tt, float a_, float b_, Exact exact) {
    float w = p - q;
    if (race_near(p, w)) w = (float)exact(a_, b_);
    const float sc = w * __builtin_amdgcn_rcpf(race_exponential(tt));
    if (!(sc > score * (1.0f - kRaceClose))) return;
    if (score > 0.0f && sc * (1.0f - kRaceClose) < score) {
      const double mine = exact(a, b) / race_exponential_64(t), other = exact(a_, b_) / race_exponential_64(tt);
      if (other < mine || (other == mine && id < i)) return;
    }
    score = sc, t = tt, a = a_, b = b_, id = i;
  }
  __device__ static inline bool race_near(float p, float w) { return __builtin_fabsf(w) < p * kRaceNear; }
  // E >= t: an entry whose largest possible w / t is no better than `bound` cannot win.
  __device__ static inline bool can_win(float p, float w, float tt, float bound) {
    return __builtin_fmaf(p, kRaceSlack, w) > bound * tt;
  }
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
      const double sc = weight(e.a, e.b) / race_exponential_64(e.t);
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

// Where a request stops, and why.
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

// The race at the position where a request stops: 28 us for 64 requests over 151936 logits, 13 us for
// one request. Philox and the weights, about 1300 cycles of a SIMD for 512 elements, are 10 us of the
// batch's; the rest of both is a chain of dependent steps (merge and decision 5 and 4 us, first loads
// 1, winner 2, the shares' meeting 1) and, on a batch, uneven shares. Requests are shared out so that
// there are about 512 workgroups (384, 640, 768 and 1024: 30.6, 29.9, 27.8 and 27.8 us against 28.0).
template <int TD, int DD>
__global__ void __launch_bounds__(kOpThreads, 4) verify_race_kernel(VerifyArgs a) {
  __shared__ RowPart tp[kMaxDrafts + 1], dp[kMaxDrafts];
  __shared__ int32_t code[kMaxDrafts + 1];
  __shared__ float xt[kMaxDrafts];
  __shared__ int32_t sh_stop;
  __shared__ uint32_t sh_bound;
  __shared__ float sh_score[kOpWaves];
  __shared__ RacePart sh_best[kOpWaves];
  __shared__ int32_t sh_token;
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
  // What the decisions need is asked for at once, each load a microsecond when there is little else
  // to do: the states of the slices of the wave's first kRows rows, and thread i's draft i.
  constexpr int kRows = 4;
  const RowPart none{-__builtin_inff(), INT32_MAX, 0.0};
  auto part_of = [&](int32_t r) {  // rows past the counts hold nothing, and are not used
    r = r < a.rows ? r : a.rows - 1;
    const RowPart p = a.parts[(n * a.rows + r) * a.slices + ((int32_t)lane < a.slices ? (int32_t)lane : 0)];
    return (int32_t)lane < a.slices ? p : none;
  };
  RowPart v[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) v[j] = part_of((int32_t)w + j * kOpWaves);
  static_assert(kMaxDrafts <= kOpThreads, "a thread a draft");
  const bool drafts = (int32_t)tid < K;
  const int32_t my_draft = drafts ? a.draft_tokens[n * K + tid] : -1;
  const float my_u = drafts ? a.uniforms[n * K + tid] : -1.0f;
  const uint64_t seed = a.seeds[n], first_position = a.positions[n];
  if (count < 0 || count > K || !(greedy || temperature_ok(T)) || !temperature_ok(Td)) {
    refuse(TSC_ROW_INVALID_PARAM);
    return;
  }
  const bool valid = (int32_t)tid < count && my_draft >= 0 && my_draft < a.V &&
                     (greedy || (my_u >= 0.0f && my_u < 1.0f));  // greedy requests use no uniforms
  const float my_x = valid && !greedy ? Row<TD>::get(trow + (int64_t)tid * a.t_sk + my_draft) : 0.0f;
  const float my_y = valid && has_draft ? Row<DD>::get(drow + (int64_t)tid * a.d_sk + my_draft) : 0.0f;
  if (tid == 0) sh_stop = count, sh_bound = 0u;
  const Scale ct = make_scale(greedy ? 1.0f : T), cd = make_scale(Td);

  // Every row's state from its slices': a wave a row, a lane a slice.
  for (int32_t r0 = (int32_t)w; r0 < a.rows; r0 += kRows * kOpWaves) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int32_t r = r0 + j * kOpWaves;
      const bool is_draft = r > K;
      const int32_t i = is_draft ? r - K - 1 : r;
      // wave-uniform
      if (r < a.rows && i <= count - (is_draft ? 1 : 0) && !(is_draft && !has_draft)) {
        RowPart p = merge_slices(v[j], is_draft ? cd : ct);
        if (greedy && p.s == p.s) p.s = 1.0;
        if (lane == 0) (is_draft ? dp[i] : tp[i]) = p;
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) v[j] = part_of(r0 + (kRows + j) * kOpWaves);
  }
  lds_barrier();
  for (int32_t i = (int32_t)tid; i <= count; i += kOpThreads) {  // the second time round past the drafts
    const RowPart t = tp[i];
    int32_t st = part_status(t), c = kBonus;
    if (i < count) {
      if (has_draft && st == TSC_ROW_OK) st = part_status(dp[i]);
      if (!valid) st = TSC_ROW_INVALID_PARAM;
      if (st == TSC_ROW_OK) {
        if (greedy) {
          c = my_draft == t.at ? kAccepted : kRejected;
          xt[i] = t.m;
        } else {
          xt[i] = my_x;
          const double p = exp(((double)my_x - (double)t.m) / (double)T) / t.s;
          double q = 1.0;
          if (has_draft) q = exp(((double)my_y - (double)dp[i].m) / (double)Td) / dp[i].s;
          c = (double)my_u * q < p ? kAccepted : kRejected;
        }
      }
    }
    code[i] = st == TSC_ROW_OK ? c : kStatus + st;
    if (code[i] != kAccepted) atomicMin(&sh_stop, i);
  }
  lds_barrier();
  const Decision dec{sh_stop, code[sh_stop]};
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
  const TB* tr = trow + (int64_t)stop * a.t_sk;
  const DB* dr = drow + (int64_t)stop * a.d_sk;
  const uint64_t position = first_position + (uint64_t)stop;
  const int64_t lo = share * a.share_len, hi = lo + a.share_len < a.V ? lo + a.share_len : a.V;
  auto exact = [&](float xe, float ye) -> double {
    double p = exp(((double)xe - (double)t.m) / (double)T) / t.s;
    if (subtract) p -= exp(((double)ye - (double)d.m) / (double)Td) / d.s;
    return p;
  };
  const float c_t = plain_scale(T), c_d = plain_scale(Td);
  const float lg_t = -__builtin_amdgcn_logf((float)t.s), lg_d = -__builtin_amdgcn_logf((float)d.s);
  RaceEntry best;
  float bound = 0.0f;  // the workgroup's best score so far, as far as this wave knows, less the margin
  const uint32_t stream = rejected ? 1u : 0u;
  constexpr int64_t kStep = (int64_t)kOpThreads * 8;
  const int64_t first = lo + (int64_t)tid * 8;
  auto race_chunk = [&](int64_t at, const float (&x)[8], const float (&y)[8]) {
    float p[8], w8[8], most = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = weight_of(x[e], t.m, c_t, lg_t);
      w8[e] = p[e];
      if (subtract) w8[e] -= weight_of(y[e], d.m, c_d, lg_d);
      if (!subtract && at + e == drafted) p[e] = w8[e] = 0.0f;
      most = __builtin_fmaxf(most, p[e]);
    }
    // t is at least 2^-24: below that share of the bound no word wins, and none is drawn.
    if (__ballot(most > bound * 0x1p-24f) == 0) return;
    uint32_t word[2][4] = {{(uint32_t)at >> 2}, {((uint32_t)at >> 2) + 1u}};
    race_words(stream, seed, position, word);
    float tt[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) tt[e] = race_t(word[e >> 2][e & 3]);
    bound = __builtin_fmaxf(bound, __uint_as_float(__hip_atomic_load(&sh_bound, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP)));
    if (bound == 0.0f) {  // the first chunk makes its own
      float sc = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!RaceEntry::race_near(p[e], w8[e]))
          sc = __builtin_fmaxf(sc, w8[e] * __builtin_amdgcn_rcpf(race_exponential(tt[e])));
      bound = wave_max(sc) * (1.0f - kRaceClose);
    }
    // Few lanes have an entry that can still win; those are computed again, one by one.
    uint32_t open = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) open |= RaceEntry::can_win(p[e], w8[e], tt[e], bound) ? 1u << e : 0u;
    if (__ballot(open != 0u) == 0) return;
    while (open != 0u) {
      const int64_t id = at + __builtin_ctz(open);
      open &= open - 1u;
      const float xe = Row<TD>::get(tr + id), ye = subtract ? Row<DD>::get(dr + id) : 0.0f;
      best.offer(weight_of(xe, t.m, c_t, lg_t), subtract ? weight_of(ye, d.m, c_d, lg_d) : 0.0f,
                 (int32_t)id, race_t(race_word((uint32_t)id, stream, seed, position)), xe, ye, exact);
    }
    const float top = wave_max(best.score) * (1.0f - kRaceClose);
    if (top > bound || bound == 0.0f) {
      bound = __builtin_fmaxf(bound, top);
      if (lane == 0) atomicMax(&sh_bound, __float_as_uint(bound));
    }
  };
  // Whole chunks are asked for kAhead steps before their turn, since there are few waves to a CU
  // (bfloat16 27 us for 1, 2 or 3 steps; float32, 64 requests over 151936, 25.8, 24.6 and 28.3: three
  // steps of both rows no longer fit the registers).
  constexpr int kAhead = 2;
  typename Row<TD>::Chunk vx[kAhead];
  typename Row<DD>::Chunk vy[kAhead] = {};
  const int64_t most_at = hi >= lo + 8 ? hi - 8 : -1;  // the last place of a whole chunk
  auto ask = [&](int j, int64_t at) {
    if (most_at < 0) return;
    at = at < most_at ? at : most_at;
    vx[j] = Row<TD>::load(tr + at);
    if (subtract) vy[j] = Row<DD>::load(dr + at);
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) ask(j, first + j * kStep);
#pragma unroll 1
  for (int64_t at = first; at - (int64_t)lane * 8 < hi; at += kStep) {
    float x[8], y[8] = {};
    if (at + 8 <= hi) {
      Row<TD>::unpack(vx[0], x);
      if (subtract) Row<DD>::unpack(vy[0], y);
    } else {
      load8<TD>(tr, at, hi, x);
      if (subtract) load8<DD>(dr, at, hi, y);
    }
#pragma unroll
    for (int j = 1; j < kAhead; ++j) vx[j - 1] = vx[j], vy[j - 1] = vy[j];
    ask(kAhead - 1, at + kAhead * kStep);
    race_chunk(at, x, y);
  }
  const RacePart won = race_winner<kOpWaves>(best, exact, sh_score, sh_best);
  // The shares meet in the workspace. Each one's first thread puts its winner there, waits for the
  // words' old values, and only then counts itself in, so that whoever counts last finds every
  // winner in, and lets a lane look at each.
  // (Releasing and acquiring the whole memory at device scope instead, for plain stores of the
  // winners, took as long as the race: every workgroup wrote back and invalidated its L2.)
  constexpr int32_t kWait = -2, kNone = -1;
  if (w == 0) {
    uint32_t count = 0;
    if (lane == 0) {
      const int64_t at = n * a.shares + share;
      const uint64_t before = __hip_atomic_exchange(&a.score[at], __builtin_bit_cast(uint64_t, won.score),
                                                    __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const uint32_t other = __hip_atomic_exchange(&a.winner[at], (uint32_t)won.id, __ATOMIC_RELAXED,
                                                   __HIP_MEMORY_SCOPE_AGENT);
      uint32_t one = 1u;  // needs both old values
      asm volatile("" : "+v"(one) : "v"((uint32_t)before), "v"((uint32_t)(before >> 32)), "v"(other));
      count = __hip_atomic_fetch_add(&a.arrived[n], one, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    int32_t token = kWait;
    if ((uint32_t)__builtin_amdgcn_readfirstlane(count) == (uint32_t)a.shares - 1u) {
      static_assert(kMaxSlices <= kWaveSize, "a lane a share");
      double score = 0.0;
      int32_t id = INT32_MAX;
      if ((int32_t)lane < a.shares) {
        const int64_t at = n * a.shares + lane;
        score = __builtin_bit_cast(double, __hip_atomic_load(&a.score[at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        id = (int32_t)__hip_atomic_load(&a.winner[at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      const double top = wave_reduce(score, MaxOp());
      id = wave_reduce(score == top ? id : INT32_MAX, MinOp());
      token = top > 0.0 ? id : kNone;
    }
    if (lane == 0) sh_token = token;
  }
  lds_barrier();
  const int32_t token = sh_token;
  if (token == kWait) return;
  // No token with p > q: the two distributions agree within rounding, and the draft is as good a
  // draw from p as any.
  finish(token != kNone ? token : drafted);
}

// ---- Over captured supports ---------------------------------------------------------------------
// A capture slot lists a position's support: its ids, their logprobs (normalised over the
// support) and their number. One workgroup per request: its waves look the drafts up in the
// lists, all positions at once; at the position where the request stops, the drafter's list goes
// into a hash table in LDS that the target's entries look themselves up in, and race. A few
// megabytes move; the time is that of the chain of lookup, decision, table and race: 9 us for
// supports of 64, 15 us for 256 requests of 4 drafts with supports of up to 2048, 16 us for 64 of 2
// with up to 8192.
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

constexpr int kCapThreads = 1024;
constexpr int kCapWaves = kCapThreads / kWaveSize;

// The slot's status: a capture that is not whole cannot be verified against. A number that is no row
// status is INVALID_PARAM: the codes of decisions are told from statuses by their range.
__device__ inline int32_t slot_status(const SupportArgs& s, int64_t slot) {
  const int32_t st = s.status ? (int32_t)s.status[slot] : TSC_ROW_OK;
  if (st != TSC_ROW_OK) return st > TSC_ROW_OK && st <= TSC_ROW_ABORTED ? st : TSC_ROW_INVALID_PARAM;
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
  // The drafts' logprobs in both lists (-inf where they are not in them): a list to a wave, or to
  // several where there are more waves than lists.
  const int32_t lists = (has_draft ? 2 : 1) * count;
  const int32_t parts = lists > 0 && lists < kCapWaves ? kCapWaves / lists : 1;
  for (int32_t k = w; k < lists * parts; k += kCapWaves) {
    const int32_t j = k % lists, part = k / lists;
    const bool is_draft = j >= count;
    const int32_t i = is_draft ? j - count : j;
    const SupportArgs& s = is_draft ? a.draft : a.target;
    const int64_t slot = n * s.sn + i * s.sk;
    const int32_t want = a.draft_tokens[n * K + i];
    if (slot_status(s, slot) != TSC_ROW_OK) continue;
    const int32_t len = s.lengths[slot];
    const int32_t* ids = s.ids + slot * s.W;
    constexpr int kU = 8;
    for (int32_t e0 = part * kWaveSize + (int32_t)lane; e0 - (int32_t)lane < len; e0 += parts * kWaveSize * kU) {
      int32_t id[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int32_t e = e0 + u * parts * kWaveSize;
        id[u] = e < len ? ids[e] : ~want;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (id[u] == want) (is_draft ? lp_d : lp_t)[i] = s.logprobs[slot * s.W + e0 + u * parts * kWaveSize];
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
  const uint64_t seed = a.seeds[n], position = a.positions[n] + (uint64_t)stop;
  // kU entries of a thread at a time: what their lists hold is asked for together.
  constexpr int kU = 4;
  int32_t id[kU];
  float lp[kU];
  auto load_entries = [&](int32_t e0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int32_t e = e0 + u * kCapThreads;
      id[u] = e < t_len ? t_ids[e] : -1;
      lp[u] = e < t_len ? t_lps[e] : -__builtin_inff();
    }
  };
  load_entries((int32_t)tid);
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
    int32_t mine[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      mine[u] = (int32_t)tid + u * kCapThreads < d_len ? d_ids[tid + u * kCapThreads] : -1;
    for (uint32_t i = tid; i < slots; i += kCapThreads) table[i] = 0u;
    lds_barrier();
    // A slot holds the entry's index + 1 (at most 16384) and 17 bits of the id's hash beside it, so
    // that an entry of another id rarely costs a read of its id.
    auto insert = [&](int32_t e, int32_t of) {
      const uint32_t h = id_hash(of);
      const uint32_t v = (h << 15) | (uint32_t)(e + 1);
      uint32_t at = (h >> 17) & mask;
      while (atomicCAS(&table[at], 0u, v) != 0u) at = (at + 1u) & mask;
    };
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if ((int32_t)tid + u * kCapThreads < d_len) insert((int32_t)tid + u * kCapThreads, mine[u]);
    for (int32_t e = (int32_t)tid + kU * kCapThreads; e < d_len; e += kCapThreads) insert(e, d_ids[e]);
    lds_barrier();
  }
  auto exact = [](float x, float y) -> double { return exp((double)x) - exp((double)y); };
  RaceEntry best;
  for (int32_t e0 = (int32_t)tid;; e0 += kU * kCapThreads) {
    float lq[kU];
    uint32_t word[kU][4];
    // The place an id's probe stops at: its entry, unless another id shares its 17 bits.
    uint32_t at[kU], found[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      lq[u] = -__builtin_inff();
      word[u][0] = (uint32_t)id[u] >> 2;
      found[u] = 0u;
      if (subtract && e0 + u * kCapThreads < t_len) {
        const uint32_t h = id_hash(id[u]);
        at[u] = (h >> 17) & mask;
        for (uint32_t v; (v = table[at[u]]) != 0u; at[u] = (at[u] + 1u) & mask) {
          if ((v >> 15) == (h & 0x1FFFFu)) {
            found[u] = v & 0x7FFFu;
            break;
          }
        }
      }
    }
    int32_t other[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      other[u] = found[u] != 0u ? d_ids[found[u] - 1u] : id[u];
      if (found[u] != 0u) lq[u] = d_lps[found[u] - 1u];
    }
    race_words(rejected ? 1u : 0u, seed, position, word);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (e0 + u * kCapThreads >= t_len) continue;
      if (other[u] != id[u]) {  // another id of the same 17 bits: on with the probe
        lq[u] = -__builtin_inff();
        const uint32_t h = id_hash(id[u]);
        for (uint32_t v; (v = table[at[u] = (at[u] + 1u) & mask]) != 0u;) {
          const uint32_t f = v & 0x7FFFu;
          if ((v >> 15) == (h & 0x1FFFFu) && d_ids[f - 1u] == id[u]) {
            lq[u] = d_lps[f - 1u];
            break;
          }
        }
      }
      if (!subtract && id[u] == drafted) continue;
      const float p = exp_fast(lp[u]), q = exp_fast(lq[u]);
      const float tt = race_t(word_of(word[u], (uint32_t)id[u]));
      if (RaceEntry::can_win(p, p - q, tt, best.score * (1.0f - kRaceClose)))
        best.offer(p, q, id[u], tt, lp[u], lq[u], exact);
    }
    if (e0 - (int32_t)tid + kU * kCapThreads >= t_len) break;
    load_entries(e0 + kU * kCapThreads);
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
