// Distillation of a student's logits from a teacher's top logits. With S a row's teacher ids,
// p = softmax over S of the teacher's values and q the student's softmax over the vocabulary,
//     loss = sum_{i in S} p_i (ln p_i - ln q_i),   dloss/dx_j = (q_j - [j in S] p_j) / T.
//
// Every pass streams whole rows. The teacher's few entries are read behind the stream, where their
// lines are in the caches, and join the gradient in LDS.
#pragma once

#include "replay_grad.h"

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
  RowPart* parts;                    // workspace [N, slices], when slices > 1
  int32_t slices;                    // 1: distill_loss_kernel reads its row itself
  int64_t slice_len;
  const float* grad_loss;  // [N]
  void* grad;              // [N, V], contiguous
  int32_t segments;        // workgroups per row of the gradient
  int64_t seg_len;
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
                    plain_scale(a.temperature[n]), sh_m, sh_s, a.parts + item);
    lds_barrier();
  }
}

// What a row's gradient is computed from; A = 0 when the row has none.
struct DistillRow {
  float m, s, vm, A;
};

template <int kW>
struct DistillShared {
  float m[kW], v[kW];
  uint32_t f[kW];
  double s[kW], a[kW], d[kW];
};

// Whether row n is read at all; if not, its loss and status are written.
__device__ inline bool distill_row_read(const DistillArgs& a, int64_t n) {
  const int32_t len = a.lengths[n];
  const bool empty = len == 0;
  if (!empty && len > 0 && len <= a.W && temperature_ok(a.temperature[n]) &&
      (a.teacher_temperature == nullptr || temperature_ok(a.teacher_temperature[n])))
    return true;
  if (threadIdx.x == 0) {
    a.loss[n] = empty ? 0.0f : __builtin_nanf("");
    a.row_status[n] = (int8_t)(empty ? TSC_ROW_NO_SUPPORT : TSC_ROW_INVALID_PARAM);
  }
  return false;
}

// A thread's first kE teacher entries (entry u at tid + u kThr), in registers.
template <int DT, int kThr>
struct TeacherEntries {
  static constexpr int kE = 2;
  int32_t id[kE];
  float v[kE], x[kE] = {};
  __device__ inline void load(const DistillArgs& a, int64_t n, int32_t len, int32_t i0) {
#pragma unroll
    for (int u = 0; u < kE; ++u) {
      const int32_t i = i0 + u * kThr;
      id[u] = i < len ? a.ids[n * a.W + i] : 0;
      v[u] = i < len ? a.values[n * a.W + i] : -__builtin_inff();
    }
  }
  // The student's logits of the ids in [lo, hi).
  __device__ inline void gather(const DistillArgs& a, int64_t n, int64_t lo, int64_t hi) {
    const auto* row = (const typename Row<DT>::Bits*)a.logits + n * a.ld;
#pragma unroll
    for (int u = 0; u < kE; ++u)
      if (id[u] >= lo && id[u] < hi) x[u] = Row<DT>::get(row + id[u]);
  }
};

// The loss and the status of row n (which distill_row_read let through), from its first entries
// and a thread's state of the student's row or, with more than one slice to a row, the slices.
// The same result for every thread.
template <int DT, int kThr>
__device__ inline DistillRow distill_row(const DistillArgs& a, int64_t n,
                                         const TeacherEntries<DT, kThr>& first, LseState st,
                                         DistillShared<kThr / kWaveSize>& sh) {
  using Entries = TeacherEntries<DT, kThr>;
  constexpr int kE = Entries::kE, kW = kThr / kWaveSize;
  const int32_t tid = (int32_t)threadIdx.x, lane = tid & (kWaveSize - 1), w = tid / kWaveSize;
  const int32_t len = a.lengths[n];
  const float T = a.temperature[n], Tt = a.teacher_temperature ? a.teacher_temperature[n] : 1.0f;
  const float c = plain_scale(T), ct = plain_scale(Tt);
  const auto max_op = [](float p, float q) { return __builtin_fmaxf(p, q); };
  auto end = [&](int32_t status, float loss) {
    if (tid == 0) a.loss[n] = loss, a.row_status[n] = (int8_t)status;
    return DistillRow{0.0f, 0.0f, 0.0f, 0.0f};
  };
  float vm = -__builtin_inff();
  uint32_t flags = 0;  // 1: an id out of range, 2: a value NaN or +inf
  auto look = [&](const Entries& t) {
#pragma unroll
    for (int u = 0; u < kE; ++u) {
      flags |= (t.id[u] < 0 || t.id[u] >= a.V ? 1u : 0u) | (t.v[u] < __builtin_inff() ? 0u : 2u);
      vm = max_op(vm, t.v[u]);
    }
  };
  look(first);
  for (int32_t i0 = tid + kThr * kE; i0 - tid < len; i0 += kThr * kE) {
    Entries t;
    t.load(a, n, len, i0);
    look(t);
  }
  if (a.slices > 1) {  // every lane of every wave then holds the whole row's state
    const RowPart none{-__builtin_inff(), 0, 0.0};
    const RowPart p = merge_slices(lane < a.slices ? a.parts[n * a.slices + lane] : none, c);
    st.m = p.m, st.s = tid == 0 || p.s != p.s ? p.s : 0.0;
  }
  vm = wave_reduce(vm, max_op);
  flags = wave_reduce(flags, [](uint32_t p, uint32_t q) { return p | q; });
  const float wm = wave_reduce(st.m, max_op);
  if (lane == 0) sh.m[w] = wm, sh.v[w] = vm, sh.f[w] = flags;
  lds_barrier();
  float m = sh.m[0];
  vm = sh.v[0], flags = sh.f[0];
#pragma unroll
  for (int i = 1; i < kW; ++i) m = max_op(m, sh.m[i]), vm = max_op(vm, sh.v[i]), flags |= sh.f[i];
  if (flags & 1u) return end(TSC_ROW_INVALID_PARAM, __builtin_nanf(""));
  if (flags & 2u) return end(TSC_ROW_NONFINITE, __builtin_nanf(""));
  if (vm == -__builtin_inff()) return end(TSC_ROW_NO_SUPPORT, 0.0f);
  // With e_i the teacher's numerators and A their sum, the loss is
  //     sum_i e_i ((v_i - vm) / Tt - (x_i - m) / T) / A - ln A + ln s.
  double A = 0.0, D = 0.0;
  const double inv_T = 1.0 / (double)T, inv_Tt = 1.0 / (double)Tt;
  auto sum = [&](const Entries& t) {
#pragma unroll
    for (int u = 0; u < kE; ++u) {
      const float d = t.v[u] - vm, e = exp2_scaled(d, ct);
      if (e > 0.0f) {  // a teacher probability of 0 takes no part, whatever the student's logit
        A += (double)e;
        D += (double)e * ((double)d * inv_Tt - ((double)t.x[u] - (double)m) * inv_T);
      }
    }
  };
  sum(first);
  for (int32_t i0 = tid + kThr * kE; i0 - tid < len; i0 += kThr * kE) {
    Entries t;
    t.load(a, n, len, i0);
    t.gather(a, n, 0, a.V);
    sum(t);
  }
  const double s = wave_reduce(rescaled(st.s, st.m, m, c), SumOp());
  A = wave_reduce(A, SumOp()), D = wave_reduce(D, SumOp());
  if (lane == 0) sh.s[w] = s, sh.a[w] = A, sh.d[w] = D;
  lds_barrier();
  double S = sh.s[0];
  A = sh.a[0], D = sh.d[0];
#pragma unroll
  for (int i = 1; i < kW; ++i) S += sh.s[i], A += sh.a[i], D += sh.d[i];
  if (!(S < __builtin_inf()) || !(__builtin_fabsf(m) < __builtin_inff()))
    return end(TSC_ROW_NONFINITE, __builtin_nanf(""));
  if (tid == 0) {
    a.loss[n] = (float)(D / A - log(A) + log(S));
    a.row_status[n] = TSC_ROW_OK;
  }
  return {m, (float)S, vm, (float)A};
}

// The loss, a row per workgroup. With one slice to a row the workgroup reads the row itself: 1024
// rows of 151936 bfloat16 logits take 66 us, 4.9 TB/s with the teacher's entries, where a bare read
// reaches 6.1. (Slices for 256-thread workgroups and a second launch: 109 us.) 64 float32 rows of
// 32000: 8.5 us, one row's latency.
constexpr int kLossThreads = 1024;

template <int DT>
__global__ void __launch_bounds__(kLossThreads, 8) distill_loss_kernel(DistillArgs a) {
  __shared__ DistillShared<kLossThreads / kWaveSize> sh;
  const int64_t n = blockIdx.x;
  DistillRow r{0.0f, 0.0f, 0.0f, 0.0f};
  if (distill_row_read(a, n)) {
    TeacherEntries<DT, kLossThreads> t;
    t.load(a, n, a.lengths[n], (int32_t)threadIdx.x);
    LseState st;
    if (a.slices == 1) {
      st = thread_stats<DT, kLossThreads>((const typename Row<DT>::Bits*)a.logits + n * a.ld, 0, a.V,
                                          plain_scale(a.temperature[n]),
                                          [&](int64_t lo, int64_t hi) { t.gather(a, n, lo, hi); });
    } else {
      t.gather(a, n, 0, a.V);
    }
    r = distill_row<DT, kLossThreads>(a, n, t, st, sh);
  }
  if (threadIdx.x == 0) {
    float* stats = a.stats + n * 4;
    stats[0] = r.m, stats[1] = r.s, stats[2] = r.vm, stats[3] = r.A;
  }
}

// The teacher's entries in [lo, hi), counted and placed by window: the first of a thread from
// registers, the rest read again.
template <int DT, int kThr, class Visit>
__device__ inline void visit_entries(const DistillArgs& a, int64_t n, int32_t len,
                                     const TeacherEntries<DT, kThr>& t, int64_t lo, int64_t hi, Visit visit) {
  constexpr int kE = TeacherEntries<DT, kThr>::kE;
#pragma unroll
  for (int u = 0; u < kE; ++u)
    if ((int32_t)threadIdx.x + u * kThr < len && t.id[u] >= lo && t.id[u] < hi)
      visit((uint32_t)(t.id[u] - lo), t.v[u]);
  for (int32_t i = (int32_t)threadIdx.x + kThr * kE; i < len; i += kThr) {
    const int64_t id = a.ids[n * a.W + i];
    if (id >= lo && id < hi) visit((uint32_t)(id - lo), a.values[n * a.W + i]);
  }
}

// Chunk of the gradient: q_j g - p_j g, q_j = 2^((x_j - m) c) / s; the entries hold -p_j g.
__device__ inline void q_minus_p(float (&x)[8], const float (&p)[8], float m, float c, float g_s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = __builtin_fmaf(exp2_scaled(x[e] - m, c), g_s, p[e]);
}

// The gradient of row[lo, hi), window by window: logits are asked for kAhead windows before their
// turn.
template <int DT, int kThr>
struct GradStream {
  using B = typename Row<DT>::Bits;
  static constexpr int kSize = Window<kThr>::kSize;
  static constexpr int kAhead = DT == TSC_DTYPE_BF16 ? 4 : 2;
  const B* row;
  B* out;
  int64_t lo, hi;
  typename Row<DT>::Chunk v[kAhead];
  __device__ inline int64_t place(int k) const { return lo + (int64_t)k * kSize + (int64_t)threadIdx.x * 8; }
  // Whole chunks only: lanes past the last one ask for the first, and store nothing.
  __device__ inline void ask(int j, int k) {
    if (lo + 8 <= hi) v[j] = Row<DT>::load_once(row + (place(k) + 8 <= hi ? place(k) : lo));
  }
  __device__ inline void start() {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) ask(j, j);
  }
  // All windows, after start(); the entries of the first are in place.
  __device__ inline void run(const Entries<kThr>& ent, float m, float c, float g_s) {
    for (int k0 = 0; lo + (int64_t)k0 * kSize < hi; k0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int k = k0 + j;
        const int64_t at = place(k);
        if (lo + (int64_t)k * kSize < hi) {  // uniform
          ent.turn(k, [&](int next) { ent.add(next); }, [&] {
            if (at < hi) {
              float x[8], p[8];
              if (at + 8 <= hi)
                Row<DT>::unpack(v[j], x);
              else
                load8<DT>(row, at, hi, x);
              ent.at_window(k).take((int)threadIdx.x, p);
              q_minus_p(x, p, m, c, g_s);
              store8<DT>(out, at, hi, x);
            }
            ask(j, k + kAhead);
          });
        }
      }
    }
  }
};

// The gradient of a segment of a row per workgroup: a row is read once and written once, 104 us for
// 1024 rows of 151936 bfloat16 logits (6.0 TB/s behind the L2). Entries added to the finished row instead
// took 185 us.
template <int DT>
__global__ void __launch_bounds__(kGradThreads, 8) distill_grad_kernel(DistillArgs a) {
  using B = typename Row<DT>::Bits;
  extern __shared__ __attribute__((aligned(16))) float dyn_lds[];
  const Entries<kGradThreads> ent(dyn_lds, a.W);
  const int64_t n = blockIdx.x / a.segments;
  const int64_t lo = (blockIdx.x - n * a.segments) * a.seg_len;
  const int64_t hi = lo + a.seg_len < a.V ? lo + a.seg_len : a.V;
  const DistillRow r{a.stats[n * 4], a.stats[n * 4 + 1], a.stats[n * 4 + 2], a.stats[n * 4 + 3]};
  B* out = (B*)a.grad + n * a.V;
  if (r.A == 0.0f) {
    fill_zero<DT, kGradThreads>(out, lo, hi);
    return;
  }
  const B* row = (const B*)a.logits + n * a.ld;
  const float T = a.temperature[n], Tt = a.teacher_temperature ? a.teacher_temperature[n] : 1.0f;
  const int32_t len = a.lengths[n] < a.W ? a.lengths[n] : a.W;
  const float c = plain_scale(T), ct = plain_scale(Tt);
  const float g = a.grad_loss[n] / T, minus_g_A = -g / r.A;
  TeacherEntries<DT, kGradThreads> t;
  t.load(a, n, len, (int32_t)threadIdx.x);
  GradStream<DT, kGradThreads> stream{row, out, lo, hi};
  stream.start();
  ent.begin();
  lds_barrier();
  visit_entries<DT, kGradThreads>(a, n, len, t, lo, hi, [&](uint32_t at, float) { ent.count(at); });
  lds_barrier();
  ent.offsets();
  lds_barrier();
  visit_entries<DT, kGradThreads>(a, n, len, t, lo, hi, [&](uint32_t at, float value) {
    ent.place(at, exp2_scaled(value - r.vm, ct) * minus_g_A);
  });
  lds_barrier();
  ent.add(0);
  lds_barrier();
  stream.run(ent, r.m, c, g / r.s);
}

// Loss and gradient, a row per workgroup: the row is read twice, but the second time soon after
// the first, while the rows in flight fit the last-level cache. 512 rows of 262144 bfloat16 logits
// with 4608 entries each: 142 us, 5.5 TB/s behind the L2. (Holding part of a row in registers from
// the first pass to the second leaves one workgroup to a CU and took 176 us.)
template <int DT>
__global__ void __launch_bounds__(kGradThreads, 8) distill_fused_kernel(DistillArgs a) {
  extern __shared__ __attribute__((aligned(16))) float dyn_lds[];
  __shared__ DistillShared<kGradWaves> sh;
  const Entries<kGradThreads> ent(dyn_lds, a.W);
  using B = typename Row<DT>::Bits;
  const int64_t n = blockIdx.x;
  B* out = (B*)a.grad + n * a.V;
  if (!distill_row_read(a, n)) {
    fill_zero<DT, kGradThreads>(out, 0, a.V);
    return;
  }
  const B* row = (const B*)a.logits + n * a.ld;
  const float T = a.temperature[n], Tt = a.teacher_temperature ? a.teacher_temperature[n] : 1.0f;
  const int32_t len = a.lengths[n];
  const float c = plain_scale(T), ct = plain_scale(Tt);
  TeacherEntries<DT, kGradThreads> t;
  t.load(a, n, len, (int32_t)threadIdx.x);
  ent.begin();
  const LseState st = thread_stats<DT, kGradThreads>(row, 0, a.V, c,
                                                     [&](int64_t lo, int64_t hi) { t.gather(a, n, lo, hi); });
  const DistillRow r = distill_row<DT, kGradThreads>(a, n, t, st, sh);  // has barriers
  if (r.A == 0.0f) {
    fill_zero<DT, kGradThreads>(out, 0, a.V);
    return;
  }
  GradStream<DT, kGradThreads> stream{row, out, 0, a.V};
  stream.start();
  visit_entries<DT, kGradThreads>(a, n, len, t, 0, a.V, [&](uint32_t at, float) { ent.count(at); });
  lds_barrier();
  ent.offsets();
  lds_barrier();
  const float g = a.grad_loss[n] / T, minus_g_A = -g / r.A;
  visit_entries<DT, kGradThreads>(a, n, len, t, 0, a.V, [&](uint32_t at, float value) {
    ent.place(at, exp2_scaled(value - r.vm, ct) * minus_g_A);
  });
  lds_barrier();
  ent.add(0);
  lds_barrier();
  stream.run(ent, r.m, c, g / r.s);
}

}  // namespace tsc
