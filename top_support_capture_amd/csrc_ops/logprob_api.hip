// Host side of the C ABI declared in include/tsc_logprob.h: argument validation and kernel launches
// on the caller's stream. Nothing here allocates device memory or synchronizes; scratch memory is
// the caller's workspace.
#include <hip/hip_runtime.h>

#include "host_common.h"
#include "logprob.h"
#include "tsc_logprob.h"

namespace {

static_assert(TSC_MAX_TOP == tsc::kTopMost, "the selection's lists hold that many");

// Whole rows for a workgroup each when there are rows enough, or short ones; slices otherwise, as
// many as the chip holds at once (two workgroups on each CU), of 8192 elements at least, in multiples of
// 4096 (a step of a workgroup for float32, half of one for bfloat16). Slices cost a second launch, and with
// alternatives a second selection. The borders count elements, not bytes: a row alone in a workgroup takes
// nearly as long in either type. Sliced against whole, us a call in a captured graph, without alternatives,
// then with 5 and the entropy:
//   bf16  65536   1 row   6.8 /  6.4, 13.0 / 11.7    64 rows 11.5 /  7.7, 20.1 / 12.6
//        100000  16 rows  8.1 / 10.6, 14.7 / 17.0    64 rows 11.8 / 11.8, 20.6 / 18.3   127 rows 13.2 / 12.4, 21.8 / 18.8
//        151936   1 row   6.8 / 11.9, 13.4 / 18.8    64 rows 12.1 / 14.4, 21.4 / 21.6   127 rows 16.7 / 15.7, 26.2 / 22.1
//        200000  16 rows 10.8 / 16.0, 20.0 / 24.2    64 rows 13.2 / 17.7, 22.0 / 26.2   127 rows 18.2 / 19.7, 26.9 / 26.8
//        262144  16 rows 11.2 / 19.1, 20.6 / 27.6    64 rows 13.0 / 20.0, 21.6 / 28.7   127 rows 18.9 / 21.9, 27.2 / 29.4
//   f32   65536   1 row   6.1 /  7.2, 11.9 / 12.5    64 rows 10.2 /  9.5, 18.6 / 14.6
//        100000  16 rows  7.7 / 10.9, 13.8 / 17.1    64 rows 11.2 / 13.3, 19.5 / 18.9   127 rows 16.6 / 15.3, 24.6 / 19.9
//        129280  16 rows  8.1 / 14.2, 14.2 / 20.5   100 rows 17.0 / 16.6, 24.9 / 21.9   127 rows 18.1 / 17.8, 25.5 / 22.1
//        151936  16 rows  9.6 / 16.3, 18.3 / 23.1    64 rows 14.9 / 17.3, 23.2 / 23.7   127 rows 20.4 / 20.1, 28.5 / 24.7
//        200000  16 rows 10.2 / 19.7, 19.2 / 27.3    64 rows 17.0 / 21.5, 25.0 / 28.4   127 rows 25.4 / 26.1, 33.6 / 29.5
//        262144  16 rows 10.0 / 23.0, 19.2 / 31.8    64 rows 18.2 / 25.5, 25.6 / 33.0   127 rows 29.6 / 31.9, 37.2 / 34.3
// With 160 rows whole ones are faster throughout (bf16 262144 24.0 / 21.8, 33.0 / 29.7). With alternatives
// the border of 160000 lies between 151936, where 64 rows are even, and 200000, where slices win by 4 us;
// more than 100 rows of those would gain up to 4 us whole, and 32 rows of 100000 2.5.
Cut pass_cut(int64_t N, int64_t V, int32_t top) {
  if (N >= 128 || V <= 65536 || (top > 0 && N >= 64 && V <= 160000)) return {1, V};
  const int64_t most = ceil_div(V, 8192) < tsc::kMaxSlices ? ceil_div(V, 8192) : tsc::kMaxSlices;
  const int64_t n = 512 / (N > 0 ? N : 1) < most ? 512 / (N > 0 ? N : 1) : most;
  const int64_t len = ceil_div(ceil_div(V, n), 4096) * 4096;
  return {(int32_t)ceil_div(V, len), len};
}

Cut segment_cut(int64_t N, int64_t V) {
  int64_t len = tsc::kLogprobGradSegment;
  while (len < tsc::kMaxSegment && N * ceil_div(V, len) > (int64_t{1} << 22)) len *= 2;
  return {(int32_t)ceil_div(V, len), len};
}

constexpr int64_t kCacheBytes = 256 << 20;  // the last-level cache

// With this many rows a smaller workgroup reads one, so that the ends of some overlap the loads of
// others. (With entropies, bf16: 4096 rows of 2000 take 18 us against 53, of 32000 57 against 69, 1024
// rows of 151936 59.5 against 59.9; but 256 rows of those 31 against 22. With 5 alternatives 512 threads:
// 4096 rows of 32000 74 us against 98, of 2000 45 against 83; with 20, of 151936 262 against 262 and, with
// 256 threads, 287.)
constexpr int64_t kManyRows = 1024;
constexpr int kSmall = 256, kSmallTop = 512;

int32_t check_rows(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld) {
  if (!dtype_ok(dtype) || N < 0 || V < 1 || V > kMaxVocab || ld < V) return TSC_ERR_INVALID_ARGUMENT;
  if (N > kMaxRows || N * ceil_div(V, tsc::kMaxSegment) > kMaxRows) return TSC_ERR_UNSUPPORTED;
  if (N > 0 && (!logits || !aligned(logits, dtype))) return TSC_ERR_INVALID_ARGUMENT;
  return TSC_OK;
}

int64_t parts_bytes(int64_t N, const Cut& cut) {
  return cut.n > 1 ? round16(N * cut.n * (int64_t)sizeof(tsc::LogprobPart)) : 0;
}

int64_t pass_bytes(int64_t N, int64_t V, int32_t top) {
  const Cut cut = pass_cut(N, V, top);
  return cut.n > 1 ? parts_bytes(N, cut) + round16(N * cut.n * top * 8) : 0;
}

// Slices' states and keys from `ws` on.
void set_parts(tsc::LogprobArgs& a, char* ws) {
  const Cut cut = pass_cut(a.N, a.V, a.top);
  a.slices = cut.n, a.slice_len = cut.len;
  a.parts = reinterpret_cast<tsc::LogprobPart*>(ws);
  a.keys = reinterpret_cast<uint64_t*>(ws + parts_bytes(a.N, cut));
}

// A kernel with the LDS of a selection by kThr threads, if it makes one.
template <int kThr, class Kernel>
hipError_t launch_top(Kernel kernel, const tsc::LogprobArgs& a, int64_t groups, bool top, std::atomic<uint64_t>& allowed,
                      hipStream_t s) {
  const size_t bytes = top ? tsc::TopLists<kThr>::kBytes : 0;
  if (top) {
    const hipError_t err = allow_lds(kernel, bytes, allowed);
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(kThr), bytes, s, a);
  return hipGetLastError();
}

// Values alone: logits past the last-level cache's size are read nontemporally (4096 rows of 151936
// bfloat16, with the first alternative, 201 us against 212). Not where the backward pass reads them
// again (83 us against 110 behind that).
bool read_once(const tsc::LogprobArgs& a, int64_t size) {
  return a.stats == nullptr && a.N * a.V * size > kCacheBytes;
}

template <int DT, int kThr, bool kEnt, bool kTop, bool kOnce>
hipError_t launch_rows(const tsc::LogprobArgs& a, hipStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  return launch_top<kThr>(&tsc::logprob_kernel<DT, kThr, kEnt, kTop, kOnce>, a, a.N, kTop, allowed, s);
}

template <int DT, bool kEnt, bool kTop>
hipError_t launch_pass(const tsc::LogprobArgs& a, hipStream_t s) {
  constexpr int kLarge = tsc::kTopThreads, kMany = kTop ? kSmallTop : kSmall;
  if (a.slices == 1) {
    const bool once = read_once(a, DT == TSC_DTYPE_F32 ? 4 : 2);
    if (a.N >= kManyRows)
      return once ? launch_rows<DT, kMany, kEnt, kTop, true>(a, s) : launch_rows<DT, kMany, kEnt, kTop, false>(a, s);
    return once ? launch_rows<DT, kLarge, kEnt, kTop, true>(a, s) : launch_rows<DT, kLarge, kEnt, kTop, false>(a, s);
  }
  static std::atomic<uint64_t> slice{0}, join{0};
  const hipError_t err =
      launch_top<kLarge>(&tsc::logprob_slice_kernel<DT, kEnt, kTop>, a, a.N * a.slices, kTop, slice, s);
  if (err != hipSuccess) return err;
  return launch_top<kTop ? kLarge : tsc::kWaveSize>(&tsc::logprob_join_kernel<DT, kEnt, kTop>, a, a.N, kTop, join, s);
}

hipError_t launch_pass(const tsc::LogprobArgs& a, int32_t dtype, bool entropy, hipStream_t s) {
  constexpr int F = TSC_DTYPE_F32, B = TSC_DTYPE_BF16;
  if (dtype == F) {
    if (entropy) return a.top ? launch_pass<F, true, true>(a, s) : launch_pass<F, true, false>(a, s);
    return a.top ? launch_pass<F, false, true>(a, s) : launch_pass<F, false, false>(a, s);
  }
  if (entropy) return a.top ? launch_pass<B, true, true>(a, s) : launch_pass<B, true, false>(a, s);
  return a.top ? launch_pass<B, false, true>(a, s) : launch_pass<B, false, false>(a, s);
}

template <int DT>
void launch_grad(const tsc::LogprobArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.N * a.segments)), block(tsc::kLogprobGradThreads);
  if (a.grad_top)
    hipLaunchKernelGGL((tsc::logprob_grad_kernel<DT, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((tsc::logprob_grad_kernel<DT, false>), grid, block, 0, s, a);
}

hipError_t launch_grad(tsc::LogprobArgs& a, int32_t dtype, hipStream_t s) {
  const Cut cut = segment_cut(a.N, a.V);
  a.segments = cut.n, a.seg_len = cut.len;
  dtype == TSC_DTYPE_F32 ? launch_grad<TSC_DTYPE_F32>(a, s) : launch_grad<TSC_DTYPE_BF16>(a, s);
  return hipGetLastError();
}

// One workgroup per row for values and gradient together, when there are rows enough or they are
// short; one launch instead of two or three.
bool fused(int64_t N, int64_t V) { return N >= 128 || V <= 65536; }

// Small workgroups where the rows of all of them that are resident (2048) stay in this part of the
// last-level cache for their second reading, beside the gradients on their way out. Small against large,
// us, with the entropy, by those rows' MB: bf16, 1024 rows, 94 MB 29 against 34, 125 MB 34 / 37, 156 MB
// 40 / 45, 172 MB 50 / 48, 352 MB 93 / 85; 4096 rows, 94 MB 89 / 108, 156 MB 146 / 164, 172 MB 166 / 171.
// float32 rows of as many bytes have half the elements, and the ends that small workgroups overlap weigh
// less: 1024 rows, 94 MB 22 / 28, 125 MB 30 / 33, 141 MB 38 / 35; 4096 rows, 94 MB 83 / 82, 109 MB 101 / 92,
// 156 MB 140 / 125.
template <int DT>
constexpr int64_t kCached = kCacheBytes * (DT == TSC_DTYPE_F32 ? 4 : 7) / 10;

// LDS that holds the first pieces of a workgroup's row for the second reading, as much as leaves room
// for two large workgroups, or eight small ones, on a CU.
template <int DT, int kThr, bool kEnt>
hipError_t launch_fused(tsc::LogprobArgs a, hipStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  constexpr size_t kHeld = (kThr == kSmall ? 16 : 64) << 10;
  const auto kernel = &tsc::logprob_fused_kernel<DT, kThr, kEnt>;
  const hipError_t err = allow_lds(kernel, kHeld, allowed);
  if (err != hipSuccess) return err;
  a.held = (int32_t)(kHeld / (kThr * 16));
  hipLaunchKernelGGL(kernel, dim3((unsigned)a.N), dim3(kThr), kHeld, s, a);
  return hipGetLastError();
}

template <int DT, bool kEnt>
hipError_t launch_fused(const tsc::LogprobArgs& a, hipStream_t s) {
  const int64_t rows = 2048 * a.V * (DT == TSC_DTYPE_F32 ? 4 : 2);  // of 8 workgroups on each CU
  return a.N >= kManyRows && rows <= kCached<DT> ? launch_fused<DT, kSmall, kEnt>(a, s)
                                                 : launch_fused<DT, tsc::kTopThreads, kEnt>(a, s);
}

hipError_t launch_fused(const tsc::LogprobArgs& a, int32_t dtype, bool entropy, hipStream_t s) {
  if (dtype == TSC_DTYPE_F32)
    return entropy ? launch_fused<TSC_DTYPE_F32, true>(a, s) : launch_fused<TSC_DTYPE_F32, false>(a, s);
  return entropy ? launch_fused<TSC_DTYPE_BF16, true>(a, s) : launch_fused<TSC_DTYPE_BF16, false>(a, s);
}

}  // namespace

extern "C" {

size_t tsc_token_logprobs_workspace(int64_t N, int64_t V, int32_t top) {
  if (N < 1 || N > kMaxRows || V < 1 || V > kMaxVocab || top < 0 || top > TSC_MAX_TOP) return 0;
  return (size_t)pass_bytes(N, V, top);
}

int32_t tsc_token_logprobs(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld,
                           const float* temperature, const int32_t* tokens, int32_t top, float* logprobs,
                           float* entropy, int32_t* top_ids, float* top_logprobs, int8_t* row_status, float* stats,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (const int32_t e = check_rows(logits, dtype, N, V, ld)) return e;
  if (top < 0 || top > V) return TSC_ERR_INVALID_ARGUMENT;
  if (top > TSC_MAX_TOP) return TSC_ERR_UNSUPPORTED;
  if (N == 0) return TSC_OK;
  if (!tokens || !logprobs || !row_status || (top > 0 && (!top_ids || !top_logprobs))) return TSC_ERR_INVALID_ARGUMENT;
  if (const int32_t e = check_workspace(workspace, workspace_bytes, pass_bytes(N, V, top))) return e;
  tsc::LogprobArgs a{};
  a.logits = logits, a.N = N, a.V = V, a.ld = ld, a.temperature = temperature, a.tokens = tokens, a.top = top;
  a.logprobs = logprobs, a.entropy = entropy, a.top_ids = top_ids, a.top_logprobs = top_logprobs;
  a.row_status = row_status, a.stats = stats;
  set_parts(a, static_cast<char*>(workspace));
  (void)hipGetLastError();  // start from a clean error state so a launch error is ours
  return launch_pass(a, dtype, entropy != nullptr, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? TSC_OK
                                                                                                       : TSC_ERR_HIP;
}

int32_t tsc_token_logprobs_backward(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld,
                                    const float* temperature, const int32_t* tokens, const float* stats, int32_t top,
                                    const int32_t* top_ids, const float* grad_logprobs, const float* grad_entropy,
                                    const float* grad_top, void* grad_logits, void* stream) {
  if (const int32_t e = check_rows(logits, dtype, N, V, ld)) return e;
  if (top < 0 || top > V) return TSC_ERR_INVALID_ARGUMENT;
  if (top > TSC_MAX_TOP) return TSC_ERR_UNSUPPORTED;
  if (N == 0) return TSC_OK;
  if (!tokens || !stats || !grad_logits || !aligned(grad_logits, dtype) || (top > 0 && grad_top && !top_ids))
    return TSC_ERR_INVALID_ARGUMENT;
  tsc::LogprobArgs a{};
  a.logits = logits, a.N = N, a.V = V, a.ld = ld, a.temperature = temperature, a.tokens = tokens, a.top = top;
  a.top_ids = const_cast<int32_t*>(top_ids), a.stats = const_cast<float*>(stats);
  a.grad_logprobs = grad_logprobs, a.grad_entropy = grad_entropy, a.grad_top = top > 0 ? grad_top : nullptr;
  a.grad = grad_logits;
  (void)hipGetLastError();
  return launch_grad(a, dtype, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? TSC_OK : TSC_ERR_HIP;
}

// Slices' states, a row's statistics, and room for entropies that the caller does not take.
size_t tsc_token_logprobs_grad_workspace(int64_t N, int64_t V) {
  if (N < 1 || N > kMaxRows || V < 1 || V > kMaxVocab || fused(N, V)) return 0;
  return (size_t)(pass_bytes(N, V, 0) + N * 16 + round16(N * 4));
}

int32_t tsc_token_logprobs_grad(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld,
                                const float* temperature, const int32_t* tokens, const float* grad_logprobs,
                                const float* grad_entropy, float* logprobs, float* entropy, int8_t* row_status,
                                void* grad_logits, void* workspace, size_t workspace_bytes, void* stream) {
  if (const int32_t e = check_rows(logits, dtype, N, V, ld)) return e;
  if (N == 0) return TSC_OK;
  if (!tokens || !grad_logprobs || !logprobs || !row_status || !grad_logits || !aligned(grad_logits, dtype))
    return TSC_ERR_INVALID_ARGUMENT;
  if (const int32_t e = check_workspace(workspace, workspace_bytes, (int64_t)tsc_token_logprobs_grad_workspace(N, V)))
    return e;
  tsc::LogprobArgs a{};
  a.logits = logits, a.N = N, a.V = V, a.ld = ld, a.temperature = temperature, a.tokens = tokens;
  a.logprobs = logprobs, a.entropy = entropy, a.row_status = row_status;
  a.grad_logprobs = grad_logprobs, a.grad_entropy = grad_entropy, a.grad = grad_logits;
  (void)hipGetLastError();
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool with_entropy = entropy || grad_entropy;
  if (fused(N, V)) return launch_fused(a, dtype, with_entropy, s) == hipSuccess ? TSC_OK : TSC_ERR_HIP;
  char* ws = static_cast<char*>(workspace);
  set_parts(a, ws);
  a.stats = reinterpret_cast<float*>(ws + pass_bytes(N, V, 0));
  if (grad_entropy && !entropy) a.entropy = a.stats + N * 4;
  if (launch_pass(a, dtype, with_entropy, s) != hipSuccess) return TSC_ERR_HIP;
  return launch_grad(a, dtype, s) == hipSuccess ? TSC_OK : TSC_ERR_HIP;
}

}  // extern "C"
