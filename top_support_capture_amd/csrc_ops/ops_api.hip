// Host side of the C ABI declared in include/tsc_verify.h and include/tsc_train.h: argument
// validation and kernel launches on the caller's stream. Nothing here allocates device memory or
// synchronizes; scratch memory is the caller's workspace.
#include <hip/hip_runtime.h>

#include <atomic>

#include "distill.h"
#include "replay_grad.h"
#include "tsc_train.h"
#include "tsc_verify.h"
#include "verify.h"

namespace {

constexpr int64_t kMaxRows = int64_t{1} << 21;  // one workgroup per row: 2^21 * 1024 threads fit a grid
constexpr int64_t kMaxVocab = INT32_MAX - 16;

bool dtype_ok(int32_t dtype) { return dtype == TSC_DTYPE_F32 || dtype == TSC_DTYPE_BF16; }

bool aligned(const void* p, int32_t dtype) {
  return reinterpret_cast<uintptr_t>(p) % (dtype == TSC_DTYPE_F32 ? 4 : 2) == 0;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Cut {
  int32_t n;
  int64_t len;  // a multiple of `unit`
};

// `rows` rows of V elements cut into slices: enough slices for `target` workgroups in all, at
// most kMaxSlices a row, none shorter than `unit` or, unless V asks for it, longer than `most`.
Cut cut_rows(int64_t rows, int64_t V, int64_t unit, int64_t most, int64_t target) {
  int64_t n = ceil_div(target, rows > 0 ? rows : 1);
  if (n < ceil_div(V, most)) n = ceil_div(V, most);
  if (n > ceil_div(V, unit)) n = ceil_div(V, unit);
  if (n > tsc::kMaxSlices) n = tsc::kMaxSlices;
  const int64_t len = ceil_div(ceil_div(V, n), unit) * unit;
  return {(int32_t)ceil_div(V, len), len};
}

// Statistics of rows: slices of 32768 elements, or shorter ones until there are 2048 workgroups.
Cut stats_cut(int64_t rows, int64_t V) { return cut_rows(rows, V, 2048, 32768, 2048); }
// The distillation's loss: rows enough for the chip, or short ones, are read by one workgroup each,
// which saves a launch and the merge (bf16, 1024 rows of 151936 65 us against 82 + 27 in slices, 200
// rows 20.0 against 17.1 + 8.6, 64 rows 17.4 against 9.0 + 7.8; 128 rows 17.5 against 19.0; float32,
// 128 rows of 151936 19.4 against 23.3, of 262144 37.7 against 33.5, 200 rows of those 49.7 against 49.3).
Cut loss_cut(int64_t N, int64_t V) {
  return N >= 128 || V <= 65536 ? Cut{1, V} : stats_cut(N, V);
}
// Gradients: segments of rows, as long as their windows allow unless there are few rows. The
// distillation's cost little more than their share of the row, and two workgroups share a CU: 512.
// The replay's each take the support's statistics again: 256 (256 rows of 151936 in one segment 23
// us, in two 28).
Cut grad_cut(int64_t N, int64_t V, int64_t target) {
  constexpr int64_t unit = tsc::Window<tsc::kGradThreads>::kSize;
  int64_t len = ceil_div(ceil_div(V, target > N ? target / N : 1), unit) * unit;
  if (len > tsc::kMaxSegment) len = tsc::kMaxSegment;
  return {(int32_t)ceil_div(V, len), len};
}
// Races: see verify_race_kernel.
Cut race_cut(int64_t N, int64_t V) { return cut_rows(N, V, 2048, 1 << 30, 512); }

unsigned grid_of(int64_t items) { return (unsigned)(items < kMaxRows ? items : kMaxRows); }

int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

int32_t launched() { return hipGetLastError() == hipSuccess ? TSC_OK : TSC_ERR_HIP; }

struct VerifyLayout {
  int64_t parts, score, winner, arrived, bytes;  // offsets, and the whole
  int32_t rows;
  Cut stats, race;
};

VerifyLayout verify_layout(int64_t N, int32_t K, int64_t V, bool has_draft) {
  VerifyLayout l;
  l.rows = K + 1 + (has_draft ? K : 0);
  l.stats = stats_cut(N * l.rows, V);
  l.race = race_cut(N, V);
  l.parts = 0;
  l.score = N * l.rows * l.stats.n * (int64_t)sizeof(tsc::RowPart);
  l.winner = l.score + N * l.race.n * 8;
  l.arrived = l.winner + N * l.race.n * 4;
  l.bytes = round16(l.arrived + N * 4);
  return l;
}

template <int TD, int DD>
void launch_verify(const tsc::VerifyArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((tsc::verify_stats_kernel<TD, DD>), dim3(grid_of(a.N * a.rows * a.slices)),
                     dim3(tsc::kOpThreads), 0, s, a);
  hipLaunchKernelGGL((tsc::verify_race_kernel<TD, DD>), dim3((unsigned)(a.N * a.shares)),
                     dim3(tsc::kOpThreads), 0, s, a);
}

// The dynamic LDS limit of a kernel is a per-device attribute, set once per device.
constexpr int kMaxDevices = 64;

// Lets `kernel` have up to `bytes` of dynamic LDS on the current device.
template <class Kernel>
hipError_t allow_lds(Kernel kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  if ((done.load(std::memory_order_acquire) >> dev) & 1u) return hipSuccess;
  err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (err == hipSuccess) done.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  return err;
}

uint32_t table_slots(int32_t W) {  // a power of two, at least twice the entries
  uint32_t n = 64;
  while (n < 2u * (uint32_t)W) n <<= 1;
  return n;
}

int64_t distill_bytes(int64_t N, int64_t V) {
  const Cut cut = loss_cut(N, V);
  return cut.n > 1 ? N * cut.n * (int64_t)sizeof(tsc::RowPart) : 0;
}

// Checks that the distillation's and the replay gradient's entry points share.
int32_t check_rows(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld, int32_t W) {
  if (!dtype_ok(dtype) || N < 0 || V < 1 || V > kMaxVocab || ld < V || W < 1)
    return TSC_ERR_INVALID_ARGUMENT;
  // One workgroup per row and segment.
  if (N > kMaxRows || W > TSC_MAX_PACKED_WIDTH || N * ceil_div(V, tsc::kMaxSegment) > kMaxRows)
    return TSC_ERR_UNSUPPORTED;
  if (N > 0 && (!logits || !aligned(logits, dtype))) return TSC_ERR_INVALID_ARGUMENT;
  return TSC_OK;
}

int32_t check_workspace(const void* workspace, size_t have, int64_t need) {
  if (have < (size_t)need) return TSC_ERR_WORKSPACE;
  if (need > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
    return TSC_ERR_INVALID_ARGUMENT;
  return TSC_OK;
}

void launch_distill_loss(const tsc::DistillArgs& a, int32_t dtype, hipStream_t s) {
  const dim3 grid(grid_of(a.N * a.slices)), part(tsc::kOpThreads);
  const dim3 rows((unsigned)a.N), block(tsc::kLossThreads);
  if (dtype == TSC_DTYPE_F32) {
    if (a.slices > 1) hipLaunchKernelGGL(tsc::distill_stats_kernel<TSC_DTYPE_F32>, grid, part, 0, s, a);
    hipLaunchKernelGGL(tsc::distill_loss_kernel<TSC_DTYPE_F32>, rows, block, 0, s, a);
  } else {
    if (a.slices > 1) hipLaunchKernelGGL(tsc::distill_stats_kernel<TSC_DTYPE_BF16>, grid, part, 0, s, a);
    hipLaunchKernelGGL(tsc::distill_loss_kernel<TSC_DTYPE_BF16>, rows, block, 0, s, a);
  }
}

// A kernel that writes gradients, with LDS for W entries and no less than `least` bytes of it.
template <int kThr, class Args>
hipError_t launch_grad(void (*kernel)(Args), const Args& a, int64_t groups, std::atomic<uint64_t>& allowed,
                       hipStream_t s, size_t least = 0, int64_t more = 0) {
  using Ent = tsc::Entries<kThr>;
  static_assert(Ent::bytes(TSC_MAX_PACKED_WIDTH) <= (size_t)Ent::kAll, "the widest rows fit");
  const hipError_t err = allow_lds(kernel, (size_t)Ent::kAll, allowed);
  if (err != hipSuccess) return err;
  const size_t need = Ent::bytes(a.W, more), bytes = need > least ? need : least;
  hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(kThr), bytes, s, a);
  return hipGetLastError();
}

hipError_t launch_distill_grad(const tsc::DistillArgs& a, int32_t dtype, hipStream_t s) {
  static std::atomic<uint64_t> f32{0}, bf16{0};
  return dtype == TSC_DTYPE_F32
             ? launch_grad<tsc::kGradThreads>(&tsc::distill_grad_kernel<TSC_DTYPE_F32>, a, a.N * a.segments, f32, s)
             : launch_grad<tsc::kGradThreads>(&tsc::distill_grad_kernel<TSC_DTYPE_BF16>, a, a.N * a.segments, bf16, s);
}

// One workgroup per row for loss and gradient together, when there are rows enough or they are
// short; one launch instead of two or three. (bf16, W = 2048, of which half is used: 256 rows of
// 151936 take 42 us against 48 and a launch, 1024 rows 160 against 170; 64 rows 35 against 30. 128
// rows 35 against 37 in slices and segments; float32, 128 rows of 151936 51 against 57, of 262144 86
// against 83, 200 rows of those 119 against 129.)
bool fused(int64_t N, int64_t V) { return V <= tsc::kMaxSegment && (N >= 128 || V <= 65536); }

// The fused kernel's second reading of a row comes from the last-level cache (256 MB), if the rows
// of all resident workgroups fit there. Two workgroups share a CU, 512 rows in all; past kCached
// bytes of rows one workgroup is kept to a CU, by asking for more than half of its LDS. (bf16,
// W = 4608, 512 rows: of 262144, 268 MB, 141 us alone against 157 in pairs; of 200000, 205 MB,
// 116 against 123; of 151936, 156 MB, 95 against 91; 1024 rows of 32000 88 against 67.)
constexpr int64_t kCached = 180 << 20;
constexpr size_t kAlone = 84 * 1024;

hipError_t launch_distill_fused(const tsc::DistillArgs& a, int32_t dtype, hipStream_t s) {
  static std::atomic<uint64_t> f32{0}, bf16{0};
  const int64_t rows = (a.N < 512 ? a.N : 512) * a.V * (dtype == TSC_DTYPE_F32 ? 4 : 2);
  const size_t least = rows > kCached ? kAlone : 0;
  return dtype == TSC_DTYPE_F32
             ? launch_grad<tsc::kGradThreads>(&tsc::distill_fused_kernel<TSC_DTYPE_F32>, a, a.N, f32, s, least)
             : launch_grad<tsc::kGradThreads>(&tsc::distill_fused_kernel<TSC_DTYPE_BF16>, a, a.N, bf16, s, least);
}

// Packed rows of so many entries that a bitmask in LDS and two passes over the row cost less than
// gathering them. Gathering costs a cache line per entry, the passes V / 64 lines or more each.
// (256 rows, gathered against streamed: bf16 of 151936, 36 us against 42 for 4096 entries, 61
// against 43 for 8192; of 32000, 15.3 against 14.6 for 2048; float32 of 100000, 57 against 56 for
// 4096.)
struct Dense {
  int32_t above, mask_bytes;
};
Dense dense_rows(int64_t V, int32_t W) {
  using Ent = tsc::Entries<tsc::kGradThreads>;
  const int64_t mask = ceil_div(V, 32) * 4, above = V / 28 > 2048 ? V / 28 : 2048;
  if (W <= above || V > tsc::kMaxSegment || Ent::bytes(W, mask) > (size_t)Ent::kAll) return {INT32_MAX, 0};
  return {(int32_t)above, (int32_t)mask};
}

template <int DT>
hipError_t launch_replay_grad(const tsc::ReplayGradArgs& a, bool streams, hipStream_t s) {
  static std::atomic<uint64_t> with{0}, without{0};
  const int64_t groups = a.N * a.segments;
  return streams ? launch_grad<tsc::kGradThreads>(&tsc::replay_grad_kernel<DT, true>, a, groups, with, s, (size_t)a.lds_bytes, a.mask_bytes)
                 : launch_grad<tsc::kGradThreads>(&tsc::replay_grad_kernel<DT, false>, a, groups, without, s);
}

// Workspace of loss and gradient in one call: slices' states, and the rows' statistics.
int64_t distill_grad_bytes(int64_t N, int64_t V) { return distill_bytes(N, V) + N * 16; }

}  // namespace

extern "C" {

size_t tsc_verify_drafts_workspace(int64_t N, int32_t K, int64_t V, int32_t has_draft) {
  if (N < 1 || N > kMaxRows || K < 0 || K > TSC_MAX_DRAFTS || V < 1 || V > kMaxVocab) return 0;
  return (size_t)verify_layout(N, K, V, has_draft != 0).bytes;
}

int32_t tsc_verify_drafts(const void* target_logits, int32_t target_dtype, int64_t target_stride_n,
                          int64_t target_stride_k, const void* draft_logits, int32_t draft_dtype,
                          int64_t draft_stride_n, int64_t draft_stride_k, int64_t N, int32_t K,
                          int64_t V, const float* temperature, const float* draft_temperature,
                          const int32_t* draft_tokens, const int32_t* draft_counts,
                          const float* uniforms, const uint64_t* seeds, const uint64_t* positions,
                          int32_t* tokens, int32_t* accepted, float* logprobs, int8_t* row_status,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(target_dtype) || (draft_logits && !dtype_ok(draft_dtype)))
    return TSC_ERR_INVALID_ARGUMENT;
  if (N < 0 || K < 0 || V < 1 || V > kMaxVocab) return TSC_ERR_INVALID_ARGUMENT;
  if (N > kMaxRows || K > TSC_MAX_DRAFTS) return TSC_ERR_UNSUPPORTED;
  if (N == 0) return TSC_OK;
  if (target_stride_n < 0 || (K > 0 && target_stride_k < 0) || draft_stride_n < 0 || draft_stride_k < 0)
    return TSC_ERR_INVALID_ARGUMENT;
  if (!target_logits || !aligned(target_logits, target_dtype) ||
      (draft_logits && !aligned(draft_logits, draft_dtype)))
    return TSC_ERR_INVALID_ARGUMENT;
  if (!temperature || !seeds || !positions || !tokens || !accepted || !logprobs || !row_status ||
      (K > 0 && (!draft_tokens || !uniforms)))
    return TSC_ERR_INVALID_ARGUMENT;
  const VerifyLayout l = verify_layout(N, K, V, draft_logits != nullptr);
  if (const int32_t e = check_workspace(workspace, workspace_bytes, l.bytes)) return e;
  char* ws = static_cast<char*>(workspace);
  const tsc::VerifyArgs a{target_logits, target_stride_n, target_stride_k,
                          K > 0 ? draft_logits : nullptr, draft_stride_n, draft_stride_k, N, V, K,
                          temperature, draft_temperature, draft_tokens, draft_counts, uniforms, seeds,
                          positions, tokens, accepted, logprobs, row_status,
                          reinterpret_cast<tsc::RowPart*>(ws + l.parts),
                          reinterpret_cast<uint64_t*>(ws + l.score),
                          reinterpret_cast<uint32_t*>(ws + l.winner),
                          reinterpret_cast<uint32_t*>(ws + l.arrived), l.rows, l.stats.n, l.race.n,
                          l.stats.len, l.race.len};
  (void)hipGetLastError();  // start from a clean error state so a launch error is ours
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int32_t dd = draft_logits ? draft_dtype : target_dtype;
  if (target_dtype == TSC_DTYPE_F32)
    dd == TSC_DTYPE_F32 ? launch_verify<TSC_DTYPE_F32, TSC_DTYPE_F32>(a, s)
                        : launch_verify<TSC_DTYPE_F32, TSC_DTYPE_BF16>(a, s);
  else
    dd == TSC_DTYPE_F32 ? launch_verify<TSC_DTYPE_BF16, TSC_DTYPE_F32>(a, s)
                        : launch_verify<TSC_DTYPE_BF16, TSC_DTYPE_BF16>(a, s);
  return launched();
}

int32_t tsc_verify_captured(const int32_t* target_ids, const float* target_logprobs,
                            const int32_t* target_lengths, const int8_t* target_status,
                            int64_t target_stride_n, int64_t target_stride_k, int32_t W,
                            const int32_t* draft_ids, const float* draft_logprobs,
                            const int32_t* draft_lengths, const int8_t* draft_status,
                            int64_t draft_stride_n, int64_t draft_stride_k, int32_t draft_W,
                            int64_t N, int32_t K, const int32_t* draft_tokens,
                            const int32_t* draft_counts, const float* uniforms,
                            const uint64_t* seeds, const uint64_t* positions, int32_t* tokens,
                            int32_t* accepted, float* logprobs, int8_t* row_status, void* stream) {
  if (N < 0 || K < 0 || W < 1 || (draft_ids && draft_W < 1)) return TSC_ERR_INVALID_ARGUMENT;
  if (N > kMaxRows || K > TSC_MAX_DRAFTS || W > TSC_MAX_PACKED_WIDTH ||
      (draft_ids && draft_W > TSC_MAX_PACKED_WIDTH))
    return TSC_ERR_UNSUPPORTED;
  if (N == 0) return TSC_OK;
  if (target_stride_n < 0 || target_stride_k < 0 || draft_stride_n < 0 || draft_stride_k < 0)
    return TSC_ERR_INVALID_ARGUMENT;
  if (!target_ids || !target_logprobs || !target_lengths || !seeds || !positions || !tokens ||
      !accepted || !logprobs || !row_status || (K > 0 && (!draft_tokens || !uniforms)) ||
      (draft_ids && (!draft_logprobs || !draft_lengths)))
    return TSC_ERR_INVALID_ARGUMENT;
  const bool has_draft = draft_ids != nullptr && K > 0;
  const uint32_t slots = has_draft ? table_slots(draft_W) : 0u;
  const tsc::CapturedArgs a{
      {target_ids, target_logprobs, target_lengths, target_status, target_stride_n, target_stride_k, W},
      {has_draft ? draft_ids : nullptr, draft_logprobs, draft_lengths, draft_status, draft_stride_n,
       draft_stride_k, draft_W},
      N, K, draft_tokens, draft_counts, uniforms, seeds, positions, tokens, accepted, logprobs,
      row_status};
  (void)hipGetLastError();
  static std::atomic<uint64_t> allowed{0};
  if (allow_lds(&tsc::verify_captured_kernel, table_slots(TSC_MAX_PACKED_WIDTH) * 4, allowed) != hipSuccess)
    return TSC_ERR_HIP;
  hipLaunchKernelGGL(tsc::verify_captured_kernel, dim3((unsigned)N), dim3(tsc::kCapThreads), slots * 4,
                     reinterpret_cast<hipStream_t>(stream), a);
  return launched();
}

size_t tsc_distill_topk_workspace(int64_t N, int64_t V) {
  if (N < 1 || N > kMaxRows || V < 1 || V > kMaxVocab) return 0;
  return (size_t)distill_bytes(N, V);
}

int32_t tsc_distill_topk(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld,
                         const float* temperature, const int32_t* teacher_ids,
                         const float* teacher_values, const int32_t* lengths, int32_t W,
                         const float* teacher_temperature, float* loss, int8_t* row_status,
                         float* stats, void* workspace, size_t workspace_bytes, void* stream) {
  if (const int32_t e = check_rows(logits, dtype, N, V, ld, W)) return e;
  if (N == 0) return TSC_OK;
  if (!temperature || !teacher_ids || !teacher_values || !lengths || !loss || !row_status || !stats)
    return TSC_ERR_INVALID_ARGUMENT;
  if (const int32_t e = check_workspace(workspace, workspace_bytes, distill_bytes(N, V))) return e;
  const Cut cut = loss_cut(N, V);
  const tsc::DistillArgs a{logits, N, V, ld, temperature, teacher_ids, teacher_values, lengths, W,
                           teacher_temperature, loss, row_status, stats,
                           static_cast<tsc::RowPart*>(workspace), cut.n, cut.len, nullptr, nullptr, 0, 0};
  (void)hipGetLastError();
  launch_distill_loss(a, dtype, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

int32_t tsc_distill_topk_backward(const void* logits, int32_t dtype, int64_t N, int64_t V,
                                  int64_t ld, const float* temperature, const int32_t* teacher_ids,
                                  const float* teacher_values, const int32_t* lengths, int32_t W,
                                  const float* teacher_temperature, const float* stats,
                                  const float* grad_loss, void* grad_logits, void* stream) {
  if (const int32_t e = check_rows(logits, dtype, N, V, ld, W)) return e;
  if (N == 0) return TSC_OK;
  if (!temperature || !teacher_ids || !teacher_values || !lengths || !stats || !grad_loss ||
      !grad_logits || !aligned(grad_logits, dtype))
    return TSC_ERR_INVALID_ARGUMENT;
  const Cut cut = grad_cut(N, V, 512);
  const tsc::DistillArgs a{logits, N, V, ld, temperature, teacher_ids, teacher_values, lengths, W,
                           teacher_temperature, nullptr, nullptr, const_cast<float*>(stats), nullptr,
                           0, 0, grad_loss, grad_logits, cut.n, cut.len};
  (void)hipGetLastError();
  return launch_distill_grad(a, dtype, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? TSC_OK : TSC_ERR_HIP;
}

int32_t tsc_distill_topk_grad(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld,
                              const float* temperature, const int32_t* teacher_ids,
                              const float* teacher_values, const int32_t* lengths, int32_t W,
                              const float* teacher_temperature, const float* grad_loss, float* loss,
                              int8_t* row_status, void* grad_logits, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (const int32_t e = check_rows(logits, dtype, N, V, ld, W)) return e;
  if (N == 0) return TSC_OK;
  if (!temperature || !teacher_ids || !teacher_values || !lengths || !grad_loss || !loss ||
      !row_status || !grad_logits || !aligned(grad_logits, dtype))
    return TSC_ERR_INVALID_ARGUMENT;
  if (const int32_t e = check_workspace(workspace, workspace_bytes, distill_grad_bytes(N, V))) return e;
  const bool one = fused(N, V);
  const Cut cut = one ? Cut{1, V} : loss_cut(N, V), seg = grad_cut(N, V, 512);
  char* stats = static_cast<char*>(workspace) + distill_bytes(N, V);
  const tsc::DistillArgs a{logits, N, V, ld, temperature, teacher_ids, teacher_values, lengths, W,
                           teacher_temperature, loss, row_status, reinterpret_cast<float*>(stats),
                           static_cast<tsc::RowPart*>(workspace), cut.n, cut.len, grad_loss,
                           grad_logits, seg.n, seg.len};
  (void)hipGetLastError();
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (one) return launch_distill_fused(a, dtype, s) == hipSuccess ? TSC_OK : TSC_ERR_HIP;
  launch_distill_loss(a, dtype, s);
  if (const int32_t e = launched()) return e;
  return launch_distill_grad(a, dtype, s) == hipSuccess ? TSC_OK : TSC_ERR_HIP;
}

size_t tsc_distill_topk_grad_workspace(int64_t N, int64_t V) {
  if (N < 1 || N > kMaxRows || V < 1 || V > kMaxVocab) return 0;
  return (size_t)distill_grad_bytes(N, V);
}

int32_t tsc_replay_logprob_backward(const void* logits, int32_t dtype, int64_t N, int64_t V,
                                    int64_t ld, const float* temperature, const int32_t* packed_ids,
                                    const int32_t* lengths, int32_t W, const int8_t* capture_status,
                                    const uint8_t* support_bits, int64_t bits_ld,
                                    const int32_t* tokens, const float* grad_selected,
                                    const float* grad_logprobs, void* grad_logits, void* stream) {
  if (const int32_t e = check_rows(logits, dtype, N, V, ld, W)) return e;
  if (N == 0) return TSC_OK;
  if (!temperature || !packed_ids || !lengths || !tokens || !grad_logits ||
      !aligned(grad_logits, dtype) || (support_bits && bits_ld < (V + 7) / 8))
    return TSC_ERR_INVALID_ARGUMENT;
  const Cut cut = grad_cut(N, V, 256);
  const Dense dense = dense_rows(V, W);
  using Ent = tsc::Entries<tsc::kGradThreads>;
  // A streamed row that its workgroup writes whole is kept in LDS as far as it goes, for the second
  // pass (bf16: 256 rows of 129280 37.1 -> 34.8 us, 512 of 151936 92 -> 85; short rows come from the
  // L2 as fast, and all of a CU's LDS costs each workgroup 0.7 us: 1024 rows of 32000 52 against 50).
  const bool hold = cut.n == 1 && V * (dtype == TSC_DTYPE_F32 ? 4 : 2) > 128 * 1024;
  const tsc::ReplayGradArgs a{logits, N, V, ld, temperature, packed_ids, lengths, W, capture_status,
                              support_bits, bits_ld, tokens, grad_selected, grad_logprobs,
                              grad_logits, cut.n, cut.len, dense.above, dense.mask_bytes,
                              (int32_t)(hold ? (size_t)Ent::kAll : Ent::bytes(W, dense.mask_bytes)), hold};
  (void)hipGetLastError();
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool streams = support_bits != nullptr || dense.mask_bytes > 0;
  const hipError_t err = dtype == TSC_DTYPE_F32 ? launch_replay_grad<TSC_DTYPE_F32>(a, streams, s)
                                                : launch_replay_grad<TSC_DTYPE_BF16>(a, streams, s);
  return err == hipSuccess ? TSC_OK : TSC_ERR_HIP;
}

}  // extern "C"
