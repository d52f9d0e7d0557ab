// Host side of the C ABI declared in include/tsc_clip.h: argument validation and kernel launches on
// the caller's stream. Nothing here allocates device memory or synchronizes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include "clip.h"
#include "host_common.h"
#include "tsc_clip.h"

namespace {

constexpr int64_t kMaxTensors = int64_t{1} << 20;
constexpr int64_t kMaxElements = int64_t{1} << 40;
constexpr int64_t kJoinInline = int64_t{1} << 20;  // reads of partial sums

int64_t size_of(int32_t dtype) { return dtype == TSC_DTYPE_F32 ? 4 : 2; }

int32_t check_list(const void* const* tensors, const int64_t* numels, const int32_t* dtypes, int64_t count) {
  if (count < 0 || (count > 0 && (!tensors || !numels || !dtypes))) return TSC_ERR_INVALID_ARGUMENT;
  if (count > kMaxTensors) return TSC_ERR_UNSUPPORTED;
  int64_t all = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (!dtype_ok(dtypes[i]) || numels[i] < 0) return TSC_ERR_INVALID_ARGUMENT;
    if (numels[i] >= kMaxElements || (all += numels[i]) >= kMaxElements) return TSC_ERR_UNSUPPORTED;
    if (numels[i] > 0 && (!tensors[i] || !aligned(tensors[i], dtypes[i]))) return TSC_ERR_INVALID_ARGUMENT;
    if (numels[i] > 0 && reinterpret_cast<uintptr_t>(tensors[i]) >> 48 != 0) return TSC_ERR_INVALID_ARGUMENT;
  }
  return TSC_OK;
}

struct Lists {
  const void* const* src;
  const int64_t* numels;
  const int32_t* dtypes;
  int64_t count;
  void* const* dst;  // null: in place
  const int32_t* dst_dtypes;
  uintptr_t begin(int64_t i) const { return reinterpret_cast<uintptr_t>(src[i]); }
  uintptr_t end(int64_t i) const { return begin(i) + (uintptr_t)(numels[i] * size_of(dtypes[i])); }
  uintptr_t out_begin(int64_t i) const { return dst ? reinterpret_cast<uintptr_t>(dst[i]) : begin(i); }
  int32_t out_dtype(int64_t i) const { return dst ? dst_dtypes[i] : dtypes[i]; }
  uintptr_t out_end(int64_t i) const { return out_begin(i) + (uintptr_t)(numels[i] * size_of(out_dtype(i))); }
  bool own(int64_t i) const { return out_begin(i) == begin(i) && out_dtype(i) == dtypes[i]; }
};

// Results that no other result and no gradient but their own overlaps, and a norm that lies in none of
// either: workgroups read it, or write it, while others write results.
int32_t check_out(const Lists& l, const float* norm) {
  if ((l.dst == nullptr) != (l.dst_dtypes == nullptr)) return TSC_ERR_INVALID_ARGUMENT;
  if (l.dst) {
    if (const int32_t e = check_list(const_cast<const void* const*>(l.dst), l.numels, l.dst_dtypes, l.count)) return e;
  }
  const uintptr_t nb = reinterpret_cast<uintptr_t>(norm), ne = nb + sizeof(float);
  std::vector<std::pair<uintptr_t, uintptr_t>> written;
  written.reserve((size_t)l.count);
  bool sorted = true;
  for (int64_t i = 0; i < l.count; ++i) {
    if (l.numels[i] == 0) continue;
    if ((l.out_begin(i) < ne && nb < l.out_end(i)) || (l.begin(i) < ne && nb < l.end(i))) return TSC_ERR_INVALID_ARGUMENT;
    if (!written.empty() && l.out_begin(i) < written.back().first) sorted = false;
    written.emplace_back(l.out_begin(i), l.out_end(i));
  }
  if (!sorted) std::sort(written.begin(), written.end());
  for (size_t i = 1; i < written.size(); ++i)
    if (written[i].first < written[i - 1].second) return TSC_ERR_INVALID_ARGUMENT;
  if (!l.dst) return TSC_OK;
  for (int64_t i = 0; i < l.count; ++i) {
    if (l.numels[i] == 0 || l.own(i)) continue;
    // The first result that ends behind the gradient's begin.
    const auto at = std::upper_bound(written.begin(), written.end(), l.begin(i),
                                     [](uintptr_t b, const auto& w) { return b < w.second; });
    if (at != written.end() && at->first < l.end(i)) return TSC_ERR_INVALID_ARGUMENT;
  }
  return TSC_OK;
}

// Tensors from index `from` on into a table, as many as fit; returns the index behind them.
template <class Table>
int64_t fill(Table& t, const Lists& l, int64_t from) {
  t.begin();
  int64_t i = from;
  for (; i < l.count; ++i)
    if (l.numels[i] > 0 && !t.add(l.src[i], l.numels[i], l.dtypes[i] == TSC_DTYPE_F32,
                                  reinterpret_cast<void*>(l.out_begin(i)), l.out_dtype(i) == TSC_DTYPE_F32))
      break;
  if (t.n > 0) t.end();
  return i;
}

template <class Table>
int64_t groups(const Table& t, int64_t most) { return t.units < most ? t.units : most; }

// Launches the sums; returns how many partial sums they leave.
int64_t launch_norm(const Lists& l, double* partials, hipStream_t s) {
  int64_t n = 0;
  for (int64_t i = 0; i < l.count;) {
    tsc::NormTable t;
    i = fill(t, l, i);
    if (t.n == 0) break;
    const int64_t g = groups(t, tsc::kClipGroups);
    hipLaunchKernelGGL(tsc::clip_norm_kernel, dim3((unsigned)g), dim3(tsc::kClipThreads), 0, s, t, partials + n);
    n += g;
  }
  return n;
}

void launch_join(const double* partials, int64_t n, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(tsc::clip_join_kernel, dim3(1), dim3(tsc::kClipThreads), 0, s, partials, (int32_t)n, norm);
}

template <int kE, tsc::ClipOut kOut>
int64_t launch_copy(const Lists& l, int64_t from, const tsc::ClipNorm& c, hipStream_t s) {
  tsc::ScaleTable<kE, kOut> t;
  const int64_t to = fill(t, l, from);
  if (t.n > 0)
    hipLaunchKernelGGL((tsc::clip_scale_kernel<kE, kOut>), dim3((unsigned)groups(t, kMaxRows)), dim3(tsc::kClipThreads), 0,
                       s, t, c);
  return to;
}

int64_t launch_in_place(const Lists& l, int64_t from, const tsc::ClipNorm& c, hipStream_t s) {
  tsc::NormTable t;
  const int64_t to = fill(t, l, from);
  if (t.n > 0)
    hipLaunchKernelGGL(tsc::clip_in_place_kernel, dim3((unsigned)groups(t, tsc::kInPlaceGroups)), dim3(tsc::kClipThreads), 0,
                       s, t, c);
  return to;
}

void launch_scale(const Lists& l, tsc::ClipNorm c, hipStream_t s) {
  // Tensors of one type whose results lie as they do themselves, as in two flat buffers, need no
  // addresses for the results: more tensors to a launch (224 of 24 MB in all take one, 11.1 us, instead of
  // two, 13.2).
  bool own = true, narrow = true, flat = true;
  uint64_t distance = 0;
  int64_t first = -1;
  for (int64_t i = 0; i < l.count; ++i) {
    if (l.numels[i] == 0) continue;
    const bool f32 = l.dtypes[i] == TSC_DTYPE_F32, to_f32 = l.out_dtype(i) == TSC_DTYPE_F32;
    const uint64_t d = tsc::NormTable::distance(l.src[i], f32, reinterpret_cast<void*>(l.out_begin(i)), to_f32);
    if (first < 0) first = i, distance = d;
    own = own && l.own(i);
    narrow = narrow && !f32 && !to_f32;
    flat = flat && d == distance && l.dtypes[i] == l.dtypes[first] && l.out_dtype(i) == l.out_dtype(first);
  }
  constexpr auto kEach = tsc::ClipOut::kEach, kFlat = tsc::ClipOut::kFlat;
  for (int64_t i = 0; i < l.count;) {
    const int64_t from = i;
    if (own) i = launch_in_place(l, from, c, s);
    else if (narrow) i = flat ? launch_copy<8, kFlat>(l, from, c, s) : launch_copy<8, kEach>(l, from, c, s);
    else i = flat ? launch_copy<4, kFlat>(l, from, c, s) : launch_copy<4, kEach>(l, from, c, s);
    for (int64_t k = from; k < i; ++k)
      if (l.numels[k] > 0) c.norm_out = nullptr;  // written by the first launch
  }
}

// Whether every workgroup of the scaling may add up the partial sums by itself, which saves a
// launch: few of either, in the smallest units that a scaling takes.
bool joins_inline(const Lists& l, int64_t partials) {
  int64_t units = 0;
  for (int64_t i = 0; i < l.count; ++i) units += ceil_div(l.numels[i], 2048);
  return partials > 0 && partials * units <= kJoinInline;
}

int32_t check_norm(float* norm, int64_t count, const void* workspace, size_t have) {
  if (!norm) return TSC_ERR_INVALID_ARGUMENT;
  return check_workspace(workspace, have, (int64_t)tsc_grad_norm_workspace(count));
}

}  // namespace

extern "C" {

size_t tsc_grad_norm_workspace(int64_t count) {
  if (count < 1 || count > kMaxTensors) return 0;
  return (size_t)(ceil_div(count, tsc::NormTable::kSize) * tsc::kClipGroups) * sizeof(double);
}

int32_t tsc_grad_norm(const void* const* tensors, const int64_t* numels, const int32_t* dtypes, int64_t count,
                      float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (const int32_t e = check_list(tensors, numels, dtypes, count)) return e;
  if (const int32_t e = check_norm(norm, count, workspace, workspace_bytes)) return e;
  (void)hipGetLastError();  // start from a clean error state so a launch error is ours
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  double* partials = static_cast<double*>(workspace);
  const int64_t n = launch_norm({tensors, numels, dtypes, count, nullptr, nullptr}, partials, s);
  launch_join(partials, n, norm, s);
  return launched();
}

int32_t tsc_clip_grad_norm(const void* const* tensors, const int64_t* numels, const int32_t* dtypes, int64_t count,
                           void* const* out, const int32_t* out_dtypes, float max_norm, float* norm, void* workspace,
                           size_t workspace_bytes, void* stream) try {
  if (const int32_t e = check_list(tensors, numels, dtypes, count)) return e;
  if (!(max_norm >= 0.0f)) return TSC_ERR_INVALID_ARGUMENT;
  const Lists l{tensors, numels, dtypes, count, out, out_dtypes};
  if (const int32_t e = check_out(l, norm)) return e;
  if (const int32_t e = check_norm(norm, count, workspace, workspace_bytes)) return e;
  (void)hipGetLastError();
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  double* partials = static_cast<double*>(workspace);
  const int64_t n = launch_norm(l, partials, s);
  if (joins_inline(l, n)) {
    launch_scale(l, {partials, (int32_t)n, max_norm, norm, nullptr}, s);
  } else {
    launch_join(partials, n, norm, s);
    launch_scale(l, {nullptr, 0, max_norm, nullptr, norm}, s);
  }
  return launched();
} catch (const std::bad_alloc&) {
  return TSC_ERR_UNSUPPORTED;  // no host memory for a list of that length
}

int32_t tsc_clip_grads(const void* const* tensors, const int64_t* numels, const int32_t* dtypes, int64_t count,
                       void* const* out, const int32_t* out_dtypes, float max_norm, const float* norm,
                       void* stream) try {
  if (const int32_t e = check_list(tensors, numels, dtypes, count)) return e;
  if (!(max_norm >= 0.0f) || !norm) return TSC_ERR_INVALID_ARGUMENT;
  const Lists l{tensors, numels, dtypes, count, out, out_dtypes};
  if (const int32_t e = check_out(l, norm)) return e;
  if (count == 0) return TSC_OK;
  (void)hipGetLastError();
  launch_scale(l, {nullptr, 0, max_norm, nullptr, norm}, reinterpret_cast<hipStream_t>(stream));
  return launched();
} catch (const std::bad_alloc&) {
  return TSC_ERR_UNSUPPORTED;  // no host memory for a list of that length
}

}  // extern "C"
