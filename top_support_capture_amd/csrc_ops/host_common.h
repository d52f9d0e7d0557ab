// What the host sides of the operators' entry points share: checks, cuts of rows, launch limits.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>

#include "row_stats.h"
#include "tsc.h"

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

unsigned grid_of(int64_t items) { return (unsigned)(items < kMaxRows ? items : kMaxRows); }

int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

int32_t launched() { return hipGetLastError() == hipSuccess ? TSC_OK : TSC_ERR_HIP; }

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

int32_t check_workspace(const void* workspace, size_t have, int64_t need) {
  if (have < (size_t)need) return TSC_ERR_WORKSPACE;
  if (need > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
    return TSC_ERR_INVALID_ARGUMENT;
  return TSC_OK;
}

}  // namespace
