/* Host-side checks of the entry points of tsc_logprob.h and tsc_clip.h, built with AddressSanitizer and
 * UndefinedBehaviorSanitizer against a host-instrumented build (tests/test_host_logprob_sanitizers.py).
 * Every call fails its argument checks or has nothing to do, so nothing is launched: the pointers
 * stand in for device buffers and are never dereferenced. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "tsc_clip.h"
#include "tsc_logprob.h"

static int failures = 0;

static void expect(int cond, const char* what) {
  if (!cond) {
    printf("FAILED: %s\n", what);
    ++failures;
  }
}

#define DPTR(T, n) ((T*)(uintptr_t)(0x10000u * (n)))

static int32_t values(int64_t N, int64_t V, int64_t ld, int32_t top, void* ws, size_t bytes) {
  return tsc_token_logprobs(DPTR(void, 1), TSC_DTYPE_BF16, N, V, ld, NULL, DPTR(int32_t, 2), top, DPTR(float, 3),
                            NULL, DPTR(int32_t, 4), DPTR(float, 5), DPTR(int8_t, 6), NULL, ws, bytes, NULL);
}

static int32_t backward(int64_t N, int64_t V, int32_t top, const int32_t* ids) {
  return tsc_token_logprobs_backward(DPTR(void, 1), TSC_DTYPE_F32, N, V, V, NULL, DPTR(int32_t, 2), DPTR(float, 3),
                                     top, ids, NULL, NULL, DPTR(float, 4), DPTR(void, 5), NULL);
}

static int32_t grad(int64_t N, int64_t V, void* ws, size_t bytes) {
  return tsc_token_logprobs_grad(DPTR(void, 1), TSC_DTYPE_F32, N, V, V, NULL, DPTR(int32_t, 2), DPTR(float, 3), NULL,
                                 DPTR(float, 4), NULL, DPTR(int8_t, 5), DPTR(void, 6), ws, bytes, NULL);
}

int main(void) {
  const int64_t big = INT64_MAX;
  expect(values(-1, 100, 100, 0, NULL, 0) == TSC_ERR_INVALID_ARGUMENT, "N < 0");
  expect(values(big, 100, 100, 0, NULL, 0) == TSC_ERR_UNSUPPORTED, "N too large");
  expect(values(2, big, big, 0, NULL, 0) == TSC_ERR_INVALID_ARGUMENT, "V too large");
  expect(values(2, 100, INT64_MIN, 0, NULL, 0) == TSC_ERR_INVALID_ARGUMENT, "ld");
  expect(values(2, 1000, 1000, INT32_MAX, NULL, 0) == TSC_ERR_INVALID_ARGUMENT, "top > V");
  expect(values(2, 1000, 1000, INT32_MIN, NULL, 0) == TSC_ERR_INVALID_ARGUMENT, "top < 0");
  expect(values(2, 1000, 1000, 129, NULL, 0) == TSC_ERR_UNSUPPORTED, "top too large");
  expect(values(1, INT32_MAX - 16, big, 128, NULL, 0) == TSC_ERR_WORKSPACE, "longest row, no workspace");
  expect(values(1 << 21, INT32_MAX - 16, big, 0, NULL, 0) == TSC_ERR_UNSUPPORTED, "more segments than a grid holds");
  expect(values(0, 100, 100, 5, NULL, 0) == TSC_OK, "no rows");
  expect(tsc_token_logprobs_workspace(127, INT32_MAX - 16, 128) > 0, "largest workspace");
  expect(tsc_token_logprobs_workspace(1, INT32_MAX, 0) == 0 && tsc_token_logprobs_workspace(1, 100, INT32_MAX) == 0,
         "workspaces of unsupported sizes");
  expect(backward(2, 100, 5, NULL) == TSC_ERR_INVALID_ARGUMENT, "no ids");
  expect(backward(2, 100, -1, NULL) == TSC_ERR_INVALID_ARGUMENT, "top < 0 backward");
  expect(backward(0, 100, 5, NULL) == TSC_OK, "no rows backward");
  expect(grad(2, INT32_MAX - 16, NULL, 0) == TSC_ERR_WORKSPACE, "gradient without its workspace");
  expect(grad(0, 100, NULL, 0) == TSC_OK, "gradient without rows");
  expect(tsc_token_logprobs_grad_workspace(127, INT32_MAX - 16) > 0, "largest gradient workspace");
  expect(tsc_token_logprobs_grad_workspace(INT64_MIN, 5) == 0, "gradient workspace of an unsupported size");

  /* A long list, in no order: its overlap is found. */
  enum { kCount = 5000 };
  const void** tensors = malloc(kCount * sizeof(void*));
  void** out = malloc(kCount * sizeof(void*));
  int64_t* numels = malloc(kCount * sizeof(int64_t));
  int32_t* dtypes = malloc(kCount * sizeof(int32_t));
  for (int i = 0; i < kCount; ++i) {
    const uintptr_t at = 0x100000u + 0x1000u * (uintptr_t)((i * 7919) % kCount);
    tensors[i] = (const void*)at;
    out[i] = (void*)(at + 0x10000000u);
    numels[i] = i % 5 == 0 ? 0 : 1024;
    dtypes[i] = i % 2 ? TSC_DTYPE_F32 : TSC_DTYPE_BF16;
  }
  char* ws = DPTR(char, 9);
  const size_t need = tsc_grad_norm_workspace(kCount);
  out[77] = (void*)((uintptr_t)out[78] + 4);
  expect(tsc_clip_grad_norm(tensors, numels, dtypes, kCount, out, dtypes, 1.0f, DPTR(float, 8), ws, need, NULL) ==
             TSC_ERR_INVALID_ARGUMENT, "results on each other");
  out[77] = (void*)((uintptr_t)tensors[78] + 4);
  expect(tsc_clip_grads(tensors, numels, dtypes, kCount, out, dtypes, 1.0f, DPTR(float, 8), NULL) ==
             TSC_ERR_INVALID_ARGUMENT, "a result on another's gradient");
  out[77] = (void*)(uintptr_t)0xFFFFFFFFFFFFF000u;
  expect(tsc_clip_grads(tensors, numels, dtypes, kCount, out, dtypes, 1.0f, DPTR(float, 8), NULL) ==
             TSC_ERR_INVALID_ARGUMENT, "an address of no memory");
  tensors[11] = tensors[12];
  expect(tsc_clip_grad_norm(tensors, numels, dtypes, kCount, NULL, NULL, 1.0f, DPTR(float, 8), ws, need, NULL) ==
             TSC_ERR_INVALID_ARGUMENT, "a gradient twice in place");
  expect(tsc_grad_norm(tensors, numels, dtypes, kCount, DPTR(float, 8), ws, need - 1, NULL) == TSC_ERR_WORKSPACE,
         "workspace too small");
  expect(tsc_grad_norm(tensors, numels, dtypes, kCount, DPTR(float, 8), ws + 8, need, NULL) == TSC_ERR_INVALID_ARGUMENT,
         "misaligned workspace");
  expect(tsc_grad_norm(tensors, numels, dtypes, big, DPTR(float, 8), ws, need, NULL) == TSC_ERR_UNSUPPORTED, "count");
  numels[3] = big;
  expect(tsc_grad_norm(tensors, numels, dtypes, kCount, DPTR(float, 8), ws, need, NULL) == TSC_ERR_UNSUPPORTED, "numel");
  numels[3] = INT64_MIN;
  expect(tsc_grad_norm(tensors, numels, dtypes, kCount, DPTR(float, 8), ws, need, NULL) == TSC_ERR_INVALID_ARGUMENT,
         "numel < 0");
  expect(tsc_clip_grads(NULL, NULL, NULL, 0, NULL, NULL, 1.0f, DPTR(float, 8), NULL) == TSC_OK, "an empty list");
  expect(tsc_grad_norm_workspace(INT64_MAX) == 0 && tsc_grad_norm_workspace(1 << 20) > 0, "list workspaces");
  free(tensors), free(out), free(numels), free(dtypes);
  printf("host logprob checks: %d failure(s)\n", failures);
  return failures;
}
