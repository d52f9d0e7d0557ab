/* Host-side checks of the entry points of tsc_verify.h and tsc_train.h, built with AddressSanitizer
 * and UndefinedBehaviorSanitizer against a host-instrumented build (tests/test_host_ops_sanitizers.py).
 * Every call fails its argument checks or has nothing to do, so nothing is launched: the pointers
 * stand in for device buffers and are never dereferenced. */
#include <stdint.h>
#include <stdio.h>

#include "tsc_train.h"
#include "tsc_verify.h"

static int failures = 0;

static void expect(int cond, const char* what) {
  if (!cond) {
    printf("FAILED: %s\n", what);
    ++failures;
  }
}

#define DPTR(T, n) ((T*)(uintptr_t)(0x10000u * (n)))

static int32_t verify(int64_t N, int32_t K, int64_t V, int64_t stride, void* ws, size_t bytes) {
  return tsc_verify_drafts(DPTR(void, 1), TSC_DTYPE_BF16, stride, stride, DPTR(void, 2), TSC_DTYPE_F32,
                           stride, stride, N, K, V, DPTR(float, 3), NULL, DPTR(int32_t, 4), NULL,
                           DPTR(float, 5), DPTR(uint64_t, 6), DPTR(uint64_t, 7), DPTR(int32_t, 8),
                           DPTR(int32_t, 9), DPTR(float, 10), DPTR(int8_t, 11), ws, bytes, NULL);
}

static int32_t captured(int64_t N, int32_t K, int32_t W, int64_t stride) {
  return tsc_verify_captured(DPTR(int32_t, 1), DPTR(float, 2), DPTR(int32_t, 3), NULL, stride, stride, W,
                             DPTR(int32_t, 1), DPTR(float, 2), DPTR(int32_t, 3), NULL, stride, stride, W,
                             N, K, DPTR(int32_t, 4), NULL, DPTR(float, 5), DPTR(uint64_t, 6),
                             DPTR(uint64_t, 7), DPTR(int32_t, 8), DPTR(int32_t, 9), DPTR(float, 10),
                             DPTR(int8_t, 11), NULL);
}

static int32_t distill(int64_t N, int64_t V, int64_t ld, int32_t W, void* ws, size_t bytes) {
  return tsc_distill_topk(DPTR(void, 1), TSC_DTYPE_BF16, N, V, ld, DPTR(float, 2), DPTR(int32_t, 3),
                          DPTR(float, 4), DPTR(int32_t, 5), W, NULL, DPTR(float, 6), DPTR(int8_t, 7),
                          DPTR(float, 8), ws, bytes, NULL);
}

int main(void) {
  const int64_t big = INT64_MAX;
  expect(verify(-1, 2, 100, 100, DPTR(void, 20), big) == TSC_ERR_INVALID_ARGUMENT, "N < 0");
  expect(verify(big, 2, 100, 100, DPTR(void, 20), big) == TSC_ERR_UNSUPPORTED, "N too large");
  expect(verify(2, INT32_MAX, 100, 100, DPTR(void, 20), big) == TSC_ERR_UNSUPPORTED, "K too large");
  expect(verify(2, 2, big, 100, DPTR(void, 20), big) == TSC_ERR_INVALID_ARGUMENT, "V too large");
  expect(verify(2, 2, 100, INT64_MIN, DPTR(void, 20), big) == TSC_ERR_INVALID_ARGUMENT, "stride < 0");
  expect(verify(1 << 21, 256, INT32_MAX - 16, big, NULL, 0) == TSC_ERR_WORKSPACE, "largest sizes, no workspace");
  expect(verify(2, 2, 100, 100, NULL, big) == TSC_ERR_INVALID_ARGUMENT, "null workspace");
  expect(verify(0, 0, 1, 0, NULL, 0) == TSC_OK, "no requests");
  expect(tsc_verify_drafts_workspace(1 << 21, 256, INT32_MAX - 16, 1) > 0, "largest workspace");
  expect(tsc_verify_drafts_workspace(big, 256, 100, 1) == 0, "workspace of an unsupported size");
  expect(tsc_verify_drafts_workspace(1, 0, 1, 1) > 0, "smallest workspace");

  expect(captured(big, 2, 16, 1) == TSC_ERR_UNSUPPORTED, "captured N too large");
  expect(captured(2, 2, INT32_MAX, 1) == TSC_ERR_UNSUPPORTED, "captured W too large");
  expect(captured(2, 2, INT32_MIN, 1) == TSC_ERR_INVALID_ARGUMENT, "captured W < 1");
  expect(captured(2, 2, 16, -1) == TSC_ERR_INVALID_ARGUMENT, "captured stride < 0");
  expect(captured(0, 2, 16, 1) == TSC_OK, "captured without requests");

  expect(distill(big, 100, 100, 16, DPTR(void, 20), big) == TSC_ERR_UNSUPPORTED, "distill N too large");
  expect(distill(2, big, big, 16, DPTR(void, 20), big) == TSC_ERR_INVALID_ARGUMENT, "distill V too large");
  expect(distill(2, 100, INT64_MIN, 16, DPTR(void, 20), big) == TSC_ERR_INVALID_ARGUMENT, "distill ld");
  expect(distill(5, INT32_MAX - 16, big, 16, NULL, 0) == TSC_ERR_WORKSPACE, "distill workspace");
  expect(distill(0, 100, 100, 16, NULL, 0) == TSC_OK, "distill without rows");
  expect(tsc_distill_topk_workspace(big, 100) == 0 && tsc_distill_topk_grad_workspace(-1, 100) == 0,
         "workspaces of unsupported sizes");
  expect(tsc_distill_topk_grad_workspace(100, INT32_MAX - 16) > 0, "largest gradient workspace");

  expect(tsc_distill_topk_backward(DPTR(void, 1), TSC_DTYPE_F32, 2, 100, 100, DPTR(float, 2), DPTR(int32_t, 3),
                                   DPTR(float, 4), DPTR(int32_t, 5), 16, NULL, NULL, DPTR(float, 6),
                                   DPTR(void, 7), NULL) == TSC_ERR_INVALID_ARGUMENT,
         "backward without stats");
  expect(tsc_distill_topk_grad(DPTR(void, 1), TSC_DTYPE_F32, 2, 100, 100, DPTR(float, 2), DPTR(int32_t, 3),
                               DPTR(float, 4), DPTR(int32_t, 5), 16, NULL, DPTR(float, 6), DPTR(float, 7),
                               DPTR(int8_t, 8), DPTR(char, 9) + 2, NULL, 0, NULL) == TSC_ERR_INVALID_ARGUMENT,
         "misaligned gradient");
  expect(tsc_replay_logprob_backward(DPTR(void, 1), TSC_DTYPE_F32, 2, 100, 100, DPTR(float, 2), DPTR(int32_t, 3),
                                     DPTR(int32_t, 4), 16, NULL, DPTR(uint8_t, 5), INT64_MIN, DPTR(int32_t, 6),
                                     NULL, NULL, DPTR(void, 7), NULL) == TSC_ERR_INVALID_ARGUMENT,
         "replay backward bits_ld");
  printf("host operator checks: %d failure(s)\n", failures);
  return failures;
}
