/* A plain C99 consumer of the training-step entry points of include/mr.h: argument checks that return before any
 * HIP call (so it runs on a machine without a GPU). */
#include <stdint.h>
#include <stdio.h>

#include "mr.h"

#define CHECK(cond)                                                     \
  do {                                                                  \
    if (!(cond)) {                                                      \
      fprintf(stderr, "check failed: %s (line %d)\n", #cond, __LINE__); \
      return 1;                                                         \
    }                                                                   \
  } while (0)

#define P(n) ((void*)(uintptr_t)(0x10000000u * (n)))

int main(void) {
  const void* bufs[3] = {P(1), P(2), P(3)};
  const void* params[200];
  const void* grads[200];
  uint64_t counts[200], elems = 0;
  mr_adamw_state st = {P(4), P(5), NULL, NULL, NULL};
  mr_adamw_hyper h = {1e-3, 0.9, 0.999, 1e-8, 0.01, 1, 0};
  int i;
  CHECK(mr_layer_norm_forward(bufs, 3, NULL, P(4), P(5), 8, 64, MR_BF16, MR_FP32, 1e-5, P(6), (char*)P(6) + 2, NULL, NULL, NULL) ==
        MR_ERR_ALIAS);
  CHECK(mr_layer_norm_forward(bufs, 3, NULL, P(4), P(5), 8, 64, MR_INT32, MR_INT32, 1e-5, NULL, P(6), NULL, NULL, NULL) ==
        MR_ERR_DTYPE);
  CHECK(mr_layer_norm_forward(NULL, 1, NULL, NULL, NULL, 0, 64, MR_BF16, MR_BF16, 1e-5, NULL, NULL, NULL, NULL, NULL) == MR_OK);
  CHECK(mr_layer_norm_backward(P(1), P(2), P(3), P(4), P(5), NULL, 8, 64, MR_FP16, MR_FP16, P(6), P(7), (char*)P(7) + 2, NULL) ==
        MR_ERR_ALIAS);
  for (i = 0; i < 200; ++i) {
    params[i] = (char*)P(1) + 4096 * i;
    grads[i] = (char*)P(2) + 4096 * (199 - i);
    counts[i] = (uint64_t)(i * 5);
  }
  CHECK(mr_adamw_state_elems(counts, 200, &elems) == MR_OK && elems % 32 == 0 && elems >= 99500);
  grads[7] = params[9]; /* found among 200 sorted outputs */
  CHECK(mr_adamw_step(params, grads, counts, 200, MR_FP32, MR_FP32, MR_STATE_FP32, &st, NULL, NULL, &h, NULL, NULL) == MR_ERR_ALIAS);
  h.step = 0;
  CHECK(mr_adamw_step(params, grads, counts, 200, MR_FP32, MR_FP32, MR_STATE_FP32, &st, NULL, NULL, &h, NULL, NULL) ==
        MR_ERR_INVALID_ARG);
  CHECK(mr_grad_norm(grads, counts, 200, MR_FP32, 1.0, 1.0, (float*)(char*)grads[100], NULL) == MR_ERR_ALIAS);
  CHECK(mr_grad_norm(grads, counts, 200, MR_FP32, 0.0, 1.0, (float*)P(9), NULL) == MR_ERR_INVALID_ARG);
  CHECK(mr_last_hip_error() == 0);
  printf("c abi ok\n");
  return 0;
}
