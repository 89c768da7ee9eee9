/* moe_shared_train.h and moe_lora.h used from plain C99: sizes and the
 * host-side validation of every entry point (each call below fails
 * validation, or has no token, before anything is enqueued, so no GPU is
 * needed).  Prints one line per failed check; exit status = number of
 * failures. */
#include <stdio.h>
#include <string.h>

#include "moe_lora.h"
#include "moe_shared_train.h"

static int failures = 0;
#define CHECK(cond)                                                  \
  do {                                                               \
    if (!(cond)) {                                                   \
      printf("FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);         \
      ++failures;                                                    \
    }                                                                \
  } while (0)

static moe_shape shape(int T, int H, moe_dtype dt) {
  moe_shape s;
  memset(&s, 0, sizeof s);
  s.T = T; s.H = H; s.E = 1; s.k = 1; s.Im = 32; s.micro_count = 1; s.dtype = dt; s.renormalize = 1;
  return s;
}

int main(void) {
  /* placeholder device pointers: never dereferenced, validation fails first */
  void* P = (void*)(size_t)4096;
  float* F = (float*)P;
  const uint64_t* rng = (const uint64_t*)P;
  const int32_t* ids = (const int32_t*)P;
  const size_t big = (size_t)1 << 40;
  const moe_shape s = shape(8, 128, MOE_BF16), none = shape(0, 128, MOE_BF16), f32 = shape(8, 128, MOE_F32);
  moe_lora_spec a;
  a.adapters = 4; a.rank = 16;

  CHECK(moe_shared_backward_workspace_size(&s, 64) == (size_t)8 * 128 * 2);
  CHECK(moe_shared_backward_workspace_size(&f32, 64) == (size_t)8 * 128 * 4);
  CHECK(moe_shared_backward_workspace_size(&s, 33) == 0);
  CHECK(moe_shared_backward_workspace_size(NULL, 64) == 0);

  CHECK(moe_dropout_add(&s, 1.0, rng, P, P, P, NULL) == MOE_ERR_INVALID_ARG);
  CHECK(moe_dropout_add(&s, 0.5, NULL, P, P, P, NULL) == MOE_ERR_INVALID_ARG);
  CHECK(moe_dropout_add(&none, 0.5, rng, NULL, NULL, NULL, NULL) == MOE_OK);
  CHECK(moe_dropout_backward(&s, 0.5, rng, NULL, P, NULL) == MOE_ERR_INVALID_ARG);
  CHECK(moe_shared_ffn_train(&s, 0, 0.0, NULL, P, P, P, NULL, F, P, P, NULL) == MOE_ERR_INVALID_ARG);
  CHECK(moe_shared_ffn_train(&s, 64, 0.0, NULL, P, P, P, NULL, NULL, P, P, NULL) == MOE_ERR_INVALID_ARG);
  CHECK(moe_shared_ffn_train(&none, 64, 0.0, NULL, P, P, P, NULL, F, P, P, NULL) == MOE_OK);
  CHECK(moe_shared_ffn_backward(&s, 64, 0.0, NULL, P, P, P, F, P, P, NULL, NULL, NULL, P, big, NULL) == MOE_ERR_INVALID_ARG);
  CHECK(moe_shared_ffn_backward(&s, 64, 0.0, NULL, P, P, P, F, P, P, P, P, P, P, 2047, NULL) == MOE_ERR_WORKSPACE);
  CHECK(moe_shared_ffn_backward(&none, 64, 0.0, NULL, P, P, P, F, P, P, P, NULL, NULL, NULL, 0, NULL) == MOE_OK);

  CHECK(moe_lora_workspace_size(&s, 64, &a) > 0);
  CHECK(moe_lora_workspace_size(&s, 64, NULL) == 0);
  CHECK(moe_lora_w13_swiglu(&s, 64, &a, P, P, P, P, F, NULL, P, P, big, NULL) == MOE_ERR_INVALID_ARG);
  CHECK(moe_lora_down(&s, 64, &a, P, P, P, P, F, ids, NULL, P, NULL, big, NULL) == MOE_ERR_WORKSPACE);
  CHECK(moe_shared_ffn_lora(&none, 64, &a, P, P, P, P, P, P, P, F, ids, P, P, P, NULL, 0, NULL) == MOE_OK);
  a.rank = MOE_LORA_MAX_RANK + 8;
  CHECK(moe_shared_ffn_lora(&s, 64, &a, P, P, P, P, P, P, P, F, ids, P, P, P, P, big, NULL) == MOE_ERR_UNSUPPORTED);
  a.rank = 8;
  a.adapters = MOE_LORA_MAX_ADAPTERS + 1;
  CHECK(moe_lora_workspace_size(&s, 64, &a) == 0);

  if (failures == 0) printf("abi_check ok\n");
  return failures;
}
