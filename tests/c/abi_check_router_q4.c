/* moe_q4.h and moe_router_grad.h used from plain C99: sizes and the host-side
 * validation of every entry point (each call below fails validation, or has
 * no token, before anything is enqueued, so no GPU is needed).  Prints one
 * line per failed check; exit status = number of failures. */
#include <stdio.h>
#include <string.h>

#include "moe_q4.h"
#include "moe_router_grad.h"

static int failures = 0;
#define CHECK(cond)                                                  \
  do {                                                               \
    if (!(cond)) {                                                   \
      printf("FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);         \
      ++failures;                                                    \
    }                                                                \
  } while (0)

static moe_shape shape(int T, int H, int E, int k, int Im, int mu, moe_dtype dt) {
  moe_shape s;
  memset(&s, 0, sizeof s);
  s.T = T; s.H = H; s.E = E; s.k = k; s.Im = Im; s.micro_count = mu; s.dtype = dt; s.renormalize = 1;
  return s;
}

static moe_q4_spec spec(int format, int group) {
  moe_q4_spec q;
  q.format = format; q.group = group;
  return q;
}

int main(void) {
  /* placeholder device pointers: never dereferenced, validation fails first */
  void* P = (void*)(size_t)4096;
  void* mis = (void*)(size_t)(4096 + 4);
  const size_t big = (size_t)1 << 40;
  const moe_shape s = shape(8, 4096, 64, 8, 768, 1, MOE_BF16);
  const moe_shape none = shape(0, 4096, 64, 8, 768, 1, MOE_BF16);
  const moe_q4_spec i128 = spec(MOE_Q4_INT4, 128), f32g = spec(MOE_Q4_E2M1, 32);

  /* stored sizes: 1 KB per 16 rows x 128 columns, scales padded to four tiles */
  {
    moe_q4_sizes z;
    const moe_shape odd = shape(8, 448, 7, 3, 160, 2, MOE_F32);
    CHECK(moe_q4_get_sizes(&s, &i128, &z) == MOE_OK);
    CHECK(z.w1_codes == (size_t)64 * 1536 * 4096 / 2 && z.w2_codes == (size_t)64 * 4096 * 768 / 2);
    CHECK(z.w1_scales == (size_t)64 * 1536 * 32 * 2 && z.w2_scales == (size_t)64 * 4096 * 8 * 2);
    CHECK(moe_q4_get_sizes(&odd, &f32g, &z) == MOE_OK);
    CHECK(z.w1_codes == (size_t)2 * 7 * 20 * 4 * 1024 && z.w2_codes == (size_t)2 * 7 * 28 * 2 * 1024);
    CHECK(z.w1_scales == (size_t)2 * 7 * 320 * 16 * 4 && z.w2_scales == (size_t)2 * 7 * 448 * 16 * 4);
    CHECK(moe_q4_get_sizes(&s, &i128, NULL) == MOE_ERR_INVALID_ARG);
    CHECK(moe_q4_get_sizes(NULL, &i128, &z) == MOE_ERR_INVALID_ARG);
  }
  /* the format, through every entry point */
  {
    const moe_q4_spec fmt = spec(2, 128), grp = spec(MOE_Q4_INT4, 16);
    const moe_shape im96 = shape(8, 4096, 64, 8, 96, 1, MOE_BF16);
    CHECK(moe_q4_quantize_w13(&s, &fmt, P, P, P, NULL) == MOE_ERR_INVALID_ARG);
    CHECK(moe_q4_quantize_down(&s, &grp, P, P, P, NULL) == MOE_ERR_INVALID_ARG);
    CHECK(moe_q4_w13_swiglu(&s, &fmt, P, P, P, P, P, P, NULL) == MOE_ERR_INVALID_ARG);
    CHECK(moe_q4_down(&s, NULL, P, P, P, P, P, NULL) == MOE_ERR_INVALID_ARG);
    CHECK(moe_forward_q4(&im96, &i128, P, P, NULL, P, P, P, P, P, P, big, NULL) == MOE_ERR_UNSUPPORTED);
  }
  /* pointers, workspaces, no tokens */
  {
    const size_t need = moe_workspace_size(&s), bal = moe_balance_workspace_size(&s);
    const size_t wg = moe_router_grad_workspace_size(&s);
    const moe_shape e65 = shape(8, 4096, 65, 8, 768, 1, MOE_BF16);
    CHECK(need > 0 && bal > 0 && wg > 0);
    CHECK(moe_balance_workspace_size(&e65) == 0 && moe_router_grad_workspace_size(&e65) == 0);
    CHECK(moe_q4_quantize_w13(&s, &i128, NULL, P, P, NULL) == MOE_ERR_INVALID_ARG);
    CHECK(moe_q4_quantize_down(&s, &i128, P, mis, P, NULL) == MOE_ERR_UNSUPPORTED);
    CHECK(moe_q4_w13_swiglu(&s, &i128, P, P, P, P, mis, P, NULL) == MOE_ERR_UNSUPPORTED);
    CHECK(moe_q4_down(&s, &i128, P, P, P, P, NULL, NULL) == MOE_ERR_INVALID_ARG);
    CHECK(moe_forward_q4(&s, &i128, P, P, NULL, P, P, P, P, P, P, need - 1, NULL) == MOE_ERR_WORKSPACE);
    CHECK(moe_forward_q4(&s, &i128, P, P, mis, P, P, P, P, P, P, need, NULL) == MOE_ERR_UNSUPPORTED);
    CHECK(moe_forward_q4(&none, &i128, P, P, NULL, P, P, P, P, P, NULL, 0, NULL) == MOE_OK);
    CHECK(moe_balance_loss(&s, P, P, NULL, P, P, P, P, bal - 1, NULL) == MOE_ERR_WORKSPACE);
    CHECK(moe_balance_loss(&s, P, P, mis, P, P, P, P, bal, NULL) == MOE_ERR_UNSUPPORTED);
    CHECK(moe_balance_loss(&s, P, NULL, NULL, P, P, P, P, bal, NULL) == MOE_ERR_INVALID_ARG);
    CHECK(moe_route_backward(&s, P, P, P, NULL, NULL, NULL, NULL, P, NULL) == MOE_ERR_INVALID_ARG); /* no gradient */
    CHECK(moe_route_backward(&s, P, P, P, NULL, NULL, NULL, P, P, NULL) == MOE_ERR_INVALID_ARG);    /* no counts */
    CHECK(moe_route_backward(&none, P, P, P, NULL, NULL, P, NULL, P, NULL) == MOE_OK);
    CHECK(moe_router_weight_grad(&s, P, P, NULL, P, NULL, P, wg - 1, NULL) == MOE_ERR_WORKSPACE);
    CHECK(moe_router_weight_grad(&s, P, P, NULL, P, mis, P, wg, NULL) == MOE_ERR_UNSUPPORTED);
    CHECK(moe_finalize_backward(&s, P, P, NULL, P, NULL) == MOE_ERR_INVALID_ARG);
    CHECK(moe_finalize_backward(&none, NULL, NULL, NULL, NULL, NULL) == MOE_OK);
  }

  printf("%s: %d failed\n", failures ? "abi_check FAILED" : "abi_check ok", failures);
  return failures;
}
