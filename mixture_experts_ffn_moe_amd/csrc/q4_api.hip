// Entry points of the layer over 4-bit expert weights (moe_q4.h): checks and
// launch sequence.
#include "../../include/moe_q4.h"
#include "api_check.h"
#include "decode_route.h"
#include "q4.h"

using namespace moe_api;
using moe::Q4;

namespace {

static_assert(moe::kQ4Int == MOE_Q4_INT4 && moe::kQ4E2m1 == MOE_Q4_E2M1, "formats of the header and the kernels");

moe_status check_q4(const Shape& s, const moe_q4_spec* q4, Q4* out) {
  if (q4 == nullptr) return MOE_ERR_INVALID_ARG;
  if (q4->format != MOE_Q4_INT4 && q4->format != MOE_Q4_E2M1) return MOE_ERR_INVALID_ARG;
  if (q4->group != 32 && q4->group != 64 && q4->group != 128) return MOE_ERR_INVALID_ARG;
  if (s.H % q4->group != 0 || s.Im % q4->group != 0) return MOE_ERR_UNSUPPORTED;
  *out = Q4{q4->format, q4->group};
  return MOE_OK;
}

void sizes_of(const Shape& s, const Q4& q, moe_q4_sizes* z) {
  const size_t mats = (size_t)s.mu * s.E, e = elem_bytes(s);
  z->w1_codes = mats * (2 * s.Im / 16) * q.kb(s.H) * moe::kQ4TileBytes;
  z->w1_scales = mats * 2 * s.Im * q.stride(s.H) * e;
  z->w2_codes = mats * (s.H / 16) * q.kb(s.Im) * moe::kQ4TileBytes;
  z->w2_scales = mats * s.H * q.stride(s.Im) * e;
}

// The router with H split over 16 workgroups per 16 tokens, and a second launch
// that adds the parts, instead of one workgroup per 16 tokens, which takes 44
// us however few they are: 256 tokens 13 us, 1024 tokens 23 us; at 2048 the
// two are even.
constexpr int kSplitRouteTokens = 1024;
bool split_route(const Shape& s) {
  return s.bf16 && s.T <= kSplitRouteTokens && s.H % (moe::kSplit * 128) == 0 &&
         moe::route_tiles_bytes(s) <= y_bytes(s, s.R());
}

}  // namespace

extern "C" {

moe_status moe_q4_get_sizes(const moe_shape* shape, const moe_q4_spec* q4, moe_q4_sizes* sizes) {
  Shape s;
  Q4 q;
  MOE_CHECK(check_shape(shape, &s));
  MOE_CHECK(check_q4(s, q4, &q));
  if (sizes == nullptr) return MOE_ERR_INVALID_ARG;
  sizes_of(s, q, sizes);
  return MOE_OK;
}

moe_status moe_q4_quantize_w13(const moe_shape* shape, const moe_q4_spec* q4, const void* w1, void* codes,
                               void* scales, void* stream) {
  Shape s;
  Q4 q;
  MOE_CHECK(check_shape(shape, &s));
  MOE_CHECK(check_q4(s, q4, &q));
  MOE_CHECK(check_ptr(w1)); MOE_CHECK(check_ptr(codes)); MOE_CHECK(check_ptr(scales));
  return hip_status(moe::launch_q4_quantize(q, s.bf16, w1, (long long)s.mu * s.E, 2 * s.Im, s.H, true, codes, scales,
                                            (hipStream_t)stream));
}

moe_status moe_q4_quantize_down(const moe_shape* shape, const moe_q4_spec* q4, const void* w2, void* codes,
                                void* scales, void* stream) {
  Shape s;
  Q4 q;
  MOE_CHECK(check_shape(shape, &s));
  MOE_CHECK(check_q4(s, q4, &q));
  MOE_CHECK(check_ptr(w2)); MOE_CHECK(check_ptr(codes)); MOE_CHECK(check_ptr(scales));
  return hip_status(moe::launch_q4_quantize(q, s.bf16, w2, (long long)s.mu * s.E, s.H, s.Im, false, codes, scales,
                                            (hipStream_t)stream));
}

moe_status moe_q4_w13_swiglu(const moe_shape* shape, const moe_q4_spec* q4, const void* x, const int32_t* perm,
                             const int32_t* offsets, const void* w1_codes, const void* w1_scales, void* h,
                             void* stream) {
  Shape s;
  Q4 q;
  MOE_CHECK(check_shape(shape, &s));
  MOE_CHECK(check_q4(s, q4, &q));
  if (s.T == 0) return MOE_OK;
  MOE_CHECK(check_ptr(x)); MOE_CHECK(check_ptr(perm)); MOE_CHECK(check_ptr(offsets));
  MOE_CHECK(check_ptr(w1_codes)); MOE_CHECK(check_ptr(w1_scales)); MOE_CHECK(check_ptr(h));
  return hip_status(moe::launch_q4_w13(s, q, x, perm, offsets, w1_codes, w1_scales, h, (hipStream_t)stream));
}

moe_status moe_q4_down(const moe_shape* shape, const moe_q4_spec* q4, const void* h, const int32_t* offsets,
                       const void* w2_codes, const void* w2_scales, void* y, void* stream) {
  Shape s;
  Q4 q;
  MOE_CHECK(check_shape(shape, &s));
  MOE_CHECK(check_q4(s, q4, &q));
  if (s.T == 0) return MOE_OK;
  MOE_CHECK(check_ptr(h)); MOE_CHECK(check_ptr(offsets)); MOE_CHECK(check_ptr(w2_codes));
  MOE_CHECK(check_ptr(w2_scales)); MOE_CHECK(check_ptr(y));
  return hip_status(moe::launch_q4_down(s, q, h, offsets, w2_codes, w2_scales, y, (hipStream_t)stream));
}

moe_status moe_forward_q4(const moe_shape* shape, const moe_q4_spec* q4, const void* x, const float* wg,
                          const float* bias, const void* w1_codes, const void* w1_scales, const void* w2_codes,
                          const void* w2_scales, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  Shape s;
  Q4 q;
  MOE_CHECK(check_shape(shape, &s));
  MOE_CHECK(check_q4(s, q4, &q));
  if (s.T == 0) return MOE_OK;
  MOE_CHECK(check_ptr(x)); MOE_CHECK(check_ptr(wg)); MOE_CHECK(check_ptr(w1_codes)); MOE_CHECK(check_ptr(w1_scales));
  MOE_CHECK(check_ptr(w2_codes)); MOE_CHECK(check_ptr(w2_scales)); MOE_CHECK(check_ptr(out));
  if (bias != nullptr) MOE_CHECK(check_ptr(bias));
  moe_workspace_layout L;
  MOE_CHECK(moe_get_workspace_layout(shape, &L));
  if (workspace == nullptr || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  if (((uintptr_t)workspace & (kAlign - 1)) != 0) return MOE_ERR_UNSUPPORTED;
  char* ws = (char*)workspace;
  float* logits = (float*)(ws + L.logits);
  int32_t* ids = (int32_t*)(ws + L.topk_ids);
  float* w = (float*)(ws + L.topk_w);
  int32_t* counts = (int32_t*)(ws + L.counts);
  int32_t* offsets = (int32_t*)(ws + L.offsets);
  int32_t* perm = (int32_t*)(ws + L.perm);
  int32_t* inv = (int32_t*)(ws + L.inv);
  void* h = ws + L.h;
  void* y = ws + L.y;
  hipStream_t st = (hipStream_t)stream;
  if (moe::q4_decode_supported(s))
    return hip_status(moe::launch_q4_decode(s, q, x, wg, bias, w1_codes, w1_scales, w2_codes, w2_scales, out, logits,
                                            ids, w, counts, offsets, perm, inv, h, ws + L.scratch, st));
  int32_t* hist = (int32_t*)(ws + L.scratch);
  if (split_route(s))  // the partial sums lie where y will
    MOE_CHECK(hip_status(moe::launch_route_tiles(s, x, wg, bias, (double*)y, logits, ids, w, hist, st)));
  else
    MOE_CHECK(hip_status(moe::launch_route(s, x, wg, bias, logits, ids, w, st, hist)));
  MOE_CHECK(hip_status(moe::launch_permute_hist(s, ids, hist, counts, offsets, perm, inv, st)));
  MOE_CHECK(hip_status(moe::launch_q4_w13(s, q, x, perm, offsets, w1_codes, w1_scales, h, st)));
  MOE_CHECK(hip_status(moe::launch_q4_down(s, q, h, offsets, w2_codes, w2_scales, y, st)));
  return hip_status(moe::launch_finalize(s, y, inv, w, out, st));
}

}  // extern "C"
