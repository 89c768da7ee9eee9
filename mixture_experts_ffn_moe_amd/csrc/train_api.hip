// Entry points of the shared expert's training step and of dropout
// (moe_shared_train.h), and of the request adapters (moe_lora.h): checks and
// launch sequences.
#include "../../include/moe_lora.h"
#include "../../include/moe_shared_train.h"
#include "api_check.h"
#include "shared_train.h"

using namespace moe_api;
using moe::Dropout;
using moe::Ffn;
using moe::Lora;

namespace {

constexpr int kMaxWidth = 1 << 20;  // H and 2 * Is: 256 rows of a tile stay below 32-bit byte offsets

// The shared expert's dimensions.  Weights are addressed with 32-bit byte
// offsets from their first row (gate and up rows of one tile).
moe_status check_ffn(const moe_shape* shape, int32_t Is, Ffn* f) {
  Shape s;
  MOE_CHECK(check_shape(shape, &s));
  if (Is <= 0) return MOE_ERR_INVALID_ARG;
  const long long lim = (1ll << 31) - 1;
  if (Is % 32 != 0 || s.H > kMaxWidth || Is > kMaxWidth / 2) return MOE_ERR_UNSUPPORTED;
  if (2ll * s.T * Is > lim || 2ll * Is * s.H * (long long)elem_bytes(s) > 0xffffffffll) return MOE_ERR_UNSUPPORTED;
  *f = Ffn{s.T, s.H, Is, s.bf16};
  return MOE_OK;
}

moe_status check_dropout(double p, const uint64_t* rng, Dropout* d) {
  if (!(p >= 0.0 && p < 1.0)) return MOE_ERR_INVALID_ARG;
  const uint32_t cut = (uint32_t)(p * 65536.0 + 0.5);
  if (cut >= 65536u) return MOE_ERR_INVALID_ARG;
  if (cut == 0) {
    *d = Dropout{nullptr, 0, 1.0f};
    return MOE_OK;
  }
  MOE_CHECK(check_ptr(rng));
  *d = Dropout{rng, cut, (float)(65536.0 / (65536u - cut))};
  return MOE_OK;
}

moe_status check_or_null(const void* p) { return p == nullptr ? MOE_OK : check_ptr(p); }

moe_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (ws == nullptr || bytes < need) return MOE_ERR_WORKSPACE;
  if (((uintptr_t)ws & (kAlign - 1)) != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t backward_bytes(const Ffn& f) { return align_up((size_t)f.T * 2 * f.I * (f.bf16 ? 2 : 4)); }

// Sorted tokens are gathered with 32-bit byte offsets from the first.
moe_status check_lora(const Ffn& f, const moe_lora_spec* spec, Lora* l) {
  if (spec == nullptr || spec->adapters <= 0 || spec->rank <= 0) return MOE_ERR_INVALID_ARG;
  if (spec->adapters > moe::kLoraMaxAdapters || spec->rank > moe::kLoraMaxRank || spec->rank % 8 != 0)
    return MOE_ERR_UNSUPPORTED;
  const long long width = f.H > f.I ? f.H : f.I;
  if ((long long)f.T * width * (f.bf16 ? 2 : 4) > 0xffffffffll) return MOE_ERR_UNSUPPORTED;
  *l = Lora{spec->adapters, spec->rank};
  return MOE_OK;
}

static_assert(moe::kLoraMaxAdapters == MOE_LORA_MAX_ADAPTERS && moe::kLoraMaxRank == MOE_LORA_MAX_RANK,
              "limits of the header and the kernels");

}  // namespace

extern "C" {

moe_status moe_dropout_add(const moe_shape* shape, double p, const uint64_t* rng, const void* y, const void* residual,
                           void* out, void* stream) {
  Shape s;
  Dropout d;
  MOE_CHECK(check_shape(shape, &s));
  MOE_CHECK(check_dropout(p, rng, &d));
  if (s.T == 0) return MOE_OK;
  MOE_CHECK(check_ptr(y)); MOE_CHECK(check_or_null(residual)); MOE_CHECK(check_ptr(out));
  return hip_status(moe::launch_dropout(s.bf16, d, (long long)s.T * s.H, y, residual, out, (hipStream_t)stream));
}

moe_status moe_dropout_backward(const moe_shape* shape, double p, const uint64_t* rng, const void* d_out, void* d_y,
                                void* stream) {
  return moe_dropout_add(shape, p, rng, d_out, nullptr, d_y, stream);
}

moe_status moe_shared_ffn_train(const moe_shape* shape, int32_t Is, double p, const uint64_t* rng, const void* x,
                                const void* w1s, const void* w2s, const void* residual, float* gu, void* hs, void* out,
                                void* stream) {
  Ffn f;
  Dropout d;
  MOE_CHECK(check_ffn(shape, Is, &f));
  MOE_CHECK(check_dropout(p, rng, &d));
  if (f.T == 0) return MOE_OK;
  MOE_CHECK(check_ptr(x)); MOE_CHECK(check_ptr(w1s)); MOE_CHECK(check_ptr(w2s)); MOE_CHECK(check_or_null(residual));
  MOE_CHECK(check_ptr(gu)); MOE_CHECK(check_ptr(hs)); MOE_CHECK(check_ptr(out));
  hipStream_t st = (hipStream_t)stream;
  MOE_CHECK(hip_status(moe::launch_train_w13(f, d, x, w1s, gu, hs, st)));
  return hip_status(moe::launch_train_down(f, hs, w2s, residual, out, st));
}

size_t moe_shared_backward_workspace_size(const moe_shape* shape, int32_t Is) {
  Ffn f;
  if (check_ffn(shape, Is, &f) != MOE_OK) return 0;
  return f.T == 0 ? kAlign : backward_bytes(f);
}

moe_status moe_shared_ffn_backward(const moe_shape* shape, int32_t Is, double p, const uint64_t* rng, const void* x,
                                   const void* w1s, const void* w2s, const float* gu, const void* hs,
                                   const void* d_out, void* d_x, void* d_w1s, void* d_w2s, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  Ffn f;
  Dropout d;
  MOE_CHECK(check_ffn(shape, Is, &f));
  MOE_CHECK(check_dropout(p, rng, &d));
  // an empty batch's d_x has no elements, and may have no address either
  if ((d_w1s == nullptr) != (d_w2s == nullptr) || (f.T > 0 && d_x == nullptr && d_w1s == nullptr))
    return MOE_ERR_INVALID_ARG;
  MOE_CHECK(check_or_null(d_x)); MOE_CHECK(check_or_null(d_w1s)); MOE_CHECK(check_or_null(d_w2s));
  if (f.T > 0) {
    if (d_w1s) MOE_CHECK(check_ptr(x));
    if (d_w1s) MOE_CHECK(check_ptr(hs));
    if (d_x) MOE_CHECK(check_ptr(w1s));
    MOE_CHECK(check_ptr(w2s)); MOE_CHECK(check_ptr(gu)); MOE_CHECK(check_ptr(d_out));
    MOE_CHECK(check_workspace(workspace, workspace_bytes, backward_bytes(f)));
  }
  return hip_status(moe::launch_train_backward(f, d, x, w1s, w2s, gu, hs, d_out, workspace, d_x, d_w1s, d_w2s,
                                               (hipStream_t)stream));
}

size_t moe_lora_workspace_size(const moe_shape* shape, int32_t Is, const moe_lora_spec* spec) {
  Ffn f;
  Lora l;
  if (check_ffn(shape, Is, &f) != MOE_OK || check_lora(f, spec, &l) != MOE_OK) return 0;
  return f.T == 0 ? kAlign : moe::lora_workspace_bytes(f, l);
}

moe_status moe_lora_w13_swiglu(const moe_shape* shape, int32_t Is, const moe_lora_spec* spec, const void* x,
                               const void* w1s, const void* a1, const void* b1, const float* scale,
                               const int32_t* adapter_ids, void* hs, void* workspace, size_t workspace_bytes,
                               void* stream) {
  Ffn f;
  Lora l;
  MOE_CHECK(check_ffn(shape, Is, &f));
  MOE_CHECK(check_lora(f, spec, &l));
  if (f.T == 0) return MOE_OK;
  MOE_CHECK(check_ptr(x)); MOE_CHECK(check_ptr(w1s)); MOE_CHECK(check_ptr(a1)); MOE_CHECK(check_ptr(b1));
  MOE_CHECK(check_ptr(scale)); MOE_CHECK(check_ptr(adapter_ids)); MOE_CHECK(check_ptr(hs));
  MOE_CHECK(check_workspace(workspace, workspace_bytes, moe::lora_workspace_bytes(f, l)));
  hipStream_t st = (hipStream_t)stream;
  return hip_status(moe::launch_lora_w13(f, l, x, w1s, a1, b1, scale, adapter_ids, hs, workspace, st));
}

moe_status moe_lora_down(const moe_shape* shape, int32_t Is, const moe_lora_spec* spec, const void* hs,
                         const void* w2s, const void* a2, const void* b2, const float* scale,
                         const int32_t* adapter_ids, const void* residual, void* out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  Ffn f;
  Lora l;
  MOE_CHECK(check_ffn(shape, Is, &f));
  MOE_CHECK(check_lora(f, spec, &l));
  if (f.T == 0) return MOE_OK;
  MOE_CHECK(check_ptr(hs)); MOE_CHECK(check_ptr(w2s)); MOE_CHECK(check_ptr(a2)); MOE_CHECK(check_ptr(b2));
  MOE_CHECK(check_ptr(scale)); MOE_CHECK(check_ptr(adapter_ids)); MOE_CHECK(check_or_null(residual));
  MOE_CHECK(check_ptr(out));
  MOE_CHECK(check_workspace(workspace, workspace_bytes, moe::lora_workspace_bytes(f, l)));
  hipStream_t st = (hipStream_t)stream;
  return hip_status(moe::launch_lora_down(f, l, hs, w2s, a2, b2, scale, adapter_ids, false, residual, out, workspace, st));
}

moe_status moe_shared_ffn_lora(const moe_shape* shape, int32_t Is, const moe_lora_spec* spec, const void* x,
                               const void* w1s, const void* w2s, const void* a1, const void* b1, const void* a2,
                               const void* b2, const float* scale, const int32_t* adapter_ids, const void* residual,
                               void* hs, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  Ffn f;
  Lora l;
  MOE_CHECK(check_ffn(shape, Is, &f));
  MOE_CHECK(check_lora(f, spec, &l));
  if (f.T == 0) return MOE_OK;
  MOE_CHECK(check_ptr(x)); MOE_CHECK(check_ptr(w1s)); MOE_CHECK(check_ptr(w2s)); MOE_CHECK(check_ptr(a1));
  MOE_CHECK(check_ptr(b1)); MOE_CHECK(check_ptr(a2)); MOE_CHECK(check_ptr(b2)); MOE_CHECK(check_ptr(scale));
  MOE_CHECK(check_ptr(adapter_ids)); MOE_CHECK(check_or_null(residual)); MOE_CHECK(check_ptr(hs));
  MOE_CHECK(check_ptr(out));
  MOE_CHECK(check_workspace(workspace, workspace_bytes, moe::lora_workspace_bytes(f, l)));
  hipStream_t st = (hipStream_t)stream;
  MOE_CHECK(hip_status(moe::launch_lora_w13(f, l, x, w1s, a1, b1, scale, adapter_ids, hs, workspace, st)));
  return hip_status(moe::launch_lora_down(f, l, hs, w2s, a2, b2, scale, adapter_ids, true, residual, out, workspace, st));
}

}  // extern "C"
