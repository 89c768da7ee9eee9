// Host-side checks and sizes shared by the entry points of every header.
#pragma once

#include "../../include/moe_mi355x.h"
#include "moe_common.h"

namespace moe_api {

using moe::Shape;

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Shape checks shared by every entry point.
inline moe_status check_shape(const moe_shape* sh, Shape* out) {
  if (sh == nullptr) return MOE_ERR_INVALID_ARG;
  const moe_shape& s = *sh;
  if (s.T < 0 || s.H <= 0 || s.E <= 0 || s.k <= 0 || s.Im <= 0 || s.micro_count <= 0)
    return MOE_ERR_INVALID_ARG;
  if (s.k > s.E) return MOE_ERR_INVALID_ARG;
  if (s.dtype != MOE_F32 && s.dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (s.renormalize != 0 && s.renormalize != 1) return MOE_ERR_INVALID_ARG;
  if (s.E > moe::kMaxExperts) return MOE_ERR_UNSUPPORTED;
  // k-steps of 64 over H (w13) and of 32 over Im (down); w13 output tiles of
  // 32 columns; down output tiles of 64 columns (the fp32 path)
  if (s.H % 64 != 0 || s.Im % 32 != 0) return MOE_ERR_UNSUPPORTED;
  const long long R = (long long)s.T * s.k;
  const long long I = (long long)s.micro_count * s.Im;
  const long long lim = (1ll << 31) - 1;
  // the GEMMs address one expert's weight block (w1: 2*Im x H, w2: H x Im)
  // with 32-bit byte offsets
  const long long expert_w1_bytes = 4ll * s.Im * s.H;
  if (R > lim || I > lim || R * s.H > lim || R * I > lim || (long long)s.T * s.H > lim ||
      (long long)s.micro_count * s.E * 2 * s.Im * s.H > lim * 8 || expert_w1_bytes > 0xffffffffll)
    return MOE_ERR_UNSUPPORTED;
  if (out) {
    out->T = s.T; out->H = s.H; out->E = s.E; out->k = s.k; out->Im = s.Im;
    out->mu = s.micro_count; out->bf16 = (s.dtype == MOE_BF16);
    out->renorm = (s.renormalize != 0);
  }
  return MOE_OK;
}

// Non-null and 16-byte aligned (the kernels move 16-byte vectors).
inline moe_status check_ptr(const void* p) {
  if (p == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(p)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

#define MOE_CHECK(expr)                 \
  do {                                  \
    const moe_status st_ = (expr);      \
    if (st_ != MOE_OK) return st_;      \
  } while (0)

inline moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

inline size_t elem_bytes(const Shape& s) { return s.bf16 ? 2 : 4; }

static_assert(moe::kYBlock == MOE_Y_BLOCK, "y block of the header and the kernels");

// A y buffer of `rows` rows: fp32 in the fp32 layer, block-scaled half in the
// bf16 layers (moe_common.h).
inline size_t y_bytes(const Shape& s, long long rows) {
  return s.bf16 ? moe::y_half_bytes(rows, s.H) : (size_t)rows * s.H * 4;
}

}  // namespace moe_api
