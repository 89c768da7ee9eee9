// Launchers of the shared expert's training step, its request adapters and
// dropout (host side; every shape and pointer is checked by the caller).
#pragma once

#include "moe_common.h"
#include "philox.h"

namespace moe {

// Dimensions of the shared expert: T tokens, model width H, its own width I.
struct Ffn {
  int T, H, I;
  bool bf16;
};

// gu [T, 2I] (fp32) = x w1^T (gate, then up), hs [T, I] = dropout(SiLU(gate) * up)
hipError_t launch_train_w13(const Ffn& f, const Dropout& d, const void* x, const void* w1, void* gu, void* hs,
                            hipStream_t st);
// out [T, H] = hs w2^T (+ residual)
hipError_t launch_train_down(const Ffn& f, const void* hs, const void* w2, const void* residual, void* out,
                             hipStream_t st);
// d_gu [T, 2I] from d_out w2, gu and the dropout; d_x [T, H] = d_gu w1,
// d_w1 [2I, H] = d_gu^T x and d_w2 [H, I] = d_out^T hs; d_x, or d_w1 and d_w2, may
// be null (not wanted).  T == 0: d_w1 and d_w2 are zeros.
hipError_t launch_train_backward(const Ffn& f, const Dropout& d, const void* x, const void* w1, const void* w2,
                                 const void* gu, const void* hs, const void* d_out, void* d_gu, void* d_x, void* d_w1,
                                 void* d_w2, hipStream_t st);

// out = residual (may be null) + dropout(y), n elements, n a multiple of 8
hipError_t launch_dropout(bool bf16, const Dropout& d, long long n, const void* y, const void* residual, void* out,
                          hipStream_t st);

// Low-rank adapters: L of rank r.
struct Lora {
  int L, r;
};
constexpr int kLoraMaxAdapters = 1024, kLoraMaxRank = 128;
size_t lora_workspace_bytes(const Ffn& f, const Lora& l);
// launch_lora_w13 leaves the tokens sorted by adapter in the workspace;
// `sorted`: launch_lora_down finds them so.
hipError_t launch_lora_w13(const Ffn& f, const Lora& l, const void* x, const void* w1, const void* a, const void* b,
                           const float* scale, const int32_t* ids, void* hs, void* ws, hipStream_t st);
hipError_t launch_lora_down(const Ffn& f, const Lora& l, const void* hs, const void* w2, const void* a, const void* b,
                            const float* scale, const int32_t* ids, bool sorted, const void* residual, void* out,
                            void* ws, hipStream_t st);

}  // namespace moe
