// Gate|up product with SwiGLU over 4-bit weights (kernel: q4_rows.h).
#include "q4_rows.h"

namespace moe {

hipError_t launch_q4_w13(const Shape& s, const Q4& q, const void* x, const int32_t* perm, const int32_t* offsets,
                         const void* codes, const void* scales, void* h, hipStream_t st) {
  Q4Rows a = {};
  a.x = x; a.perm = perm; a.offsets = offsets; a.codes = (const uint8_t*)codes; a.scales = scales; a.out = h;
  a.E = s.E; a.k = s.k; a.K = s.H; a.ldx = s.H; a.N = 2 * s.Im; a.S = q.stride(s.H); a.KB = q.kb(s.H);
  a.segments = 1; a.tiles = s.mu * (s.Im / 8); a.Im = s.Im;
  return launch_rows<true>(s, q, a, st);
}

}  // namespace moe
