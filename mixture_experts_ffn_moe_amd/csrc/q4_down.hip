// Down product over 4-bit weights, the micro-shards summed in the accumulator
// (kernel: q4_rows.h).
#include "q4_rows.h"

namespace moe {

hipError_t launch_q4_down(const Shape& s, const Q4& q, const void* h, const int32_t* offsets, const void* codes,
                          const void* scales, void* y, hipStream_t st) {
  Q4Rows a = {};
  a.x = h; a.offsets = offsets; a.codes = (const uint8_t*)codes; a.scales = scales; a.out = y;
  a.ye = s.bf16 ? (int8_t*)y + (size_t)s.R() * s.H * 2 : nullptr;
  a.E = s.E; a.k = s.k; a.K = s.Im; a.ldx = s.mu * s.Im; a.N = s.H; a.S = q.stride(s.Im); a.KB = q.kb(s.Im);
  a.segments = s.mu; a.tiles = s.H / 16;
  return launch_rows<false>(s, q, a, st);
}

}  // namespace moe
