// Gated block for few tokens, fp16 weights; and the choice by weight type.
#include "nm_glu_decode.hpp"

namespace nm {
hipError_t launch_glu_decode_bf16(const GluArgs& a, hipStream_t s);
hipError_t launch_glu_decode(const GluArgs& a, hipStream_t s) {
  return a.wdt == NM_F16 ? launch_glu_decode_wt<NM_F16>(a, s) : launch_glu_decode_bf16(a, s);
}
}  // namespace nm
