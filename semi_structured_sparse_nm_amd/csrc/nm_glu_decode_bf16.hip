// Gated block for few tokens, bfloat16 weights.
#include "nm_glu_decode.hpp"

namespace nm {
hipError_t launch_glu_decode_bf16(const GluArgs& a, hipStream_t s) { return launch_glu_decode_wt<NM_BF16>(a, s); }
}  // namespace nm
