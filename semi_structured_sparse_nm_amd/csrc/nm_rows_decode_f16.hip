// Products of grouped rows, few rows an expert: fp16 weights.
#include "nm_rows_decode.hpp"

namespace nm {
hipError_t launch_rows_decode_f16(const RowsArgs& a, hipStream_t s) { return launch_rows_decode_wt<NM_F16>(a, s); }
}  // namespace nm
