// Products of grouped rows, few rows an expert: 8-bit weights; and the choice
// by weight type.
#include "nm_rows_decode.hpp"

namespace nm {
hipError_t launch_rows_decode_i8(const RowsArgs& a, hipStream_t s) { return launch_rows_decode_wt<NM_I8>(a, s); }
hipError_t launch_rows_decode(const RowsArgs& a, hipStream_t s) {
  if (a.wdt == NM_I8) return launch_rows_decode_i8(a, s);
  return a.wdt == NM_F16 ? launch_rows_decode_f16(a, s) : launch_rows_decode_bf16(a, s);
}
}  // namespace nm
