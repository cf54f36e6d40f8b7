// Products of grouped rows, a middle number of rows an expert: 8-bit weights; and
// the choice by weight type.
#include "nm_rows_wide.hpp"

namespace nm {
hipError_t launch_rows_wide_i8(const RowsArgs& a, int tm, hipStream_t s) {
  return launch_rows_wide_wt<NM_I8>(a, tm, s);
}
hipError_t launch_rows_wide(const RowsArgs& a, int tm, hipStream_t s) {
  if (a.wdt == NM_I8) return launch_rows_wide_i8(a, tm, s);
  return a.wdt == NM_F16 ? launch_rows_wide_f16(a, tm, s) : launch_rows_wide_bf16(a, tm, s);
}
}  // namespace nm
