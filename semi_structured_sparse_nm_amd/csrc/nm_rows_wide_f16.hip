// Products of grouped rows, a middle number of rows an expert: fp16 weights.
#include "nm_rows_wide.hpp"

namespace nm {
hipError_t launch_rows_wide_f16(const RowsArgs& a, int tm, hipStream_t s) {
  return launch_rows_wide_wt<NM_F16>(a, tm, s);
}
}  // namespace nm
