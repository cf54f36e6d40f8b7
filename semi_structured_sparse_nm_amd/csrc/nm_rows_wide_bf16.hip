// Products of grouped rows, a middle number of rows an expert: bf16 weights.
#include "nm_rows_wide.hpp"

namespace nm {
hipError_t launch_rows_wide_bf16(const RowsArgs& a, int tm, hipStream_t s) {
  return launch_rows_wide_wt<NM_BF16>(a, tm, s);
}
}  // namespace nm
