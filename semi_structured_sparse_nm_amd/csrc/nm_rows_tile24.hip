// Tile products of grouped rows on 2:4 weights: instantiations.
#include "nm_tile24.hpp"

namespace nm {

namespace {

// Tile shapes, rows x outputs: 256 x 256, 128 x 256, 128 x 128, 64 x 128.
template <int WT, int OUT>
hipError_t launch_shape(const RowsTile& p, hipStream_t s) {
  switch (p.shape) {
    case 0: return launch_rows24_cfg<WT, OUT, 4, 4, 3>(p, s);
    case 1: return launch_rows24_cfg<WT, OUT, 2, 4, 4>(p, s);
    case 2: return launch_rows24_cfg<WT, OUT, 2, 2, 6>(p, s);
    default: return launch_rows24_cfg<WT, OUT, 1, 2, 8>(p, s);
  }
}

}  // namespace

hipError_t launch_rows_tile24(int wdt, int ydt, const RowsTile& p, hipStream_t s) {
  if (wdt == NM_I8) {
    if (ydt == NM_F16) return launch_shape<NM_I8, NM_F16>(p, s);
    if (ydt == NM_BF16) return launch_shape<NM_I8, NM_BF16>(p, s);
    return launch_shape<NM_I8, NM_F32>(p, s);
  }
  if (ydt != wdt) return hipErrorInvalidValue;
  return wdt == NM_F16 ? launch_shape<NM_F16, NM_F16>(p, s) : launch_shape<NM_BF16, NM_BF16>(p, s);
}

}  // namespace nm
