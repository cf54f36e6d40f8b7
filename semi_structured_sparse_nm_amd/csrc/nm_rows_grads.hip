// Gradients of grouped rows: instantiations.
#include "nm_tile.hpp"

namespace nm {
hipError_t launch_rows_grads(int et, const RowsTile& x, const RowsTile& w, int shape, hipStream_t s) {
  if (et == TILE_F16) return launch_grads<TILE_F16, NM_F16>(x, w, shape, s);
  if (et == TILE_BF16) return launch_grads<TILE_BF16, NM_BF16>(x, w, shape, s);
  return hipErrorInvalidValue;
}
}  // namespace nm
