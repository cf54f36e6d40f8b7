// Tile products of grouped rows on the dense matrix cores: fp16.
#include "nm_tile.hpp"

namespace nm {
hipError_t launch_rows_tile_f16(int ydt, const RowsTile& a, hipStream_t s) {
  return ydt == NM_F16 ? launch_tile_op<TILE_F16, TILE_ROWS, NM_F16>(a, s) : hipErrorInvalidValue;
}
}  // namespace nm
