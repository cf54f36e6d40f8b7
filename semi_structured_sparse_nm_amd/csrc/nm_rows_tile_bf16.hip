// Tile products of grouped rows on the dense matrix cores: bf16.
#include "nm_tile.hpp"

namespace nm {
hipError_t launch_rows_tile_bf16(int ydt, const RowsTile& a, hipStream_t s) {
  return ydt == NM_BF16 ? launch_tile_op<TILE_BF16, TILE_ROWS, NM_BF16>(a, s) : hipErrorInvalidValue;
}
}  // namespace nm
