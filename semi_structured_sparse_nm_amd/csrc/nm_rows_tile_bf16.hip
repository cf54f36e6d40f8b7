// Tile products of grouped rows on the dense matrix cores: bf16.
#include "nm_tile.hpp"

namespace nm {
hipError_t launch_rows_tile_bf16(TileOp op, int ydt, const RowsTile& a, hipStream_t s) {
  if (ydt != NM_BF16) return hipErrorInvalidValue;
  return op == TILE_COLS ? launch_tile_op<TILE_BF16, TILE_COLS, NM_BF16>(a, s)
                         : launch_tile_op<TILE_BF16, TILE_ROWS, NM_BF16>(a, s);
}
}  // namespace nm
