// Tile product instantiations, operand type mx (one file per type so that they compile in parallel).
#include "nm_tile.hpp"

namespace nm {
hipError_t launch_tile_mx(TileOp op, int ydt, const TileArgs& a, hipStream_t s) {
  return launch_tile<TILE_MX>(op, ydt, a, s);
}
}  // namespace nm
