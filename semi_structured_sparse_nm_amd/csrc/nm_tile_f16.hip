// Tile product instantiations, operand type f16 (one file per type so that they compile in parallel).
#include "nm_tile.hpp"

namespace nm {
hipError_t launch_tile_f16(TileOp op, int ydt, const TileArgs& a, hipStream_t s) {
  return launch_tile<TILE_F16>(op, ydt, a, s);
}
}  // namespace nm
