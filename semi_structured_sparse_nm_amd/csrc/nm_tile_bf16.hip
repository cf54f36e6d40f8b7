// Tile product instantiations, operand type bf16 (one file per type so that they compile in parallel).
#include "nm_tile.hpp"

namespace nm {
hipError_t launch_tile_bf16(TileOp op, int ydt, const TileArgs& a, hipStream_t s) {
  return launch_tile<TILE_BF16>(op, ydt, a, s);
}
}  // namespace nm
