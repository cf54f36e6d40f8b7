// Tile products of grouped rows on the dense matrix cores: 8-bit rows; and the
// choice by element type.
#include "nm_tile.hpp"

namespace nm {
hipError_t launch_rows_tile_f16(int ydt, const RowsTile& a, hipStream_t s);
hipError_t launch_rows_tile_bf16(int ydt, const RowsTile& a, hipStream_t s);
hipError_t launch_rows_tile(int et, int ydt, const RowsTile& a, hipStream_t s) {
  if (et == TILE_F16) return launch_rows_tile_f16(ydt, a, s);
  if (et == TILE_BF16) return launch_rows_tile_bf16(ydt, a, s);
  if (ydt == NM_F16) return launch_tile_op<TILE_I8, TILE_ROWS, NM_F16>(a, s);
  if (ydt == NM_BF16) return launch_tile_op<TILE_I8, TILE_ROWS, NM_BF16>(a, s);
  return launch_tile_op<TILE_I8, TILE_ROWS, NM_F32>(a, s);
}
}  // namespace nm
