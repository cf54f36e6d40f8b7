// Products of grouped rows, few rows an expert: 8-bit weights; and the choice
// by weight type.
#include "nm_rows_decode.hpp"

namespace nm {
// Tiles of 16 rows: those an expert has as a mean.  Waves of a workgroup along K:
// as many as find eight blocks each (what a wave does once, before and after them,
// is 300 vector and 350 scalar instructions), but no fewer workgroups than compute
// units; the workgroup's other waves have row blocks of their own.
void rows_decode_plan(const Geometry& g, int64_t T, int64_t E, int* nt, int* ks, int64_t* workgroups) {
  const int64_t some = std::min(T, E);
  *nt = stream_tiles(g.nRB * some, (T + some - 1) / some);
  const int64_t units = units_most(T, E, 16 * *nt);
  *ks = kGluWaves;
  while (*ks > 1 && g.nKB < 8 * *ks && g.nRB * units * (*ks / 2) / kGluWaves >= device_cu_count()) *ks /= 2;
  const int64_t rows = 8 * (kGluWaves / *ks);          // row blocks of eight workgroups
  *workgroups = (g.nRB + rows - 1) / rows * 8 * units;
}
hipError_t launch_rows_decode_i8(const RowsArgs& a, hipStream_t s) { return launch_rows_decode_wt<NM_I8>(a, s); }
hipError_t launch_rows_decode(const RowsArgs& a, hipStream_t s) {
  if (a.wdt == NM_I8) return launch_rows_decode_i8(a, s);
  return a.wdt == NM_F16 ? launch_rows_decode_f16(a, s) : launch_rows_decode_bf16(a, s);
}
}  // namespace nm
