// Gated block on 2:4 weights through the sparse tile kernel: instantiations.
#include "nm_tile24.hpp"

namespace nm {

namespace {

// Tile shapes (tokens x outputs), with the microseconds a slab and, besides, a
// tile takes.  Measured at K = 4096 (64 slabs), one tile on every compute
// unit, and the least of rounds times (slabs x first + second) picks the
// fastest or is within 10% of it for 11008 and 4096 outputs and 32 to 2048
// tokens: e.g. 11008 outputs, 64 tokens 26 us (128 x 128: 39), 128 tokens 33
// (64 x 64: 44), 256 tokens 44 (256 x 128: 58), 512 tokens 62 (128 x 128: 85).
struct Shape24 {
  int tokens, outputs;
  double slab, tile;
};
constexpr Shape24 kShapes24[4] = {{256, 128, 1.0, 5.0}, {128, 128, 0.55, 5.0}, {128, 64, 0.40, 5.0}, {64, 64, 0.31, 5.0}};

double shape24_time(const Shape24& h, int64_t T, int64_t R, int64_t nslab, int cus) {
  const int64_t tiles = (T + h.tokens - 1) / h.tokens * ((R + h.outputs - 1) / h.outputs);
  return (double)((tiles + cus - 1) / cus) * (nslab * h.slab + h.tile);
}

template <int WT>
hipError_t launch_shape24(int shape, const Tile24Args& p, hipStream_t s) {
  switch (shape) {
    case 0: return launch_tile24_cfg<WT, 4, 4, 3>(p, s);
    case 1: return launch_tile24_cfg<WT, 2, 4, 4>(p, s);
    case 2: return launch_tile24_cfg<WT, 2, 2, 6>(p, s);
    default: return launch_tile24_cfg<WT, 1, 2, 8>(p, s);
  }
}

}  // namespace

double glu_tile24_time(int64_t T, int64_t R, int64_t nslab, int cus, int* shape) {
  double best = 0;
  int only;
  if (ffn_tile_override("tile24", &only, nullptr)) {
    if (shape) *shape = only;
    return 0;
  }
  for (int i = 0; i < 4; ++i) {
    const double t = shape24_time(kShapes24[i], T, R, nslab, cus);
    if (i == 0 || t < best) {
      best = t;
      if (shape) *shape = i;
    }
  }
  return best;
}

// tokens in X's own rows (a.X, a.ldx: 16-byte pieces), both weights 2:4
hipError_t launch_glu_tile24(const GluArgs& g, hipStream_t s) {
  Tile24Args p{};
  TileArgs& a = p.t;
  a.A = static_cast<const uint8_t*>(g.X);
  a.lda = g.ldx * 2;
  a.Mr = g.T;
  a.Nr = g.g.R;
  a.ka = (int)(g.g.K / 8);
  a.nslab = (int)g.g.nKB;
  a.C = g.H;
  a.ldc = g.ldh;
  a.P[0] = g.P[0];
  a.P[1] = g.P[1];
  a.ldp = g.ldp;
  a.p32 = g.p32;
  a.act = g.act;
  a.split = 1;
  a.sps = a.nslab;
  for (int i = 0; i < 2; ++i) {
    p.values[i] = g.values[i];
    p.meta[i] = g.meta[i];
  }
  int shape = 0;
  glu_tile24_time(g.T, g.g.R, a.nslab, device_cu_count(), &shape);
  return g.wdt == NM_F16 ? launch_shape24<NM_F16>(shape, p, s) : launch_shape24<NM_BF16>(shape, p, s);
}

}  // namespace nm
