// Gated block on 2:4 weights through the sparse tile kernel: instantiations.
#include "nm_tile24.hpp"

namespace nm {

// tokens in X's own rows (a.X, a.ldx: 16-byte pieces), both weights 2:4
hipError_t launch_glu_tile24(const GluArgs& g, hipStream_t s) {
  Tile24Args p{};
  TileArgs& a = p.t;
  a.A[0] = a.A[1] = static_cast<const uint8_t*>(g.X);
  a.lda = g.ldx * 2;
  a.Mr = g.T;
  a.Nr = g.g.R;
  a.ka = (int)(g.g.K / 8);
  a.nslab = (int)g.g.nKB;
  a.C[0] = g.H;
  a.ldc = g.ldh;
  a.P[0] = g.P[0];
  a.P[1] = g.P[1];
  a.ldp = g.ldp;
  a.act = g.act;
  a.batch = 1;
  a.split = 1;
  a.sps = a.nslab;
  for (int i = 0; i < 2; ++i) {
    p.values[i] = g.values[i];
    p.meta[i] = g.meta[i];
  }
  // fewer tokens a tile where 256 of them would leave compute units idle
  const int64_t nt = (g.g.R + 127) / 128;
  const int cus = device_cu_count();
  auto rounds = [&](int bm) { return ((g.T + bm - 1) / bm * nt + cus - 1) / cus; };
  const bool wide = rounds(256) * 1.0 <= rounds(128) * 0.62;
  if (g.wdt == NM_F16)
    return wide ? launch_tile24_cfg<NM_F16, 4, 3>(p, s) : launch_tile24_cfg<NM_F16, 2, 4>(p, s);
  return wide ? launch_tile24_cfg<NM_BF16, 4, 3>(p, s) : launch_tile24_cfg<NM_BF16, 2, 4>(p, s);
}

}  // namespace nm
