// How a product of grouped rows multiplies: time models of its paths.
//
// Fitted to 1084 products of 17 to 2048 rows an expert, 1 to 64 experts, 300 to
// 11008 outputs, K 512 to 11008, seven patterns, 8 and 16 bits, every path and tile
// shape measured with weights that change between calls
// (profiles/rows_plan_products.csv): the wide and tile models are 4 to 10% off as a
// root mean square, the streamed one 24 to 32%; the path taken costs 2.1% against the
// fastest as a mean over them, 8% or more in one of ten, 51% at most.
// For example, streamed, wide (64 rows), wide (128), best tiles, in microseconds:
// 8-bit 4:8, 48 rows, 11008 x 4096 25, 33, 41, 42; 256 rows 59, 34, 41, 49; 32 experts
// of 1536 x 2048, 16-bit 4:8, 256 rows 42, 30, 37, 149, 4096 rows -, 49, 63, 175;
// 16-bit 2:4, 4096 rows of 8 experts of 2048 x 4096 587, 102, 97, 69.
#include <algorithm>

#include "nm_rows.hpp"

namespace nm {

namespace {

// What a pattern costs the paths that expand in registers: 2:4 as it is, dense,
// up to four kept of eight columns and more (byte permutes by a table), and the
// 16-bit 5:8 (value by value).
enum Kind { SPARSE, DENSE, FEW, MANY, SHIFTED, KINDS };
Kind kind_of(const Geometry& g) {
  if (g.N == 2 && g.M == 4) return SPARSE;
  if (g.N == g.M) return DENSE;
  if (g.eb == 2 && g.N == 5) return SHIFTED;
  return 8 * g.N / g.M <= 4 ? FEW : MANY;
}

// Microseconds: a workgroup besides its slabs, a slab with one workgroup on every
// compute unit, what a further workgroup on the compute unit costs of one alone, and
// the part of a slab's time that stays with few workgroups.
struct Wide {
  double base, slab, more, idle;
};
constexpr Wide kWide[2][2][KINDS] = {
    // 8 bits (slabs of 128 columns): 64 rows, 128 rows
    {{{4.97, 0.632, 0.833, 0.779}, {6.07, 1.07, 0.868, 0.836}, {5.10, 0.805, 0.785, 0.865}, {5.67, 1.15, 0.776, 0.862},
      {}},
     {{6.10, 0.831, 0.963, 0.671}, {7.77, 1.15, 0.923, 0.811}, {6.75, 1.15, 0.951, 0.802}, {7.38, 1.41, 0.925, 0.807},
      {}}},
    // 16 bits (64 columns)
    {{{3.41, 0.601, 0.785, 0.677}, {4.94, 1.03, 0.904, 0.867}, {4.35, 0.669, 0.790, 0.816}, {4.69, 0.823, 0.819, 0.818},
      {5.01, 1.32, 0.873, 0.920}},
     {{4.89, 0.741, 0.951, 0.680}, {6.32, 1.20, 0.888, 0.765}, {5.73, 0.997, 0.833, 0.778}, {6.02, 1.20, 0.974, 0.739},
      {6.26, 1.64, 0.981, 0.843}}}};

// A workgroup besides its blocks, a wave's block, and that for each 16-row tile.
struct Stream {
  double base, block, tile;
};
constexpr Stream kStream[2][KINDS] = {
    {{1.12, 0.153, 0.224}, {1.98, 0.237, 0.223}, {1.56, 0.172, 0.223}, {1.31, 0.471, 0.253}, {}},
    {{0.20, 0.119, 0.267}, {0.34, 0.418, 0.235}, {0.56, 0.232, 0.231}, {1.07, 0.300, 0.213}, {0.59, 0.663, 0.143}}};

// Tile shapes (rows x outputs): a tile besides its slabs, a slab with one tile on
// every compute unit, and with few.
struct Shape {
  int bm, bn;
};
constexpr Shape kShapes[4] = {{256, 256}, {128, 256}, {128, 128}, {64, 128}};
struct Tile {
  double base, busy, idle;
};
constexpr Tile kTiles[2][2][4] = {
    // 8 bits: dense, 2:4
    {{{8.01, 1.30, 1.01}, {5.46, 0.777, 0.546}, {3.46, 0.487, 0.337}, {2.82, 0.312, 0.241}},
     {{8.77, 0.920, 0.643}, {6.43, 0.611, 0.429}, {4.22, 0.380, 0.291}, {3.31, 0.270, 0.241}}},
    // 16 bits
    {{{4.79, 1.62, 1.00}, {3.55, 0.908, 0.533}, {2.46, 0.523, 0.327}, {2.20, 0.330, 0.226}},
     {{5.70, 0.910, 0.611}, {3.82, 0.606, 0.373}, {2.88, 0.367, 0.265}, {2.27, 0.281, 0.238}}}};

constexpr double kRate = 4.4e6;              // bytes of weights a microsecond

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// units of u rows: of several experts each one's last is half full as a mean
double units(int64_t T, int64_t E, int64_t u) {
  return E == 1 ? (double)ceil_div(T, u) : (double)T / u + 0.5 * (double)std::min(T, E);
}

// rounds of n workgroups over the compute units: whole ones of one expert; of
// several, whose sizes the host does not know, part of one more
double rounds(double n, int64_t E, int cus, double more) {
  const double r = n / cus;
  return std::max(1.0, E == 1 ? (double)(int64_t)(r + 0.999999) : r + more);
}

double wide_time(const Geometry& g, int64_t T, int64_t E, int tm, double bytes, int cus) {
  const Wide& w = kWide[g.eb - 1][tm == 8][kind_of(g)];
  const double n = units(T, E, 16 * tm) * (double)ceil_div(g.R, 256), r = rounds(n, E, cus, 0.55);
  // (two workgroups of 64 rows share a compute unit, those of 128 follow each other)
  const double in_turn = tm == 4 ? std::max(1.0, w.more * r) : n <= cus ? 1.0 : 1.0 + w.more * (r - 1.0);
  const double slab = w.slab * (w.idle + (1.0 - w.idle) * std::min(1.0, n / cus));
  return 3.0 + std::max((w.base + g.nKB * slab) * in_turn, bytes / kRate);
}

double stream_time(const Geometry& g, int64_t T, int64_t E, double bytes, int cus) {
  const Stream& w = kStream[g.eb - 1][kind_of(g)];
  int nt, ks;
  int64_t most;
  rows_decode_plan(g, T, E, &nt, &ks, &most);
  const double n = units(T, E, 16 * nt) * (double)ceil_div(g.nRB, 8 / ks), r = n / cus;
  const double in_turn = std::max(1.0, E == 1 && r < 3 ? (double)(int64_t)(r + 0.999999) : r + 1.0);
  return 4.7 + std::max(in_turn * (w.base + (double)ceil_div(g.nKB, ks) * (w.block + w.tile * nt)), bytes / kRate);
}

double tile_time(const Tile& c, const Shape& h, double row_units, int64_t R, int64_t nslab, int64_t E, int cus) {
  const double n = row_units * (double)ceil_div(R, h.bn);
  const double slab = c.idle + (c.busy - c.idle) * std::min(1.0, n / cus);
  return 5.0 + rounds(n, E, cus, 0.45) * (c.base + nslab * slab);
}

}  // namespace

namespace {

// The tile product's shape, cut and rest, and its time by the model.
RowsPlan tiles_plan(RowsPath path, const Geometry& g, int64_t T, int64_t E, int cus, double* time) {
  const bool sparse = path != ROWS_DENSE, small_table = sparse && g.eb == 1 && E >= kRowsTable / 2;
  const Tile* tiles = kTiles[g.eb - 1][sparse];
  auto time_of = [&](int i, int64_t R) {
    return tile_time(tiles[i], kShapes[i], units(T, E, kShapes[i].bm), R, g.nKB, E, cus);
  };
  RowsPlan best{path, 3};
  *time = 0;
  auto take = [&](double t, const RowsPlan& p) {
    if (*time > 0 && t >= *time) return;
    *time = t;
    best = p;
  };
  int only = 0;
  const bool forced = ffn_tile_override(sparse ? "tile24" : "tile", &only, nullptr);
  for (int i = 0; i < 4; ++i) {
    // (the 8-bit shapes whose table of boundaries is the smaller one)
    if (small_table && i % 2 == 0) continue;
    if (forced && i != (small_table ? only | 1 : only)) continue;
    take(time_of(i, g.R), RowsPlan{path, i});
    if (E > 1 || forced) continue;
    // one weight: whole rounds in one shape, then the rest in smaller tiles (a second
    // launch costs 3 us of the 5 that a first one does)
    const int64_t mt = ceil_div(T, kShapes[i].bm), nt = ceil_div(g.R, kShapes[i].bn);
    const int64_t cut = mt * nt / cus * cus / mt * kShapes[i].bn;
    if (cut == 0 || cut >= g.R) continue;
    const double t = time_of(i, cut);
    for (int j = i + 1; j < 4; ++j) take(t + time_of(j, g.R - cut) - 2.0, RowsPlan{path, i, cut, j});
  }
  return best;
}

}  // namespace

int grads_tile_shape(const Geometry& g, int64_t T, int64_t E, bool dx, bool dw, int cus, int* lead) {
  int best = 0, only;
  double least = 0;
  const bool forced = ffn_tile_override("tile", &only, nullptr);
  for (int i = forced ? only : 0; i < (forced ? only + 1 : 4); ++i) {
    const Shape& h = kShapes[i];
    const double nx = dx ? units(T, E, h.bm) * (double)ceil_div(g.K, h.bn) : 0.0;
    const double nw = dw ? (double)(E * ceil_div(g.R, h.bm)) * (double)ceil_div(g.K, h.bn) : 0.0;
    const Tile& c = kTiles[1][0][i];
    const double slab = c.idle + (c.busy - c.idle) * std::min(1.0, (nx + nw) / cus);
    const double tx = dx ? c.base + (double)ceil_div(g.R, 64) * slab : 0.0;
    const double tw = c.base + ((double)T / 64.0 / E + 0.5) * slab;
    // all of it on every compute unit, and half of the longer kind's tile at the end
    const double longer = std::max(tx, dw ? tw : 0.0);
    const double t = std::max(longer, (nx * tx + nw * tw) / cus + 0.5 * longer);
    if (least == 0 || t < least) {
      least = t;
      best = i;
      *lead = (int)std::min(tx / tw + 0.5, 64.0);
    }
  }
  return best;
}

RowsPlan rows_plan(const Geometry& g, int64_t T, int64_t E, int cus) {
  // (re-packing takes up to 64 threads a block in one launch)
  const bool repack = repack24_supported(g) && E * g.nRB * g.nKB < (1ll << 26);
  double time;
  const RowsPlan tiles =
      tiles_plan(g.N == 2 && g.M == 4 ? ROWS_SPARSE : repack ? ROWS_REPACK : ROWS_DENSE, g, T, E, cus, &time);
  // a launch has fewer than 2^32 threads
  int nt, ks;
  int64_t most;
  rows_decode_plan(g, T, E, &nt, &ks, &most);
  const bool can_stream = most < (1 << 22);
  auto can_wide = [&](int tm) { return units_most(T, E, 16 * tm) * ceil_div(g.R, 256) < (1 << 22); };
  int v;
  if (ffn_tile_override("wide", &v, nullptr) && can_wide(v ? 8 : 4)) return {ROWS_WIDE, v ? 8 : 4};
  if (ffn_tile_override("stream", &v, nullptr)) return v && can_stream ? RowsPlan{ROWS_STREAM, 0} : tiles;
  if (ffn_tile_override("tile", &v, nullptr) || ffn_tile_override("tile24", &v, nullptr)) return tiles;
  const int64_t groups = std::min(T, E), mean = ceil_div(T, groups);
  // (by the mean alone, the host knows no more: sixteen rows of each of 32 experts of 1536
  // x 2048, 16-bit 2:4, 32 us evenly, 33 by a router, 25 all of one expert's, wide 24, 24
  // and 20; of 8 experts of 2048 x 4096 23, 23 and 20, the fastest others 23, 23 and 22;
  // four rows of each of the 32 25, 25 and 13, others 24, 24 and 14)
  if (mean <= 16 && can_stream) return {ROWS_STREAM, 0};

  const double dense = (double)E * (double)(g.nRB * g.nKB) * 2048.0;
  const double bytes = (double)E * (double)(g.values_bytes() + g.meta_bytes());
  if (tiles.path == ROWS_REPACK) time += (bytes + dense * (0.5 + 0.125 / g.eb)) / 4.7e6;
  if (tiles.path == ROWS_DENSE && g.N != g.M) time += 2.0 + (bytes + dense) / 3.1e6;
  RowsPlan best = tiles;
  if (mean <= 1024 && can_stream) {
    const double t = stream_time(g, T, E, bytes, cus);
    if (t < time) {
      time = t;
      best = {ROWS_STREAM, 0};
    }
  }
  for (const int tm : {4, 8}) {
    if (!can_wide(tm)) continue;
    const double t = wide_time(g, T, E, tm, bytes, cus);
    if (t < time) {
      time = t;
      best = {ROWS_WIDE, tm};
    }
  }
  return best;
}

}  // namespace nm
