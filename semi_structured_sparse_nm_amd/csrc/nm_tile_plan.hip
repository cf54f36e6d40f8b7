// Choice of the tile product's shape and split of the reduction, and the sum
// of a split's slices.
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "nm_ffn.hpp"

namespace nm {

int device_cu_count() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) dev = 0;
  return cu_count(dev);
}

// Two 4:8 weights of 1000 x 3000, 64 tokens: four tiles 10.4 us on 63 compute
// units, one tile 7.0 on 252; of 3000 x 2000: four 9.0 on 188, two 9.6.
int stream_tiles(int64_t blocks, int64_t T) {
  int nt = T <= 16 ? 1 : T <= 32 ? 2 : 4;
  while (nt > 1 && blocks * ((T + 16 * nt - 1) / (16 * nt)) < device_cu_count() / 2) nt /= 2;
  return nt;
}

// The debug override NM_FFN_TILE=<kind>:<shape>[:<split>], kind "tile" (the dense
// tile product) or "tile24" (the sparse one): that shape, and for a product
// that takes one that split, or the next smaller one its slabs divide into;
// kind "stream", 0 or 1: whether a product streams its weights.  For tests.
bool ffn_tile_override(const char* kind, int* shape, int* split) {
  const char* e = getenv("NM_FFN_TILE");
  if (!e) return false;
  const char* c = strchr(e, ':');
  if (!c || (size_t)(c - e) != strlen(kind) || strncmp(e, kind, c - e)) return false;
  const int v = atoi(c + 1);
  if (v < 0 || v > 3) return false;
  *shape = v;
  c = strchr(c + 1, ':');
  if (c && split) *split = std::max(0, std::min(16, atoi(c + 1)));
  return true;
}

// Microseconds a slab takes with few workgroups running and with one on every
// compute unit (their operands' traffic, and for the forward products the power
// the matrix cores draw, slow each other down), and a tile besides its slabs.
// Fitted to products of 64 to 2048 tokens by 411 to 11008 x 182 to 11008; the
// choice is within 7% of the fastest shape and split there.  For example 2048 tokens, two 4:8 weights
// of 11008 x 4096, gated: 256 x 256 tiles 290 us, 128 x 256 306; 600 tokens, 1614
// x 2364: 68, 44, 128 x 128 32 and 64 x 128 41; at 4 bits 26, 17, 12 and 18.
namespace {

struct TileShape {
  int bm, bn;
  double idle[2], busy[2], tile;   // [1]: microscaled operands
  double slab(bool mx, int64_t items, int cus) const {
    return idle[mx] + (busy[mx] - idle[mx]) * std::min(1.0, (double)items / cus);
  }
};
constexpr TileShape kShapes[4] = {{256, 256, {0.93, 1.10}, {1.50, 1.60}, 6.0},
                                  {128, 256, {0.47, 0.72}, {0.85, 0.97}, 5.0},
                                  {128, 128, {0.42, 0.50}, {0.60, 0.65}, 4.0},
                                  {64, 128, {0.25, 0.35}, {0.34, 0.42}, 3.5}};

int64_t tiles(int64_t Mr, int64_t Nr, int bm, int bn) { return (Mr + bm - 1) / bm * ((Nr + bn - 1) / bn); }

// the slices' sums written and read back, and a launch
double split_time(int64_t Mr, int64_t Nr, int split) {
  return split > 1 ? (double)Mr * Nr * (8.0 * split + 2.0) / 8e6 + 5.0 : 0.0;
}

// plan(shape, split, slabs of a slice) -> time, over all of them
template <class F>
TilePlan best_plan(int smax, int nslab, F&& time) {
  int only = -1, only_split = 0;
  ffn_tile_override("tile", &only, &only_split);
  if (only_split) {
    // the most slices up to the forced ones that the slabs divide into
    const int sps = (nslab + std::min(only_split, smax) - 1) / std::min(only_split, smax);
    only_split = (nslab + sps - 1) / sps;
  }
  TilePlan best{0, 1, nslab, 0, 0};
  for (int i = 0; i < 4; ++i) {
    if (only >= 0 && i != only) continue;
    for (int s = 1; s <= smax; ++s) {
      const int sps = (nslab + s - 1) / s;
      const int split = (nslab + sps - 1) / sps;
      if (split != s || (only_split && s != only_split)) continue;
      TilePlan p{i, split, sps, 0, 0};
      p.time = time(kShapes[i], p);
      if (best.time == 0 || p.time < best.time) best = p;
    }
  }
  return best;
}

}  // namespace

TilePlan plan_tile(TileOp op, bool mx, int64_t Mr, int64_t Nr, int nslab, int cus) {
  return best_plan(op == TILE_LINEAR ? std::min(16, nslab) : 1, nslab, [&](const TileShape& h, TilePlan& p) {
    const int64_t items = tiles(Mr, Nr, h.bm, op == TILE_GLU ? h.bn / 2 : h.bn) * p.split;
    return (double)((items + cus - 1) / cus) * (p.sps * h.slab(mx, items, cus) + h.tile) + split_time(Mr, Nr, p.split);
  });
}

// The products' items are dealt to an XCD's workgroups as TileWalk does.  Its
// own constants, fitted to 18 sizes of 3 to 2048 tokens in every shape and
// split: a slab with few and with all compute units at work, a tile of the
// input's gradient and of a weight's besides its slabs (its mask is read).  The
// choice is within 5% of the fastest at 16 of them, within 9% at the others
// (for example 30 tokens, two weights of 3490 x 3688: 128 x 128 tiles 67 us, 256
// x 256 81; 1024 tokens, 11008 x 4096: 573 and 477).
TilePlan plan_back(int64_t T, int64_t R, int64_t K, int nslab_x, int nslab_w, bool dx, bool dw, int cus) {
  struct Cost {
    double idle, busy, x, w;
  };
  static const Cost costs[4] = {{0.69, 1.30, 6.1, 10.8},
                                {0.39, 0.67, 5.0, 6.6},
                                {0.29, 0.375, 2.7, 3.8},
                                {0.11, 0.25, 1.4, 2.55}};
  return best_plan(dx ? std::min(16, nslab_x) : 1, nslab_x, [&](const TileShape& h, TilePlan& p) {
    const Cost& c = costs[p.shape];
    const int64_t a = dx ? (tiles(T, K, h.bm, h.bn) * p.split + 7) / 8 : 0;
    const int64_t b = dw ? (2 * tiles(R, K, h.bm, h.bn) + 7) / 8 : 0;
    const int64_t w = std::min<int64_t>(a + b, (cus + 7) / 8), q = a % w;
    const double slab = c.idle + (c.busy - c.idle) * std::min(1.0, 8.0 * (double)(a + b) / cus);
    const double ta = p.sps * slab + c.x, tb = nslab_w * slab + c.w;
    const int64_t most = (b + w - q - 1) / (w - q), near = (int64_t)(ta / tb);
    double best = 0;
    for (const int64_t lead : {int64_t(0), near, near + 1, most}) {
      if (lead > most || (lead && !q)) continue;
      const int64_t rest = std::max<int64_t>(0, (b - lead * (w - q) + w - 1) / w);
      const double t = std::max((double)((a + w - 1) / w) * ta + rest * tb, (double)(a / w) * ta + (lead + rest) * tb);
      if (best == 0 || t < best) {
        best = t;
        p.lead = (int)lead;
      }
    }
    // (and a launch, of which small calls wait for the host's part)
    if (p.split > 1) best += (double)T * (double)K * (8.0 * p.split + 2.0) / 16.4e6 + 4.5;
    return best;
  });
}

namespace {

template <int OUT>
__global__ void __launch_bounds__(256) tile_reduce_kernel(const float* part, int split, int64_t T, int64_t R,
                                                          const float* bias, int act, void* C, int64_t ldc) {
  const int64_t pr = (R + 3) / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= T * pr) return;
  const int64_t t = i / pr, r = (i - t * pr) * 4;
  const int n = (int)min(R - r, (int64_t)4);
  float y[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < split; ++s) {
    const float* p = part + ((int64_t)s * T + t) * R + r;
    if (n == 4) {
      const v4f v = *reinterpret_cast<const v4f_any*>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] += v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) y[e] += p[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (bias && e < n) y[e] += bias[r + e];
    if (act == NM_ACT_GELU) y[e] = gelu_f32(y[e]);
  }
  store4<OUT>(C, t * ldc + r, y, n);
}

}  // namespace

hipError_t launch_tile_reduce(const float* part, int split, int64_t T, int64_t R, const float* bias, int act, void* C,
                              int64_t ldc, int ydt, hipStream_t s) {
  const int64_t n = T * ((R + 3) / 4);
  const dim3 grid((unsigned)((n + 255) / 256)), block(256);
  if (ydt == NM_F16)
    hipLaunchKernelGGL((tile_reduce_kernel<NM_F16>), grid, block, 0, s, part, split, T, R, bias, act, C, ldc);
  else if (ydt == NM_BF16)
    hipLaunchKernelGGL((tile_reduce_kernel<NM_BF16>), grid, block, 0, s, part, split, T, R, bias, act, C, ldc);
  else
    hipLaunchKernelGGL((tile_reduce_kernel<NM_F32>), grid, block, 0, s, part, split, T, R, bias, act, C, ldc);
  return hipGetLastError();
}

}  // namespace nm
