// Choice of the tile product's shape and split of the reduction, and the sum
// of a split's slices.
#include <algorithm>

#include "nm_ffn.hpp"

namespace nm {

int device_cu_count() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) dev = 0;
  return cu_count(dev);
}

TilePlan plan_tile(TileOp op, int64_t Mr, int64_t Nr, int nslab, int batch, int ebytes_out, int cus) {
  struct Shape {
    int bm, bn;
    double slab, tile;   // microseconds a slab and, besides, a tile takes
  };
  static const Shape shapes[3] = {{256, 256, 1.45, 6.0}, {128, 256, 0.95, 4.0}, {128, 128, 0.75, 3.0}};
  TilePlan best{0, 1, nslab};
  double best_t = 0;
  for (int i = 0; i < 3; ++i) {
    const int bn = op == TILE_GLU ? shapes[i].bn / 2 : shapes[i].bn;
    const int64_t tiles = (Mr + shapes[i].bm - 1) / shapes[i].bm * ((Nr + bn - 1) / bn) * batch;
    const int smax = op == TILE_LINEAR ? std::min(16, nslab) : 1;
    for (int s = 1; s <= smax; ++s) {
      const int sps = (nslab + s - 1) / s;
      const int split = (nslab + sps - 1) / sps;
      if (split != s) continue;
      const int64_t rounds = (tiles * split + cus - 1) / cus;
      double t = rounds * (sps * shapes[i].slab + shapes[i].tile) + 4.0;
      // the slices' sums written and read back at about 4 TB/s, and a launch
      if (split > 1) t += (double)Mr * Nr * (8.0 * split + ebytes_out) / 4e6 + 5.0;
      if (best_t == 0 || t < best_t) {
        best_t = t;
        best = TilePlan{i, split, sps};
      }
    }
  }
  return best;
}

namespace {

template <int OUT>
__global__ void __launch_bounds__(256) tile_reduce_kernel(const float* part, int split, int64_t T, int64_t R,
                                                          const float* bias, int act, void* C, int64_t ldc,
                                                          bool vec) {
  const int64_t pr = (R + 3) / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= T * pr) return;
  const int64_t t = i / pr, r = (i - t * pr) * 4;
  const int n = (int)min(R - r, (int64_t)4);
  float y[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < split; ++s) {
    const float* p = part + ((int64_t)s * T + t) * R + r;
    if (R % 4 == 0) {
      const v4f v = *reinterpret_cast<const v4f*>(p);
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
  store4<OUT>(C, t * ldc + r, y, n, vec);
}

}  // namespace

hipError_t launch_tile_reduce(const float* part, int split, int64_t T, int64_t R, const float* bias, int act, void* C,
                              int64_t ldc, int ydt, hipStream_t s) {
  const int64_t n = T * ((R + 3) / 4);
  const dim3 grid((unsigned)((n + 255) / 256)), block(256);
  const bool vec = vec4_ok(C, ldc, ydt == NM_F32 ? 4 : 2);
  if (ydt == NM_F16)
    hipLaunchKernelGGL((tile_reduce_kernel<NM_F16>), grid, block, 0, s, part, split, T, R, bias, act, C, ldc, vec);
  else if (ydt == NM_BF16)
    hipLaunchKernelGGL((tile_reduce_kernel<NM_BF16>), grid, block, 0, s, part, split, T, R, bias, act, C, ldc, vec);
  else
    hipLaunchKernelGGL((tile_reduce_kernel<NM_F32>), grid, block, 0, s, part, split, T, R, bias, act, C, ldc, vec);
  return hipGetLastError();
}

}  // namespace nm
