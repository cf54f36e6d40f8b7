// Operands of the products of grouped rows: packed weights as dense blocks and
// transposed, rows of whole slabs, for the gradients.  All of them are bound by
// HBM: every element is read once and written once, in 16-byte pieces.
#include <algorithm>

#include "nm_expand_cols.hpp"
#include "nm_rows.hpp"

namespace nm {

namespace {

// whether expert e may have rows (surely not where its offsets say so as they are)
__device__ __forceinline__ bool may_have_rows(const RowGroups& o, int e) {
#if defined(__HIP_DEVICE_COMPILE__)
  return row_bound(o, e + 1) > row_bound(o, e);
#else
  return true;
#endif
}

// A thread makes 16 bytes of a dense block: piece q % 8 of its row q / 8.
template <int EB, int M>
__global__ void __launch_bounds__(256) rows_dense_kernel(Geometry g, const uint8_t* values, const uint8_t* meta,
                                                         RowGroups rows, uint8_t* dense) {
  const int64_t per = g.nRB * g.nKB;
  for (int64_t b = (int64_t)blockIdx.x * 2 + (threadIdx.x >> 7); b < per * rows.E; b += (int64_t)gridDim.x * 2) {
    if (!may_have_rows(rows, (int)(b / per))) continue;
    const int rr = (threadIdx.x & 127) >> 3, piece = threadIdx.x & 7;
    v4i o;
    if constexpr (EB == 1) {
      o = expand16_i8<M>(g, values, meta, b, rr, piece);
    } else {
      // (blocks of all experts are one row of blocks to expand8)
      Geometry one = g;
      one.nKB = 1;
      uint32_t h[4];
      expand8(one, values, meta, b * 16 + rr, 8 * piece, h);
      o = v4i{(int)h[0], (int)h[1], (int)h[2], (int)h[3]};
    }
    *reinterpret_cast<v4i*>(dense + b * 2048 + rr * 128 + 16 * piece) = o;
  }
}

// 128 rows x 64 columns of one expert's weight, expanded and transposed into
// blocks, and the kept bits.  Pitch 130 halves: the four 16-column runs of a
// packed row and its block's sixteen rows fall on different banks.
__device__ __forceinline__ void prepare_weight(const RowsPrepareArgs& a, int64_t b, uint16_t* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  uint16_t(*tile)[130] = reinterpret_cast<uint16_t(*)[130]>(lds);
  const Geometry& g = a.g;
  const int64_t rt = (g.R + 127) / 128, e = b / (rt * g.nKB);
  if (!may_have_rows(a.rows, (int)e)) return;
  uint16_t* kept = reinterpret_cast<uint16_t*>(a.mask + b * 1024);
  b -= e * rt * g.nKB;
  const int64_t kb = b % g.nKB, r0 = (b / g.nKB) * 128;
  const uint8_t* values = a.values + e * (int64_t)g.values_bytes();
  const uint8_t* meta = a.meta + e * (int64_t)g.meta_bytes();
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int rl = 16 * (it * 4 + (threadIdx.x >> 6)) + (lane >> 2), cl = (lane & 3) * 16;
    const int64_t r = r0 + rl;
    uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (r < g.R) {
      const int keep = (int)expand16(g, values, meta, r, kb * 64 + cl, o);
      if (a.mask) {
        // four lanes have a row's sixteen columns each: lane lq gathers bits 4 lq ..
        const int lq = lane & 3;
        const int k0 = __builtin_amdgcn_update_dpp(0, keep, 0x00, 0xf, 0xf, false);
        const int k1 = __builtin_amdgcn_update_dpp(0, keep, 0x55, 0xf, 0xf, false);
        const int k2 = __builtin_amdgcn_update_dpp(0, keep, 0xaa, 0xf, 0xf, false);
        const int k3 = __builtin_amdgcn_update_dpp(0, keep, 0xff, 0xf, 0xf, false);
        auto four = [&](int k) { return k >> (4 * lq) & 15; };
        kept[(lq * 16 + (lane >> 2)) * 8 + rl / 16] =
            (uint16_t)(four(k0) | four(k1) << 4 | four(k2) << 8 | four(k3) << 12);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) tile[cl + i][rl] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
  }
  if (!a.wt) return;
  __syncthreads();
  const int64_t Rs = (g.R + 63) / 64;                   // blocks along R
  uint16_t* wt = a.wt + e * ((g.K + 15) / 16 * Rs * 1024);
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int q = it * 256 + threadIdx.x;
    const int kl = q >> 4, rl = (q & 15) * 8;
    const int64_t k = kb * 64 + kl, s = (r0 + rl) >> 6;
    if (k < g.K && s < Rs) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(&tile[kl][rl]);
      *reinterpret_cast<v4i*>(wt + ((k >> 4) * Rs + s) * 1024 + (k & 15) * 64 + (rl & 63)) =
          v4i{(int)p[0], (int)p[1], (int)p[2], (int)p[3]};
    }
  }
#endif
}

constexpr int kPadPieces = 4 * 256;                     // of a workgroup in one step

// x's rows as rows of whole slabs of 64 columns, by n workgroups, this one b.
__device__ __forceinline__ void pad_rows(const uint16_t* x, int64_t ldx, int64_t T, int64_t cols, uint16_t* y,
                                         int64_t b, int64_t n) {
  const int64_t per = (cols + 63) / 64 * 8, total = T * per;
  for (int64_t q0 = b * kPadPieces; q0 < total; q0 += n * kPadPieces) {
    v4i o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t q = q0 + 256 * i + threadIdx.x, t = q / per, c = (q - t * per) * 8;
      o[i] = v4i{0, 0, 0, 0};
      if (q < total && c < cols) o[i] = load_piece(x + t * ldx, c, cols);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t q = q0 + 256 * i + threadIdx.x;
      if (q < total) *reinterpret_cast<v4i*>(y + q * 8) = o[i];
    }
  }
}

// What the gradients' products read, in one launch; workgroups take, by index,
// tiles of the weights (they pass through LDS), rows of X and of dY.
__global__ void __launch_bounds__(256) rows_prepare_kernel(RowsPrepareArgs a, int64_t n_weight, int64_t n_x) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[64 * 130];
  int64_t b = blockIdx.x;
  if (b < n_weight) return prepare_weight(a, b, lds);
  b -= n_weight;
  if (b < n_x) return pad_rows(a.X, a.ldx, a.rows.T, a.g.K, a.xp, b, n_x);
  pad_rows(a.dY, a.lddy, a.rows.T, a.g.R, a.yp, b - n_x, (int64_t)gridDim.x - n_weight - n_x);
}

}  // namespace

hipError_t launch_rows_dense(const Geometry& g, const uint8_t* values, const uint8_t* meta, const RowGroups& rows,
                             uint8_t* dense, hipStream_t s) {
  const int64_t n = g.nRB * g.nKB * rows.E;
  const dim3 grid(grid_1d(n * 128, 256)), block(256);
  if (g.eb == 1 && g.M == 4)
    hipLaunchKernelGGL((rows_dense_kernel<1, 4>), grid, block, 0, s, g, values, meta, rows, dense);
  else if (g.eb == 1)
    hipLaunchKernelGGL((rows_dense_kernel<1, 8>), grid, block, 0, s, g, values, meta, rows, dense);
  else
    hipLaunchKernelGGL((rows_dense_kernel<2, 4>), grid, block, 0, s, g, values, meta, rows, dense);
  return hipGetLastError();
}

hipError_t launch_rows_prepare(const RowsPrepareArgs& a, hipStream_t s) {
  const int64_t n_weight = a.wt || a.mask ? a.rows.E * ((a.g.R + 127) / 128) * a.g.nKB : 0;
  auto pads = [&](int64_t cols) {
    return std::min<int64_t>((a.rows.T * ((cols + 63) / 64) * 8 + kPadPieces - 1) / kPadPieces, 4096);
  };
  const int64_t n_x = a.xp ? pads(a.g.K) : 0, n_y = a.yp ? pads(a.g.R) : 0;
  hipLaunchKernelGGL(rows_prepare_kernel, dim3((unsigned)(n_weight + n_x + n_y)), dim3(256), 0, s, a, n_weight, n_x);
  return hipGetLastError();
}

}  // namespace nm
