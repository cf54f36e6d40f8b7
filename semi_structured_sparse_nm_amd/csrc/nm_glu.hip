// Data movement around the gated block's tile products: packed weights
// expanded to dense rows or dense columns, the activation's backward step,
// padded activation rows.  All of them are bound by HBM: every element is
// read once and written once, in 16-byte pieces.
#include "nm_expand_cols.hpp"

namespace nm {

namespace {

// blockIdx.y: the weight.  A wave covers one packed block (16 rows x 64
// columns), lane 4 r + q its columns 16 q .. of row r.
__global__ void __launch_bounds__(256) expand_dense_kernel(Geometry g, DenseArgs a) {
  const uint8_t* values = blockIdx.y ? a.values[1] : a.values[0];
  const uint8_t* meta = blockIdx.y ? a.meta[1] : a.meta[0];
  uint16_t* dense = blockIdx.y ? a.dense[1] : a.dense[0];
  const int lane = threadIdx.x & 63;
  const int64_t blk = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (blk >= g.nRB * g.nKB) return;
  const int64_t rb = blk / g.nKB, kb = blk - rb * g.nKB;
  const int64_t r = rb * 16 + (lane >> 2), c = kb * 64 + (lane & 3) * 16;
  if (r >= g.R) return;
  uint32_t o[8];
  expand16(g, values, meta, r, c, o);
  v4i* d = reinterpret_cast<v4i*>(dense + r * (g.nKB * 64) + c);
  d[0] = v4i{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
  d[1] = v4i{(int)o[4], (int)o[5], (int)o[6], (int)o[7]};
}

template <int WT>
__device__ __forceinline__ void load8(const uint16_t* p, int64_t r, int64_t R, float (&f)[8]) {
  const v4i x = load_piece(p, r, R);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = from_16<WT>(((uint32_t)x[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
}
// eight kept products from r: binary32, or 16-bit with infinities made finite
template <int WT, bool P32>
__device__ __forceinline__ void load_kept(const void* P, int64_t row, int64_t r, int64_t R, float (&f)[8]) {
  if constexpr (P32) {
    const float* p = static_cast<const float*>(P) + row + r;
    if (r + 8 <= R) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const v4f x = *reinterpret_cast<const v4f_any*>(p + 4 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * i + e] = x[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = r + i < R ? p[i] : 0.f;
    }
  } else {
    load8<WT>(static_cast<const uint16_t*>(P) + row, r, R, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = finite_16<WT>(f[i]);
  }
}

// what rounding x0, x1 to the pair h left, rounded (0 where it gave an infinity)
template <int WT>
__device__ __forceinline__ uint32_t rest_16x2(float x0, float x1, uint32_t h) {
  const float h0 = from_16<WT>(h & 0xFFFFu), h1 = from_16<WT>(h >> 16);
  return pack_16x2<WT>(__builtin_isinf(h0) ? 0.f : x0 - h0, __builtin_isinf(h1) ? 0.f : x1 - h1);
}

// What the backward pass's products read, in one launch; workgroups take, by
// index, one of three kinds of tile:
//
//  - 64 tokens x 64 outputs of dG and dU, as rows (d) and transposed (dt).  They
//    are rounded to the weights' 16-bit type here: operands of the matrix
//    instruction in both products that follow (half a step each, as any
//    16-bit operand).  A kept product past the type's range (fp16: the forward
//    pass has it in binary32 and H stays finite) counts as the largest value:
//    as an infinity it would meet the slope's zero and make whole rows NaN.
//  - 128 rows x 64 columns of one weight, expanded and transposed (wt), with
//    the bits of the kept columns.
//  - 64 tokens x 64 columns of X, transposed (xt).
//
// Tiles pass through LDS; every element is read and written once, in 16-byte
// pieces of at least 128 contiguous bytes: 595 MB in 120 us (5 TB/s, a large
// copy's rate) for 2048 tokens and two 2:4 weights of 11008 x 4096, 685 in 137
// with the kept products in binary32.
template <int WT, int TH, bool P32, int PARTS>
__device__ __forceinline__ void prepare_dact(const PrepareArgs& a, int64_t b, uint16_t* lds) {
  // pitch 66 halves: eight pieces of a row (8 rows apart here) and eight
  // tokens fall on different banks
  uint16_t(*tile)[64][66] = reinterpret_cast<uint16_t(*)[64][66]>(lds);
  const int64_t tt = (a.T + 63) / 64;
  const int64_t t0 = (b % tt) * 64, r0 = (b / tt) * 64;
#pragma unroll
  for (int it = 0; it < 512 / TH; ++it) {
    const int q = it * TH + threadIdx.x;
    const int tl = q >> 3, rl = (q & 7) * 8;
    const int64_t t = t0 + tl, r = r0 + rl;
    uint32_t og[PARTS][4] = {}, ou[PARTS][4] = {};
    if (t < a.T && r < a.g.R) {
      float h[8], g[8], u[8];
      load8<WT>(a.dH + t * a.lddh, r, a.g.R, h);
      load_kept<WT, P32>(a.G, t * a.ldp, r, a.g.R, g);
      load_kept<WT, P32>(a.U, t * a.ldp, r, a.g.R, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float dg[2], du[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y, dy;
          glu_act_slope(a.act, g[2 * i + e], y, dy);
          const bool in = r + 2 * i + e < a.g.R;
          dg[e] = in ? h[2 * i + e] * u[2 * i + e] * dy : 0.f;
          du[e] = in ? h[2 * i + e] * y : 0.f;
        }
        og[0][i] = pack_16x2<WT>(dg[0], dg[1]);
        ou[0][i] = pack_16x2<WT>(du[0], du[1]);
        if constexpr (PARTS == 2) {
          og[1][i] = rest_16x2<WT>(dg[0], dg[1], og[0][i]);
          ou[1][i] = rest_16x2<WT>(du[0], du[1], ou[0][i]);
        }
      }
    }
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      if (a.d && t < a.T) {
        uint16_t* d = a.d + t * (2 * PARTS * a.Rp) + 2 * p * a.Rp + r;
        *reinterpret_cast<v4i*>(d) = v4i{(int)og[p][0], (int)og[p][1], (int)og[p][2], (int)og[p][3]};
        *reinterpret_cast<v4i*>(d + a.Rp) = v4i{(int)ou[p][0], (int)ou[p][1], (int)ou[p][2], (int)ou[p][3]};
      }
      if (a.dt) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          tile[2 * p][rl + e][tl] = (uint16_t)(og[p][e >> 1] >> (16 * (e & 1)));
          tile[2 * p + 1][rl + e][tl] = (uint16_t)(ou[p][e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
  if (!a.dt) return;
  __syncthreads();
#pragma unroll
  for (int it = 0; it < PARTS * 1024 / TH; ++it) {
    const int q = it * TH + threadIdx.x;
    const int w = (q >> 9) & 1, rl = (q >> 3) & 63, tl = (q & 7) * 8;
    if (r0 + rl < a.g.R) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(&tile[q >> 9][rl][tl]);
      *reinterpret_cast<v4i*>(a.dt + (((int64_t)w * a.g.R + r0 + rl) * PARTS + (q >> 10)) * a.Tp + t0 + tl) =
          v4i{(int)p[0], (int)p[1], (int)p[2], (int)p[3]};
    }
  }
}

template <int TH, int PARTS>
__device__ __forceinline__ void prepare_weight(const PrepareArgs& a, int64_t b, uint16_t* lds) {
  // pitch 130 halves: the four 16-column runs of a packed row and its block's
  // sixteen rows fall on different banks
  uint16_t(*tile)[130] = reinterpret_cast<uint16_t(*)[130]>(lds);
  const Geometry& g = a.g;
  const int64_t rt = (g.R + 127) / 128;
  const int w = b >= rt * g.nKB;
  b -= w * rt * g.nKB;
  const int64_t kb = b % g.nKB, r0 = (b / g.nKB) * 128;
  const uint8_t* values = w ? a.values[1] : a.values[0];
  const uint8_t* meta = w ? a.meta[1] : a.meta[0];
  uint8_t* mask = w ? a.mask[1] : a.mask[0];
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int it = 0; it < 512 / TH; ++it) {
    const int rl = 16 * (it * (TH / 64) + (threadIdx.x >> 6)) + (lane >> 2), cl = (lane & 3) * 16;
    const int64_t r = r0 + rl;
    uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (r < g.R) {
      const uint32_t keep = expand16(g, values, meta, r, kb * 64 + cl, o);
      if (mask) *reinterpret_cast<uint16_t*>(mask + r * (g.nKB * 8) + kb * 8 + cl / 8) = (uint16_t)keep;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) tile[cl + e][rl] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
  }
  if (!a.wt) return;
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 1024 / TH; ++it) {
    const int q = it * TH + threadIdx.x;
    const int kl = q >> 4, rl = (q & 15) * 8;
    if (kb * 64 + kl < g.K && r0 + rl < a.Rp) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(&tile[kl][rl]);
#pragma unroll
      for (int h = 0; h < PARTS; ++h)
        *reinterpret_cast<v4i*>(a.wt + ((kb * 64 + kl) * PARTS + h) * (2 * a.Rp) + w * a.Rp + r0 + rl) =
            v4i{(int)p[0], (int)p[1], (int)p[2], (int)p[3]};
    }
  }
}

template <int TH, int PARTS>
__device__ __forceinline__ void prepare_tokens(const PrepareArgs& a, int64_t b, uint16_t* lds) {
  uint16_t(*tile)[66] = reinterpret_cast<uint16_t(*)[66]>(lds);
  const int64_t tt = a.Tp / 64, K = a.g.K;
  const int64_t t0 = (b % tt) * 64, k0 = (b / tt) * 64;
#pragma unroll
  for (int it = 0; it < 512 / TH; ++it) {
    const int q = it * TH + threadIdx.x;
    const int tl = q >> 3, kl = (q & 7) * 8;
    const int64_t t = t0 + tl, k = k0 + kl;
    v4i o = {0, 0, 0, 0};
    if (t < a.T && k < K) o = load_piece(a.X + t * a.ldx, k, K);
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[kl + e][tl] = (uint16_t)((uint32_t)o[e >> 1] >> (16 * (e & 1)));
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 512 / TH; ++it) {
    const int q = it * TH + threadIdx.x;
    const int kl = q >> 3, tl = (q & 7) * 8;
    if (k0 + kl < K) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(&tile[kl][tl]);
#pragma unroll
      for (int h = 0; h < PARTS; ++h)
        *reinterpret_cast<v4i*>(a.xt + ((k0 + kl) * PARTS + h) * a.Tp + t0 + tl) =
            v4i{(int)p[0], (int)p[1], (int)p[2], (int)p[3]};
    }
  }
}

template <int WT, int TH, bool P32, int PARTS>
__global__ void __launch_bounds__(TH) glu_prepare_kernel(PrepareArgs a, int64_t n_act, int64_t n_weight) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * PARTS * 64 * 66];
  static_assert(2 * 64 * 66 >= 64 * 130, "the weight tile fits");
  int64_t b = blockIdx.x;
  if (b < n_act) return prepare_dact<WT, TH, P32, PARTS>(a, b, lds);
  b -= n_act;
  if (b < n_weight) return prepare_weight<TH, PARTS>(a, b, lds);
  prepare_tokens<TH, PARTS>(a, b - n_weight, lds);
}

__global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t* X, int64_t ldx, int64_t T, int64_t K,
                                                       uint16_t* Y, int64_t Kp) {
  const int64_t pr = Kp / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < T * pr; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / pr, k = (i - t * pr) * 8;
    const v4i o = k < K ? load_piece(X + t * ldx, k, K) : v4i{0, 0, 0, 0};
    *reinterpret_cast<v4i*>(Y + t * Kp + k) = o;
  }
}

}  // namespace

hipError_t launch_expand_dense(const Geometry& g, const DenseArgs& a, hipStream_t s) {
  const int64_t n = g.nRB * g.nKB;
  hipLaunchKernelGGL(expand_dense_kernel, dim3((unsigned)((n + 3) / 4), 2), dim3(256), 0, s, g, a);
  return hipGetLastError();
}

hipError_t launch_glu_prepare(const PrepareArgs& a, int wdt, hipStream_t s) {
  const int64_t n_act = (a.T + 63) / 64 * (a.Rp / 64);
  const int64_t n_weight = 2 * ((a.g.R + 127) / 128) * a.g.nKB;
  const int64_t n_x = a.xt ? a.Tp / 64 * a.g.nKB : 0;
  const unsigned grid = (unsigned)(n_act + n_weight + n_x);
  // few workgroups: twice the threads each, half the passes one after another
  // (1152 tokens, 428 x 1116: 11.6 us against 14.1; 2048, 11008 x 4096: 135
  // against 120)
  const bool wide = grid < 8u * device_cu_count();
  auto launch = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, s, a, n_act, n_weight);
  };
  auto pick = [&](auto wt, auto p32, auto parts) {
    constexpr int WT = decltype(wt)::value, PARTS = decltype(parts)::value;
    constexpr bool P32 = decltype(p32)::value;
    wide ? launch(glu_prepare_kernel<WT, 512, P32, PARTS>, 512) : launch(glu_prepare_kernel<WT, 256, P32, PARTS>, 256);
  };
  auto pick_type = [&](auto wt) {
    if (!a.p32) return pick(wt, ic<0>(), ic<1>());
    a.parts == 2 ? pick(wt, ic<1>(), ic<2>()) : pick(wt, ic<1>(), ic<1>());
  };
  wdt == NM_F16 ? pick_type(ic<NM_F16>()) : pick_type(ic<NM_BF16>());
  return hipGetLastError();
}

hipError_t launch_pad_rows(const void* X, int64_t ldx, int64_t T, int64_t K, void* Y, int64_t Kp, hipStream_t s) {
  const int64_t n = T * (Kp / 8);
  hipLaunchKernelGGL(pad_rows_kernel, dim3(grid_1d(n, 256)), dim3(256), 0, s,
                     static_cast<const uint16_t*>(X), ldx, T, K, static_cast<uint16_t*>(Y), Kp);
  return hipGetLastError();
}

}  // namespace nm
