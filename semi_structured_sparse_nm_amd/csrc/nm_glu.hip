// Data movement around the gated block's tile products: packed weights
// expanded to dense rows or dense columns, the activation's backward step,
// padded activation rows.  All of them are bound by HBM: every element is
// read once and written once, in 16-byte pieces.
#include "nm_ffn.hpp"

namespace nm {

namespace {

// Eight dense columns c .. c + 7 (c % 8 == 0, c < nKB * 64) of packed row r
// (16-bit weights): two groups of M = 4 or one of M = 8.  o: the eight values
// as four dwords, zeros where pruned; returns the kept bits.
__device__ __forceinline__ uint32_t expand8(const Geometry& g, const uint8_t* values, const uint8_t* meta, int64_t r,
                                            int64_t c, uint32_t (&o)[4]) {
  const int64_t blk = (r >> 4) * g.nKB + (c >> 6);
  const int rr = (int)(r & 15);
  const int cnt = g.N * (8 / g.M);                     // kept values of the eight columns
  const int s0 = (int)(c & 63) / 8 * cnt;
  const uint8_t* v = values + blk * g.vblk + ((int64_t)rr * g.C + s0) * 2;
  if (g.N == g.M) {
    const v4i x = *reinterpret_cast<const v4i*>(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (uint32_t)x[i];
    return 0xFF;
  }
  uint32_t e[4] = {0u, 0u, 0u, 0u};
  if (cnt == 4) {
    const v2i x = *reinterpret_cast<const v2i*>(v);
    e[0] = (uint32_t)x[0];
    e[1] = (uint32_t)x[1];
  } else if (cnt == 2) {
    e[0] = *reinterpret_cast<const uint32_t*>(v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) e[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(v)[i] << (16 * (i & 1));
  }
  const uint32_t* m = reinterpret_cast<const uint32_t*>(meta + blk * g.mblk + (int64_t)rr * g.MR);
  const int bit = s0 * g.w, d = bit >> 5;
  const uint64_t lo = m[d], hi = 4 * d + 4 < g.MR ? m[d + 1] : 0u;
  const uint32_t pos = (uint32_t)((lo | hi << 32) >> (bit & 31));
  uint64_t q0 = 0, q1 = 0;                             // columns 0..3, 4..7
  uint32_t keep = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < cnt) {
      const uint64_t el = (e[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
      uint32_t p = (pos >> (i * g.w)) & ((1u << g.w) - 1u);
      if (g.M == 4 && i >= g.N) p += 4;
      keep |= 1u << p;
      const uint64_t sh = el << (16 * (p & 3));
      if (p < 4) q0 |= sh; else q1 |= sh;
    }
  }
  o[0] = (uint32_t)q0; o[1] = (uint32_t)(q0 >> 32);
  o[2] = (uint32_t)q1; o[3] = (uint32_t)(q1 >> 32);
  return keep;
}

__global__ void __launch_bounds__(256) expand_dense_kernel(Geometry g, const uint8_t* values, const uint8_t* meta,
                                                           uint16_t* dense) {
  const int64_t pr = g.nKB * 8;                        // 8-column pieces per row
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= g.R * pr) return;
  const int64_t r = i / pr, c = (i - r * pr) * 8;
  uint32_t o[4];
  expand8(g, values, meta, r, c, o);
  *reinterpret_cast<v4i*>(dense + r * pr * 8 + c) = v4i{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
}

// One workgroup per 64 rows x 64 columns: the pieces land transposed in LDS
// (row pitch 72 halves: the 16-byte reads stay aligned) and leave as rows of dt.
__global__ void __launch_bounds__(256) expand_transposed_kernel(Geometry g, const uint8_t* values,
                                                                const uint8_t* meta, uint16_t* dt, int64_t ldt,
                                                                uint8_t* mask) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[64][72];
  const int64_t c0 = (int64_t)blockIdx.x * 64, r0 = (int64_t)blockIdx.y * 64;
  for (int q = threadIdx.x; q < 512; q += 256) {
    const int rl = q & 63, cl = (q >> 6) * 8;
    const int64_t r = r0 + rl;
    uint32_t o[4] = {0u, 0u, 0u, 0u};
    if (r < g.R) {
      const uint32_t keep = expand8(g, values, meta, r, c0 + cl, o);
      if (mask) mask[r * (g.nKB * 8) + (c0 + cl) / 8] = (uint8_t)keep;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[cl + e][rl] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
  }
  __syncthreads();
  for (int q = threadIdx.x; q < 512; q += 256) {
    const int kl = q >> 3, rl = (q & 7) * 8;
    if (c0 + kl < g.K)
      *reinterpret_cast<v4i*>(dt + (c0 + kl) * ldt + r0 + rl) = *reinterpret_cast<const v4i*>(&tile[kl][rl]);
  }
}

template <int WT>
__device__ __forceinline__ void load8(const uint16_t* p, int64_t r, int64_t R, bool vec, float (&f)[8]) {
  if (vec && r + 8 <= R) {
    const v4i x = *reinterpret_cast<const v4i*>(p + r);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = from_16<WT>(((uint32_t)x[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = r + i < R ? from_16<WT>(p[r + i]) : 0.f;
  }
}

// One workgroup per 64 tokens x 64 outputs.  dG and dU are rounded to the
// weights' 16-bit type here: they are operands of the matrix instruction in
// both products that follow (half a step each, as any 16-bit operand).
template <int WT>
__global__ void __launch_bounds__(256) glu_dact_kernel(const uint16_t* dH, int64_t lddh, const uint16_t* G,
                                                       const uint16_t* U, int64_t ldp, int64_t T, int64_t R,
                                                       int64_t Rp, uint16_t* d, int64_t ldd, uint16_t* dt, int64_t Tp,
                                                       int act, bool vec) {
  // pitch 66 halves: eight pieces of a row (8 rows apart here) and eight
  // tokens fall on different banks
  __shared__ __attribute__((aligned(16))) uint16_t tile[2][64][66];
  const int64_t t0 = (int64_t)blockIdx.x * 64, r0 = (int64_t)blockIdx.y * 64;
  for (int q = threadIdx.x; q < 512; q += 256) {
    const int tl = q >> 3, rl = (q & 7) * 8;
    const int64_t t = t0 + tl, r = r0 + rl;
    uint32_t og[4] = {0u, 0u, 0u, 0u}, ou[4] = {0u, 0u, 0u, 0u};
    if (t < T && r < R) {
      float h[8], g[8], u[8];
      load8<WT>(dH + t * lddh, r, R, vec, h);
      load8<WT>(G + t * ldp, r, R, vec, g);
      load8<WT>(U + t * ldp, r, R, vec, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float dg[2], du[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y, dy;
          glu_act_slope(act, g[2 * i + e], y, dy);
          const bool in = r + 2 * i + e < R;
          dg[e] = in ? h[2 * i + e] * u[2 * i + e] * dy : 0.f;
          du[e] = in ? h[2 * i + e] * y : 0.f;
        }
        og[i] = pack_16x2<WT>(dg[0], dg[1]);
        ou[i] = pack_16x2<WT>(du[0], du[1]);
      }
    }
    if (d && t < T) {
      *reinterpret_cast<v4i*>(d + t * ldd + r) = v4i{(int)og[0], (int)og[1], (int)og[2], (int)og[3]};
      *reinterpret_cast<v4i*>(d + t * ldd + Rp + r) = v4i{(int)ou[0], (int)ou[1], (int)ou[2], (int)ou[3]};
    }
    if (dt) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        tile[0][rl + e][tl] = (uint16_t)(og[e >> 1] >> (16 * (e & 1)));
        tile[1][rl + e][tl] = (uint16_t)(ou[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
  if (!dt) return;
  __syncthreads();
  for (int q = threadIdx.x; q < 1024; q += 256) {
    const int w = q >> 9, rl = (q >> 3) & 63, tl = (q & 7) * 8;
    if (r0 + rl < R) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(&tile[w][rl][tl]);
      *reinterpret_cast<v4i*>(dt + ((int64_t)w * R + r0 + rl) * Tp + t0 + tl) =
          v4i{(int)p[0], (int)p[1], (int)p[2], (int)p[3]};
    }
  }
}

__global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t* X, int64_t ldx, int64_t T, int64_t K,
                                                       uint16_t* Y, int64_t Kp) {
  const int64_t pr = Kp / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= T * pr) return;
  const int64_t t = i / pr, k = (i - t * pr) * 8;
  uint32_t o[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (k + e < K) o[e >> 1] |= (uint32_t)X[t * ldx + k + e] << (16 * (e & 1));
  *reinterpret_cast<v4i*>(Y + t * Kp + k) = v4i{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
}

}  // namespace

hipError_t launch_expand_dense(const Geometry& g, const uint8_t* values, const uint8_t* meta, uint16_t* dense,
                               hipStream_t s) {
  const int64_t n = g.R * g.nKB * 8;
  hipLaunchKernelGGL(expand_dense_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, g, values, meta, dense);
  return hipGetLastError();
}

hipError_t launch_expand_transposed(const Geometry& g, const uint8_t* values, const uint8_t* meta, uint16_t* dt,
                                    int64_t ldt, uint8_t* mask, hipStream_t s) {
  hipLaunchKernelGGL(expand_transposed_kernel, dim3((unsigned)g.nKB, (unsigned)((g.R + 63) / 64)), dim3(256), 0, s, g,
                     values, meta, dt, ldt, mask);
  return hipGetLastError();
}

hipError_t launch_glu_dact(const void* dH, int64_t ldh, const void* G, const void* U, int64_t ldp, int64_t T,
                           int64_t R, int64_t Rp, void* d, int64_t ldd, void* dt, int64_t Tp, int act, int wdt,
                           hipStream_t s) {
  const bool vec = ldh % 8 == 0 && ldp % 8 == 0 && (uintptr_t)dH % 16 == 0 && (uintptr_t)G % 16 == 0 &&
                   (uintptr_t)U % 16 == 0;
  const dim3 grid((unsigned)((T + 63) / 64), (unsigned)(Rp / 64));
  auto h = static_cast<const uint16_t*>(dH);
  auto g = static_cast<const uint16_t*>(G);
  auto u = static_cast<const uint16_t*>(U);
  if (wdt == NM_F16)
    hipLaunchKernelGGL((glu_dact_kernel<NM_F16>), grid, dim3(256), 0, s, h, ldh, g, u, ldp, T, R, Rp,
                       static_cast<uint16_t*>(d), ldd, static_cast<uint16_t*>(dt), Tp, act, vec);
  else
    hipLaunchKernelGGL((glu_dact_kernel<NM_BF16>), grid, dim3(256), 0, s, h, ldh, g, u, ldp, T, R, Rp,
                       static_cast<uint16_t*>(d), ldd, static_cast<uint16_t*>(dt), Tp, act, vec);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const void* X, int64_t ldx, int64_t T, int64_t K, void* Y, int64_t Kp, hipStream_t s) {
  const int64_t n = T * (Kp / 8);
  hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                     static_cast<const uint16_t*>(X), ldx, T, K, static_cast<uint16_t*>(Y), Kp);
  return hipGetLastError();
}

}  // namespace nm
