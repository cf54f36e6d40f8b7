// Dense columns of a packed row, any N:M chosen at run time: for the kernels
// that write dense copies or transposes of packed weights.
#pragma once

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
  } else if (cnt % 2 == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (2 * i < cnt) e[i] = reinterpret_cast<const uint32_t*>(v)[i];
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

// Sixteen dense columns c .. c + 15 (c % 16 == 0): one 16-byte piece of the
// packed row where four of eight are kept.
__device__ __forceinline__ uint32_t expand16(const Geometry& g, const uint8_t* values, const uint8_t* meta, int64_t r,
                                             int64_t c, uint32_t (&o)[8]) {
  uint32_t h[4];
  uint32_t keep = expand8(g, values, meta, r, c, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = h[i];
  keep |= expand8(g, values, meta, r, c + 8, h) << 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[4 + i] = h[i];
  return keep;
}

// Sixteen dense columns c .. c + 15 (c % 16 == 0) of packed row r of 8-bit
// weights: four groups of M = 4 or two of M = 8.  o: the values as four dwords.
template <int M>
__device__ __forceinline__ v4i expand16_i8(const Geometry& g, const uint8_t* values, const uint8_t* meta, int64_t blk,
                                           int rr, int piece) {
  const int cnt = g.N * (16 / M);                      // kept values of the sixteen columns
  const uint8_t* v = values + blk * g.vblk + rr * g.C + piece * cnt;
  if (g.N == M) return *reinterpret_cast<const v4i*>(v);
  // (cnt is even: the run starts at any even byte)
  uint32_t e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(v) + 2 * i;
    e[i] = 4 * i < cnt ? h[0] : 0u;
    if (4 * i + 2 < cnt) e[i] |= (uint32_t)h[1] << 16;
  }
  const uint32_t* m = reinterpret_cast<const uint32_t*>(meta + blk * g.mblk + (int64_t)rr * g.MR);
  const int bit = piece * cnt * g.w, d = bit >> 5, last = g.MR / 4 - 1;
  // up to 42 bits of positions from any bit: three dwords, as two from bit 0
  const uint32_t w0 = m[d], w1 = m[min(d + 1, last)], w2 = m[min(d + 2, last)];
  const uint32_t p0 = __builtin_amdgcn_alignbit(w1, w0, bit & 31), p1 = __builtin_amdgcn_alignbit(w2, w1, bit & 31);
  uint32_t o[4] = {0u, 0u, 0u, 0u};
  constexpr int W = M == 4 ? 2 : 3;
#pragma unroll
  for (int q = 0; q < 16 / M; ++q) {
    const int s = q * g.N * W;                         // the group's first bit
    const uint32_t pos = s >= 32 ? p1 >> (s - 32) : __builtin_amdgcn_alignbit(p1, p0, s);
#pragma unroll
    for (int j = 0; j < M; ++j) {
      if (j < g.N) {
        const int i = q * g.N + j;                     // i < 16
        const uint32_t word = i < 4 ? e[0] : i < 8 ? e[1] : i < 12 ? e[2] : e[3];
        const uint32_t p = pos >> (W * j) & (M - 1);
        const uint32_t x = (word >> (8 * (i & 3)) & 0xFFu) << (8 * (p & 3));
        if (M == 4) {
          o[q] |= x;
        } else {
          o[2 * (q & 1)] |= p < 4 ? x : 0u;
          o[2 * (q & 1) + 1] |= p < 4 ? 0u : x;
        }
      }
    }
  }
  return v4i{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
}

}  // namespace

}  // namespace nm
