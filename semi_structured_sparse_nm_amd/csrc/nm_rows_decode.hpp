// Products of grouped rows, few rows an expert: each expert's packed weight is
// streamed once from HBM for every unit of 16 NT of its rows.
//
//   Y[s][r] = act(sum_k X[s][k] W_e[r][k] (x scale[s] x wscale[e][r]) + bias[e][r])
//
// With so few rows the bound is the packed weights' bytes.  A workgroup owns
// one 16-row block of one expert's weight and one unit of its rows (found from
// the offsets by the workgroup itself: the host does not know them, and starts
// as many as there could be), or a few row blocks where K is short; the waves of
// a row block take its blocks along K in turn, straight to registers, U blocks in
// flight per wave.  2:4 windows go to the
// sparse matrix instruction as they are; other patterns are expanded in
// registers for the dense one.  Activations come from the caches, 128 bytes of
// eight rows a load, and change to the instruction's order in the wave's own
// LDS; the waves' sums meet in LDS, added in wave order.  (The gated block's
// streamed kernel with one weight; why each of this is so is measured there.)
//
// 8-bit elements: sums are exact in 32-bit integers, converted once, then
// multiplied by the row's scale and the channel's in binary32 (two roundings,
// far below the output's).
#pragma once

#include <algorithm>

#include "nm_i8_device.hpp"
#include "nm_rows_frag.hpp"

namespace nm {

namespace {

#if defined(__HIP_DEVICE_COMPILE__)
// Zeros in `n` outputs from r0 on of every units-th of the rows that belong to
// no expert.  (Behind the product: it waits for the offsets once more.)
__device__ __forceinline__ void zero_rows_of_none(const RowsArgs& a, int64_t r0, int n, int unit, int units) {
  if (!a.zero_rest) return;
  int first, last;
  rows_taken(a.rows, first, last);
  const int rest = first + (int)a.rows.T - last;
  const int64_t r1 = min(r0 + n, a.g.R);
  for (int i = unit + units * (threadIdx.x >> 4); i < rest; i += units * (kGluWaves * 4)) {
    const int64_t t = i < first ? i : last + (i - first);
    for (int64_t r = r0 + (threadIdx.x & 15); r < r1; r += 16) {
      if (a.ydt == NM_F32) static_cast<float*>(a.Y)[t * a.ldy + r] = 0.f;
      else static_cast<uint16_t*>(a.Y)[t * a.ldy + r] = 0;
    }
  }
}
#endif

// SHORT: 16-bit rows whose K is no multiple of eight (groups of four only);
// 8-bit rows are whole pieces.  XQ: NM_I8, or the type of rows that the
// workgroup quantises itself, first their maxima, then their elements into LDS,
// while its first blocks are on their way.  GROUPED: rows with offsets; else one
// expert has them all.
template <int WT, int N, int M, int NT, bool SHORT, int XQ, bool GROUPED>
__global__ void __launch_bounds__(kGluWaves * 64) rows_decode_kernel(RowsArgs a, int units, int ks) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = kGluWaves;
  constexpr bool QX = XQ != NM_I8;
  constexpr int U = QX ? 8 : NT == 4 ? 2 : 4;
  typedef RowsFrag<WT, N, M> Frag;
  typedef acc_of<WT> Acc;
  typedef typename Frag::Entry Entry;
  constexpr int XB = WT == NM_I8 ? 1 : 2;              // bytes of an activation
  // a wave's activations of one block, then its sums
  __shared__ __attribute__((aligned(16))) v4f red[NW][2 * NT][64];
  __shared__ __attribute__((aligned(16))) Entry table[Frag::TABLE ? 256 : 1];
  __shared__ uint32_t top[QX ? 16 : 1][QX ? NW : 1];
  __shared__ float xscale[WT == NM_I8 ? 16 * NT : 1];
  extern __shared__ __attribute__((aligned(16))) uint8_t xq[];   // QX: rows of Kp + 16 bytes
  fill_table<Frag, XB>(table);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lg = lane >> 4;
  // ks waves share a row block along K, the workgroup has NW / ks row blocks;
  // workgroups 8 apart (neighbours on their XCD) take the units of the same ones
  const int lks = 31 - __builtin_clz(ks), nblk = NW >> lks;
  const int b = blockIdx.x >> 3, q8 = __builtin_amdgcn_readfirstlane(b / units);
  const int64_t rb0 = (int64_t)(q8 * 8 + (blockIdx.x & 7)) * nblk;
  const int unit = b - q8 * units;
  if (rb0 >= a.g.nRB) return;
  RowUnit ru = {0, unit * (16 * NT), 0, (int)a.rows.T, 0};
  if constexpr (GROUPED) ru = find_unit<16 * NT>(a.rows, unit);
  if (ru.e < 0) {
    if constexpr (GROUPED) zero_rows_of_none(a, rb0 * 16, 16 * nblk, unit, units);
    return;
  }
  const int nrows = min(ru.end - ru.row, 16 * NT);
  const int nKB = (int)a.g.nKB;
  const int KX = (int)a.g.K;                           // columns of a row that may be read
  // the wave's row block (past the last: that one again, its results are not stored)
  const int64_t blk0 = (ru.e * a.g.nRB + min(rb0 + (wave >> lks), a.g.nRB - 1)) * nKB;
  const uint8_t* values = a.values + blk0 * Frag::VBLK;
  const uint8_t* meta = a.meta + blk0 * Frag::MBLK;
  const int k0 = wave & (ks - 1);

  // What the end needs, asked for first (a wave's loads come back in order): the
  // thread's output channel is the same in every step there.
  float sw = 0.f, bias = 0.f, sx = 0.f;
  if constexpr (WT == NM_I8) {
    const int64_t r = (rb0 + ((threadIdx.x >> 4) & (nblk - 1))) * 16 + (threadIdx.x & 15);
    if (r < a.g.R) {
      sw = a.wscale[ru.e * a.g.R + r];
      if (a.bias) bias = a.bias[ru.e * a.g.R + r];
    }
    if (!QX && threadIdx.x < 16 * NT) sx = a.xscale[min(ru.row + (int)threadIdx.x, ru.end - 1)];
  }
  const int pitch = nKB * 128 + 16;
  // QX: the first PR pieces that the thread quantises, asked for before the
  // weights: of row i / pr the piece threadIdx.x + 512 (i % pr).  It reads all of
  // them twice, later ones the second time from the caches.
  constexpr int PR = 4;
  constexpr int EB = XQ == NM_F32 ? 4 : 2;
  typedef Eight<QX ? XQ : NM_F16> Piece;
  const int pr = (nKB * 16 + NW * 64 - 1) / (NW * 64);
  Piece held[QX ? PR : 1];
  auto load_piece_of = [&](int r, int i, Piece& e) __attribute__((always_inline)) {
    const int k = 8 * (threadIdx.x + NW * 64 * i);
    e.clear();
    if (k < KX) e.load(static_cast<const uint8_t*>(a.X) + (int64_t)(ru.row + r) * a.ldx * EB, k, KX);
  };
  if constexpr (QX) {
    int r = 0, c = 0;
#pragma unroll
    for (int i = 0; i < PR; ++i) {
      held[i].clear();
      if (r < nrows) load_piece_of(r, c, held[i]);
      if (++c == pr) ++r, c = 0;
    }
  }

  Frag f[U];
  auto load_blocks = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int kb = b0 + ks * i;
      if (i == 0 || kb < nKB) {
        const int at = __builtin_amdgcn_readfirstlane(min(kb, nKB - 1));
        f[i].load(values + at * Frag::VBLK, meta + at * Frag::MBLK, li, lg);
      }
    }
  };
  load_blocks(k0);

  if constexpr (QX) {
    // the rows' maxima, each wave's part; then the elements
    auto every_piece = [&](auto&& g) __attribute__((always_inline)) {
      int r = 0, c = 0;
#pragma unroll
      for (int i = 0; i < PR; ++i) {
        if (r < nrows) g(r, c, held[i]);
        if (++c == pr) ++r, c = 0;
      }
      for (; r < nrows;) {
        Piece e;
        load_piece_of(r, c, e);
        g(r, c, e);
        if (++c == pr) ++r, c = 0;
      }
    };
    uint32_t m = 0;
    every_piece([&](int r, int c, const Piece& e) __attribute__((always_inline)) {
      m = max(c ? m : 0u, e.top());
      if (c == pr - 1) {
        const uint32_t w = wave_max(m);
        if (lane == 0) top[r][wave] = w;
      }
    });
    __syncthreads();
    every_piece([&](int r, int c, const Piece& e) __attribute__((always_inline)) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) m = max(m, top[r][w]);
      const float s = scale_of<XQ>(m);
      if (threadIdx.x == 0) xscale[r] = s;
      const int k = 8 * (threadIdx.x + NW * 64 * c);
      if (k < nKB * 128)
        *reinterpret_cast<v2i*>(xq + r * pitch + k) = s == s ? codes_of<XQ>(e, s, __builtin_amdgcn_rcpf(s)) : v2i{0, 0};
    });
    __syncthreads();
  }

  // activations: load h of row tile j brings rows 8 h .. 8 h + 7 of it, lane l
  // piece l % 8 (16 bytes) of row 8 h + l / 8; rows past the expert's last
  // repeat it (their results are not stored).  A 16-bit row's last piece may
  // hold fewer than eight columns: it is read as the row's last eight and
  // shifted, so nothing past the row is read.
  const int piece = lane & 7;
  const int short_by = SHORT ? 8 - (KX & 7) : 0;
  const bool tall = nrows > 8;                         // (else no second half of the one tile)
  const uint8_t* xr[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xr[j][h] = static_cast<const uint8_t*>(a.X) +
                 (int64_t)min(ru.row + 16 * j + 8 * h + (lane >> 3), ru.end - 1) * (a.ldx * XB) + 16 * piece;
  uint8_t* const xs = reinterpret_cast<uint8_t*>(&red[wave][0][0]);
  const int put = (lane >> 3) * 128 + 16 * (piece ^ (lane >> 3));
  const int get0 = li * 128 + 16 * (Frag::kpiece(0, lg) ^ (li & 7));
  const int get1 = li * 128 + 16 * (Frag::kpiece(1, lg) ^ (li & 7));
  const uint8_t* const xqr = xq + min(li, nrows - 1) * pitch;
  Acc acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = Acc{0, 0, 0, 0};

  for (int b0 = k0;;) {
    if constexpr (QX) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int kb = b0 + ks * i;
        if (kb < nKB) {
          const v4i x0 = *reinterpret_cast<const v4i*>(xqr + kb * 128 + 16 * Frag::kpiece(0, lg));
          const v4i x1 = *reinterpret_cast<const v4i*>(xqr + kb * 128 + 16 * Frag::kpiece(1, lg));
          v4i a0, a1;
          f[i].ready(lg, a0, a1, table);
          acc[0] = rows_mul<WT, Frag::SPARSE>(a0, a1, x0, x1, acc[0]);
        }
      }
    } else {
      v4i x[U][NT][2];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int kb = b0 + ks * i;
        if (i == 0 || kb < nKB) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k = kb * Frag::SLAB + 16 / XB * piece;
              x[i][j][h] = v4i{0, 0, 0, 0};
              if ((NT > 1 || h == 0 || tall) && k < KX)
                x[i][j][h] = load16(xr[j][h] + kb * 128 - (SHORT && k + 8 > KX ? 2 * short_by : 0));
            }
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int kb = b0 + ks * i;
        if (kb < nKB) {
          if (SHORT && kb == nKB - 1) {
            const bool last = kb * Frag::SLAB + 8 * piece + 8 > KX;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) x[i][j][h] = last ? shift_out(x[i][j][h], short_by) : x[i][j][h];
          }
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) *reinterpret_cast<v4i*>(xs + 2048 * j + 1024 * h + put) = x[i][j][h];
          __builtin_amdgcn_wave_barrier();
          v4i a0, a1;
          f[i].ready(lg, a0, a1, table);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const v4i x0 = *reinterpret_cast<const v4i*>(xs + 2048 * j + get0);
            const v4i x1 = *reinterpret_cast<const v4i*>(xs + 2048 * j + get1);
            acc[j] = rows_mul<WT, Frag::SPARSE>(a0, a1, x0, x1, acc[j]);
          }
          __builtin_amdgcn_wave_barrier();
        }
      }
    }
    b0 += ks * U;
    if (b0 >= nKB) break;
    load_blocks(b0);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) red[wave][2 * j][lane] = __builtin_bit_cast(v4f, acc[j]);
  if (WT == NM_I8 && !QX && threadIdx.x < 16 * NT) xscale[threadIdx.x] = sx;
  __syncthreads();
  // 16 NT rows x 16 outputs of each row block: the sums of its ks waves
  const int per = 16 * nblk;
  for (int q = threadIdx.x; q < 16 * NT * per; q += NW * 64) {
    const int row = q & 15, blk = (q >> 4) & (nblk - 1), tok = q >> (4 + 3 - lks);
    const int ln = 16 * (row >> 2) + (tok & 15), v = row & 3, j = tok >> 4;
    const int64_t r = (rb0 + blk) * 16 + row, t = ru.row + tok;
    if (r >= a.g.R || t >= ru.end) continue;
    float y;
    if constexpr (WT == NM_I8) {
      int sum = 0;
      // (all eight reads at once: of no more than ks waves)
#pragma unroll
      for (int w = 0; w < NW; ++w)
        sum += reinterpret_cast<const int*>(&red[(blk << lks) + (w & (ks - 1))][2 * j][ln])[v] & (w < ks ? -1 : 0);
      y = (float)sum * xscale[tok] * sw;
      if (a.bias) y += bias;
      if (a.act == NM_ACT_GELU) y = gelu_f32(y);
    } else {
      y = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float part = reinterpret_cast<const float*>(&red[(blk << lks) + (w & (ks - 1))][2 * j][ln])[v];
        y += w < ks ? part : 0.f;
      }
    }
    const int64_t o = t * a.ldy + r;
    if constexpr (WT == NM_I8) {
      if (a.ydt == NM_F32) static_cast<float*>(a.Y)[o] = y;
      else if (a.ydt == NM_F16) static_cast<uint16_t*>(a.Y)[o] = (uint16_t)pack_16x2<NM_F16>(y, 0.f);
      else static_cast<uint16_t*>(a.Y)[o] = (uint16_t)pack_16x2<NM_BF16>(y, 0.f);
    } else {
      static_cast<uint16_t*>(a.Y)[o] = (uint16_t)pack_16x2<WT>(y, 0.f);
    }
  }
  if constexpr (GROUPED) zero_rows_of_none(a, rb0 * 16, 16 * nblk, unit, units);
#endif
}

template <int WT, int N, int M, bool SHORT>
hipError_t launch_rows_decode_rows(const RowsArgs& a, hipStream_t s) {
  const int64_t T = a.rows.T, E = a.rows.E;
  int nt, ks;
  int64_t workgroups;
  rows_decode_plan(a.g, T, E, &nt, &ks, &workgroups);
  const int64_t units = units_most(T, E, 16 * nt);
  const dim3 grid((unsigned)workgroups), block(kGluWaves * 64);
  auto go = [&](auto kernel, int64_t lds) {
    hipLaunchKernelGGL(kernel, grid, block, (unsigned)lds, s, a, (int)units, ks);
    return hipGetLastError();
  };
  auto pick = [&](auto grouped) {
    constexpr bool G = decltype(grouped)::value;
    if constexpr (WT == NM_I8) {
      const int64_t lds = T * (a.g.nKB * 128 + 16);
      if (a.xdt == NM_F16) return go(rows_decode_kernel<WT, N, M, 1, SHORT, NM_F16, G>, lds);
      if (a.xdt == NM_BF16) return go(rows_decode_kernel<WT, N, M, 1, SHORT, NM_BF16, G>, lds);
      if (a.xdt == NM_F32) return go(rows_decode_kernel<WT, N, M, 1, SHORT, NM_F32, G>, lds);
    }
    if (nt == 1) return go(rows_decode_kernel<WT, N, M, 1, SHORT, NM_I8, G>, 0);
    if (nt == 2) return go(rows_decode_kernel<WT, N, M, 2, SHORT, NM_I8, G>, 0);
    return go(rows_decode_kernel<WT, N, M, 4, SHORT, NM_I8, G>, 0);
  };
  // (only 8-bit products come without offsets)
  if constexpr (WT == NM_I8)
    if (!a.rows.at) return pick(ic<0>());
  return pick(ic<1>());
}

template <int WT, int N, int M>
hipError_t launch_rows_decode_nm(const RowsArgs& a, hipStream_t s) {
  if constexpr (M == 4 && WT != NM_I8)
    if (a.g.K % 8) return launch_rows_decode_rows<WT, N, M, true>(a, s);
  return launch_rows_decode_rows<WT, N, M, false>(a, s);
}

template <int WT>
hipError_t launch_rows_decode_wt(const RowsArgs& a, hipStream_t s) {
  switch (a.g.M * 16 + a.g.N) {
    case 4 * 16 + 1: return launch_rows_decode_nm<WT, 1, 4>(a, s);
    case 4 * 16 + 2: return launch_rows_decode_nm<WT, 2, 4>(a, s);
    case 4 * 16 + 3: return launch_rows_decode_nm<WT, 3, 4>(a, s);
    case 4 * 16 + 4: return launch_rows_decode_nm<WT, 4, 4>(a, s);
    case 8 * 16 + 1: return launch_rows_decode_nm<WT, 1, 8>(a, s);
    case 8 * 16 + 2: return launch_rows_decode_nm<WT, 2, 8>(a, s);
    case 8 * 16 + 3: return launch_rows_decode_nm<WT, 3, 8>(a, s);
    case 8 * 16 + 4: return launch_rows_decode_nm<WT, 4, 8>(a, s);
    case 8 * 16 + 5: return launch_rows_decode_nm<WT, 5, 8>(a, s);
    case 8 * 16 + 6: return launch_rows_decode_nm<WT, 6, 8>(a, s);
    case 8 * 16 + 7: return launch_rows_decode_nm<WT, 7, 8>(a, s);
    case 8 * 16 + 8: return launch_rows_decode_nm<WT, 8, 8>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

}  // namespace nm
