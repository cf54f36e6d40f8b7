// Products of grouped rows, a middle number of rows an expert: a workgroup
// multiplies 64 or 128 rows of one expert with 256 outputs.
//
// Weights come packed from HBM straight to the registers of the one wave that
// has their 32 outputs, two slabs ahead, and are expanded there once for all the
// rows (2:4 go to the sparse matrix instruction as they are): neither a dense
// copy of the weights nor their way through LDS exists.  The rows are shared
// through LDS: 128 bytes of each a slab, loaded to registers two slabs ahead and
// written a slab ahead, one barrier a slab.  Every wave reads all of them, so LDS
// is read for 1024 cycles a slab of 128 rows, as long as the dense products take.
#pragma once

#include <algorithm>

#include "nm_rows_frag.hpp"
#include "nm_tile_common.hpp"

namespace nm {

namespace {

constexpr int kWideWaves = 8;
constexpr int kWideOut = 32 * kWideWaves;              // outputs of a workgroup

template <int WT, int N, int M, int TM>
__global__ void __launch_bounds__(kWideWaves * 64) rows_wide_kernel(RowsArgs a, int nt) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = kWideWaves, BM = 16 * TM, NP = BM * 8 / (NW * 64);
  typedef RowsFrag<WT, N, M> Frag;
  typedef acc_of<WT> Acc;
  typedef typename Frag::Entry Entry;
  constexpr int XB = WT == NM_I8 ? 1 : 2;
  __shared__ __attribute__((aligned(1024))) uint8_t rows[2][BM * 128];
  __shared__ __attribute__((aligned(16))) Entry table[Frag::TABLE ? 256 : 1];
  fill_table<Frag, XB>(table);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lg = lane >> 4;

  auto zero_rest = [&]() {
    if (!a.zero_rest || !a.rows.at) return;
    int first, last;
    rows_taken(a.rows, first, last);
    const int rest = first + (int)a.rows.T - last;
    for (int i = blockIdx.x; i < rest; i += gridDim.x) {
      const int64_t o = (int64_t)(i < first ? i : last + (i - first)) * a.ldy;
      for (int64_t n = threadIdx.x; n < a.g.R; n += NW * 64) {
        if (a.ydt == NM_F32) static_cast<float*>(a.Y)[o + n] = 0.f;
        else static_cast<uint16_t*>(a.Y)[o + n] = 0;
      }
    }
  };
  // XCD x takes a contiguous run of the items, an expert's units of one column
  // tile next to each other: they share its weights in the XCD's L2
  const int total = count_units<BM>(a.rows) * nt, per = (total + 7) / 8;
  const int j8 = blockIdx.x >> 3, L = (blockIdx.x & 7) * per + j8;
  if (j8 >= per || L >= total) return zero_rest();
  const RowUnit ru = find_unit<BM>(a.rows, L, nt);
  const int n = ru.n;
  const int nKB = (int)a.g.nKB, last = nKB - 1;
  const int KX = (int)a.g.K;
  // the wave's row blocks (past the last: that one again, its results are not stored)
  const uint8_t* values[2];
  const uint8_t* meta[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t b = (ru.e * a.g.nRB + min((int64_t)n * (kWideOut / 16) + 2 * wave + i, a.g.nRB - 1)) * nKB;
    values[i] = a.values + b * Frag::VBLK;
    meta[i] = a.meta + b * Frag::MBLK;
  }

  // rows: piece q % 8 (16 bytes) of row q / 8 (past the expert's last: that one)
  const int piece = threadIdx.x & 7, row0 = threadIdx.x >> 3;
  const uint8_t* x0 = static_cast<const uint8_t*>(a.X) + (int64_t)ru.row * (a.ldx * XB);
  const int rlast = ru.end - 1 - ru.row;
  uint32_t xoff[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) xoff[i] = (uint32_t)min(row0 + NW * 8 * i, rlast) * (uint32_t)(a.ldx * XB);
  struct Rows {
    v4i x[NP];
  };
  auto load_rows = [&](Rows& r, int s) __attribute__((always_inline)) {
    s = min(s, last);
    // (a piece past the row's end: the slab's first one, so that no branch splits
    // the loads; store_rows makes it zeros)
    const uint32_t p = s * Frag::SLAB + 16 / XB * piece < KX ? 16 * piece : 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) r.x[i] = load16(x0 + s * 128 + (xoff[i] + p));
  };
  const int put = row0 * 128 + 16 * (piece ^ (row0 & 7));
  // (8-bit rows are whole slabs)
  auto store_rows = [&](const Rows& r, int s, int p) __attribute__((always_inline)) {
    const bool in = WT == NM_I8 || s * Frag::SLAB + 16 / XB * piece < KX;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      *reinterpret_cast<v4i*>(rows[p] + put + NW * 1024 * i) = in ? r.x[i] : v4i{0, 0, 0, 0};
  };
  struct Blocks {
    Frag f[2];
  };
  auto load_blocks = [&](Blocks& b, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      b.f[i].load(values[i] + min(s, last) * Frag::VBLK, meta[i] + min(s, last) * Frag::MBLK, li, lg);
  };
  const int get0 = li * 128 + 16 * (Frag::kpiece(0, lg) ^ (li & 7));
  const int get1 = li * 128 + 16 * (Frag::kpiece(1, lg) ^ (li & 7));
  Acc acc[2][TM];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = Acc{0, 0, 0, 0};

  // slab s is multiplied from rows[P]; r1 holds the rows of slab s + 1, r0 those
  // of s + 2, b the blocks of s
  auto step = [&](int s, auto pc, Rows& r1, Blocks& b) __attribute__((always_inline)) {
    constexpr int P = decltype(pc)::value;
    store_rows(r1, s + 1, P ^ 1);
    load_rows(r1, s + 3);
    // (each row tile is read from LDS before the products of the one in front of it)
    v4i x0[2], x1[2];
    auto read_tile = [&](int j) __attribute__((always_inline)) {
      x0[j & 1] = *reinterpret_cast<const v4i*>(rows[P] + 2048 * j + get0);
      x1[j & 1] = *reinterpret_cast<const v4i*>(rows[P] + 2048 * j + get1);
    };
    read_tile(0);
    v4i a0[2], a1[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      b.f[i].ready(lg, a0[i], a1[i], table);
      // (6:8 and 7:8 of 8 bits: one block's temporaries at a time, or two workgroups
      // do not fit a compute unit's registers)
      if (WT == NM_I8 && Frag::TABLE && N > 5) __builtin_amdgcn_sched_barrier(0);
    }
    load_blocks(b, s + 2);
    __builtin_amdgcn_sched_barrier(0);                  // (the loads are not sunk behind the products)
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      if (j + 1 < TM) read_tile(j + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[i][j] = rows_mul<WT, Frag::SPARSE>(a0[i], a1[i], x0[j & 1], x1[j & 1], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt(63, 0));         // slab s + 1 is written, slab s read
    barrier_nofence();
  };
  Rows r0, r1;
  Blocks b0, b1;
  // (in the loop's order: its waits count the loads behind the awaited ones)
  load_rows(r0, 0);
  __builtin_amdgcn_sched_barrier(0);
  load_rows(r1, 1);
  load_blocks(b0, 0);
  __builtin_amdgcn_sched_barrier(0);
  store_rows(r0, 0, 0);
  load_rows(r0, 2);
  __builtin_amdgcn_sched_barrier(0);
  load_blocks(b1, 1);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(waitcnt(63, 0));
  barrier_nofence();
  // (one way out of the loop: with two the sums are copied at every step)
  int s = 0;
  for (; s + 1 < nKB; s += 2) {
    step(s, ic<0>(), r1, b0);
    step(s + 1, ic<1>(), r0, b1);
  }
  if (s < nKB) step(s, ic<0>(), r1, b0);

  const int64_t n0 = (int64_t)n * kWideOut + 32 * wave;
  if constexpr (WT == NM_I8) {
    const float* sw = a.wscale + ru.e * a.g.R;
    const float* bias = a.bias ? a.bias + ru.e * a.g.R : nullptr;
    if (a.ydt == NM_F16)
      tile_rows_i8<NM_F16, TM, 2>(a.Y, a.ldy, ru.end, a.g.R, a.xscale, sw, bias, a.act, ru.row, n0, acc);
    else if (a.ydt == NM_BF16)
      tile_rows_i8<NM_BF16, TM, 2>(a.Y, a.ldy, ru.end, a.g.R, a.xscale, sw, bias, a.act, ru.row, n0, acc);
    else
      tile_rows_i8<NM_F32, TM, 2>(a.Y, a.ldy, ru.end, a.g.R, a.xscale, sw, bias, a.act, ru.row, n0, acc);
  } else {
    tile_rows<false, WT, TM, 2>(a.Y, a.ldy, ru.end, a.g.R, nullptr, NM_ACT_NONE, nullptr, 0, ru.row, n0, acc);
  }
  zero_rest();
#endif
}

template <int WT, int N, int M>
hipError_t launch_rows_wide_nm(const RowsArgs& a, int tm, hipStream_t s) {
  const int nt = (int)((a.g.R + kWideOut - 1) / kWideOut);
  const int64_t most = units_most(a.rows.T, a.rows.E, 16 * tm) * nt;
  const dim3 grid((unsigned)((most + 7) / 8 * 8)), block(kWideWaves * 64);
  if (tm == 4)
    hipLaunchKernelGGL((rows_wide_kernel<WT, N, M, 4>), grid, block, 0, s, a, nt);
  else
    hipLaunchKernelGGL((rows_wide_kernel<WT, N, M, 8>), grid, block, 0, s, a, nt);
  return hipGetLastError();
}

template <int WT>
hipError_t launch_rows_wide_wt(const RowsArgs& a, int tm, hipStream_t s) {
  switch (a.g.M * 16 + a.g.N) {
    case 4 * 16 + 1: return launch_rows_wide_nm<WT, 1, 4>(a, tm, s);
    case 4 * 16 + 2: return launch_rows_wide_nm<WT, 2, 4>(a, tm, s);
    case 4 * 16 + 3: return launch_rows_wide_nm<WT, 3, 4>(a, tm, s);
    case 4 * 16 + 4: return launch_rows_wide_nm<WT, 4, 4>(a, tm, s);
    case 8 * 16 + 1: return launch_rows_wide_nm<WT, 1, 8>(a, tm, s);
    case 8 * 16 + 2: return launch_rows_wide_nm<WT, 2, 8>(a, tm, s);
    case 8 * 16 + 3: return launch_rows_wide_nm<WT, 3, 8>(a, tm, s);
    case 8 * 16 + 4: return launch_rows_wide_nm<WT, 4, 8>(a, tm, s);
    case 8 * 16 + 5: return launch_rows_wide_nm<WT, 5, 8>(a, tm, s);
    case 8 * 16 + 6: return launch_rows_wide_nm<WT, 6, 8>(a, tm, s);
    case 8 * 16 + 7: return launch_rows_wide_nm<WT, 7, 8>(a, tm, s);
    case 8 * 16 + 8: return launch_rows_wide_nm<WT, 8, 8>(a, tm, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

}  // namespace nm
