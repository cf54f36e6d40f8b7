// Tile product of the feed-forward operators on the dense matrix cores:
//
//   C[m][n] = sum_k A[m][k] B[n][k]       (both operands reduction-contiguous)
//
// fp16 / bf16 operands on v_mfma_f32_16x16x32, microscaled 4-bit operands on
// v_mfma_scale_f32_16x16x128 (its E8M0 scales applied by the instruction),
// binary32 accumulation.  Both instructions take 16 bytes per lane and
// operand and the same cycles, so one kernel serves them: a slab is 128
// bytes of the reduction (64 halves or 256 4-bit values), two instructions.
//
// A workgroup computes a BM x BN tile; its waves form a WM x WN grid.  Slab s
// of both operands sits in one of two LDS stages, filled by direct-to-LDS
// loads while the slab before is multiplied; one wait and one barrier per
// slab.  A stage row is 128 bytes, its 16-byte piece c at position
// c ^ (row % 8), so that the 16 rows x 4 pieces a fragment read touches fall
// on different banks.  B rows are the instruction's first operand (D rows),
// so a lane ends up with four consecutive n of one m: outputs and the kept
// bits of a group of four are consecutive in memory.
//
// Rows past Mr / Nr re-read the last row (their results are not stored);
// 16-byte pieces past ka / kb read zeros, so the reduction's tail adds
// nothing.  TILE_GLU: half of a wave's B rows are gate rows, the other half
// the up rows of the same outputs, so g and u of one output meet in one
// lane and the activation and product need no exchange.
#pragma once

#include "nm_ffn.hpp"

namespace nm {

namespace {

#if defined(__HIP_DEVICE_COMPILE__)
template <int OA, int OB>
__device__ __forceinline__ v4f mfma_mx_op(v4i a, v4i b, v4f c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                          v8i{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, OA, sa,
                                                          OB, sb);
}
// scale byte oa of sa, ob of sb; oa and ob share the step (bit 0) and fold to
// constants in the unrolled loops
__device__ __forceinline__ v4f mfma_mx(v4i a, v4i b, v4f c, int sa, int oa, int sb, int ob) {
  switch (oa * 4 + ob) {
    case 0: return mfma_mx_op<0, 0>(a, b, c, sa, sb);
    case 2: return mfma_mx_op<0, 2>(a, b, c, sa, sb);
    case 8: return mfma_mx_op<2, 0>(a, b, c, sa, sb);
    case 10: return mfma_mx_op<2, 2>(a, b, c, sa, sb);
    case 5: return mfma_mx_op<1, 1>(a, b, c, sa, sb);
    case 7: return mfma_mx_op<1, 3>(a, b, c, sa, sb);
    case 13: return mfma_mx_op<3, 1>(a, b, c, sa, sb);
    default: return mfma_mx_op<3, 3>(a, b, c, sa, sb);
  }
}
template <int ET>
__device__ __forceinline__ v4f mfma_16(v4i a, v4i b, v4f c) {
  if constexpr (ET == TILE_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0,
                                                   0);
}
#endif

template <int ET, int OP, int OUT, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(WM * WN * 64) tile_kernel(TileArgs a, int gm) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;   // 16 x 16 tiles of a wave
  constexpr bool MX = ET == TILE_MX;
  constexpr int ROWS = BM + BN;
  constexpr int DATA = ROWS * 128;
  constexpr int STAGE = DATA + (MX ? ROWS * 8 : 0);
  constexpr int NL = ROWS / 8 / NW;                     // 1 KB loads of a wave per slab
  constexpr int NU = ROWS / 32;                         // scale units per slab
  static_assert(ROWS / 8 % NW == 0 && BM / 8 % NW == 0, "whole loads per wave, each of one operand");
  static_assert(2 * STAGE <= 160 * 1024, "LDS");
  static_assert(OP != TILE_GLU || (BN / WN / 2) % 32 == 0, "whole scale units per half");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wm = wave % WM, wn = wave / WM;

  // work item: XCD x (blockIdx % 8) takes a contiguous run of the list, in
  // groups of gm row tiles, row tile fastest inside a group: the workgroups
  // of an XCD that run together share both operands' slabs through its L2
  const int ntile = a.mt * a.nt;
  const int total = ntile * a.split * a.batch;
  const int per = (total + 7) / 8;
  int L = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (L >= min(((int)(blockIdx.x & 7) + 1) * per, total)) return;
  const int z = L / ntile;
  L -= z * ntile;
  const int bat = z / a.split, ks = z - bat * a.split;
  const int grp = L / (gm * a.nt);
  const int in = L - grp * gm * a.nt;
  const int rows_g = min(gm, a.mt - grp * gm);
  const int tn_i = in / rows_g;
  const int tm_i = grp * gm + in - tn_i * rows_g;
  constexpr int BNO = OP == TILE_GLU ? BN / 2 : BN;     // outputs per tile
  const int64_t m0 = (int64_t)tm_i * BM;
  const int64_t n0 = (int64_t)tn_i * BNO;

  const int s0 = ks * a.sps;
  const int s1 = min(s0 + a.sps, a.nslab);

  // ---- operand loads: load d fills LDS rows 8 d .. 8 d + 7, lane l row
  // 8 d + l / 8, position l % 8 = piece (l % 8) ^ (l / 8)
  const int piece = (lane & 7) ^ (lane >> 3);
  constexpr int HB = BN / WN / 2;                       // TILE_GLU: rows per half
  const uint8_t* Ab = (bat ? a.A[1] : a.A[0]) + m0 * a.lda;
  const v4i ra = make_rsrc(Ab, 0x7fffffff);
  const v4i rb0 = make_rsrc((OP != TILE_GLU && bat ? a.B[1] : a.B[0]) + n0 * a.ldb, 0x7fffffff);
  const v4i rb1 = make_rsrc(a.B[1] + (OP == TILE_GLU ? n0 * a.ldb : 0), 0x7fffffff);
  const int mlast = (int)min(a.Mr - m0, (int64_t)BM) - 1;
  const int nlast = (int)min(a.Nr - n0, (int64_t)BNO) - 1;
  int voff[NL];
#pragma unroll
  for (int j = 0; j < NL; ++j) {
    const int d = wave + NW * j;                        // j < BM / 8 / NW: A rows
    int row = 8 * d + (lane >> 3);
    if (j < BM / 8 / NW) {
      row = min(row, mlast);
      voff[j] = row * (int)a.lda + 16 * piece;
    } else {
      row -= BM;
      if constexpr (OP == TILE_GLU) row = row / (2 * HB) * HB + row % HB;
      row = min(row, nlast);
      voff[j] = row * (int)a.ldb + 16 * piece;
    }
  }
  // pieces past the end of a row, in the last slab: an offset no resource holds
  const int nfull_a = a.ka >> 3, nfull_b = a.kb >> 3;
  const int cut_a = piece >= (a.ka & 7) ? (int)0x80000000 : 0;
  const int cut_b = piece >= (a.kb & 7) ? (int)0x80000000 : 0;
  auto issue = [&](int s, int st) {
    uint8_t* sp = lds + st * STAGE;
    const int so = __builtin_amdgcn_readfirstlane(s * 128);
    const int ca = s < nfull_a ? 0 : (s > nfull_a ? (int)0x80000000 : cut_a);
    const int cb = s < nfull_b ? 0 : (s > nfull_b ? (int)0x80000000 : cut_b);
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      const int d = wave + NW * j;
      if (j < BM / 8 / NW) {
        lds_dma16(ra, lds_addr(sp + 1024 * d), voff[j] | ca, so);
      } else if constexpr (OP == TILE_GLU) {
        const int half = (8 * d - BM) / HB & 1;
        if (half)
          lds_dma16(rb1, lds_addr(sp + 1024 * d), voff[j] | cb, so);
        else
          lds_dma16(rb0, lds_addr(sp + 1024 * d), voff[j] | cb, so);
      } else {
        lds_dma16(rb0, lds_addr(sp + 1024 * d), voff[j] | cb, so);
      }
    }
    if constexpr (MX) {
      // unit u of the stage: LDS rows 32 u ..; row groups past the end repeat
      // the last one
#pragma unroll
      for (int j = 0; j < (NU + NW - 1) / NW; ++j) {
        const int u = wave + NW * j;
        if (NU % NW == 0 || u < NU) {
          const uint8_t* base;
          int64_t grp32;
          if (u < BM / 32) {
            base = a.As;
            grp32 = min(m0 / 32 + u, (a.Mr - 1) / 32);
          } else {
            int row = 32 * u - BM;
            base = a.Bs[0];
            if constexpr (OP == TILE_GLU) {
              if (row / HB & 1) base = a.Bs[1];
              row = row / (2 * HB) * HB + row % HB;
            }
            grp32 = min((n0 + row) / 32, (a.Nr - 1) / 32);
          }
          const v4i rs = make_rsrc(base + (grp32 * a.nslab + s) * 256, 256);
          const v4i rsu = v4i{__builtin_amdgcn_readfirstlane(rs[0]), __builtin_amdgcn_readfirstlane(rs[1]), rs[2],
                              rs[3]};
          lds_dma4(rsu, lds_addr(sp + DATA + 256 * u), 4 * lane, 0);
        }
      }
    }
  };

  v4f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // fragment addresses: row li of a 16-row tile, piece 4 kk + lq
  const int arow = (wm * TM * 16 + li) * 128;
  const int brow = (BM + wn * TN * 16 + li) * 128;
  const int pos[2] = {16 * (lq ^ (li & 7)), 16 * ((4 + lq) ^ (li & 7))};

  issue(s0, 0);
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 15));
  barrier_nofence();
  for (int s = s0; s < s1; ++s) {
    const int st = (s - s0) & 1;
    if (s + 1 < s1) issue(s + 1, st ^ 1);
    const uint8_t* sp = lds + st * STAGE;
    int sa[MX ? TM / 2 : 1], sb[MX ? TN / 2 : 1];
    if constexpr (MX) {
#pragma unroll
      for (int j = 0; j < TM / 2; ++j)
        sa[j] = *reinterpret_cast<const int*>(sp + DATA + (wm * TM / 2 + j) * 256 + 4 * lane);
#pragma unroll
      for (int i = 0; i < TN / 2; ++i)
        sb[i] = *reinterpret_cast<const int*>(sp + DATA + (BM / 32 + wn * TN / 2 + i) * 256 + 4 * lane);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      v4i fb[TN], fa[TM];
#pragma unroll
      for (int j = 0; j < TM; ++j) fa[j] = *reinterpret_cast<const v4i*>(sp + arow + j * 2048 + pos[kk]);
#pragma unroll
      for (int i = 0; i < TN; ++i) fb[i] = *reinterpret_cast<const v4i*>(sp + brow + i * 2048 + pos[kk]);
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          if constexpr (MX)
            acc[i][j] = mfma_mx(fb[i], fa[j], acc[i][j], sb[i / 2], 2 * (i & 1) + kk, sa[j / 2], 2 * (j & 1) + kk);
          else
            acc[i][j] = mfma_16<ET>(fb[i], fa[j], acc[i][j]);
        }
    }
    // the next slab has landed, and every wave is done with this one
    __builtin_amdgcn_s_waitcnt(waitcnt(0, 15));
    barrier_nofence();
  }

  // ---- epilogue: lane (li, lq) holds n = .. + 16 i + 4 lq + v of row m = .. + 16 j + li
  const int64_t mrow = m0 + wm * TM * 16 + li;
  if constexpr (OP == TILE_GLU) {
    constexpr int H = TN / 2;
    const int64_t ncol = n0 + wn * H * 16 + 4 * lq;
    const bool vec = (a.ldc % 4 == 0) && ((uintptr_t)a.C[0] % 8 == 0);
    const bool vecp = a.P[0] && (a.ldp % 4 == 0) && ((uintptr_t)a.P[0] % 8 == 0) && ((uintptr_t)a.P[1] % 8 == 0);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t m = mrow + 16 * j;
      if (m >= a.Mr) continue;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const int64_t n = ncol + 16 * i;
        const int left = (int)min(a.Nr - n, (int64_t)4);
        if (left <= 0) continue;
        float g[4], u[4], h[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          g[v] = acc[i][j][v];
          u[v] = acc[i + H][j][v];
          h[v] = glu_act(a.act, g[v]) * u[v];
        }
        store4<OUT>(a.C[0], m * a.ldc + n, h, left, vec);
        if (a.P[0]) {
          store4<OUT>(a.P[0], m * a.ldp + n, g, left, vecp);
          store4<OUT>(a.P[1], m * a.ldp + n, u, left, vecp);
        }
      }
    }
  } else {
    constexpr int EB = OUT == NM_F32 ? 4 : 2;
    uint8_t* C = static_cast<uint8_t*>(bat ? a.C[1] : a.C[0]) + (int64_t)ks * a.cs * EB;
    const bool vec = (a.ldc % 4 == 0) && ((uintptr_t)C % (4 * EB) == 0);
    const uint8_t* mask = OP == TILE_MASKED ? (bat ? a.mask[1] : a.mask[0]) : nullptr;
    const int64_t ncol = n0 + wn * TN * 16 + 4 * lq;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int64_t n = ncol + 16 * i;
      const int left = (int)min(a.Nr - n, (int64_t)4);
      if (left <= 0) continue;
      float b[4] = {0.f, 0.f, 0.f, 0.f};
      if (OP == TILE_LINEAR && a.bias) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (v < left) b[v] = a.bias[n + v];
      }
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int64_t m = mrow + 16 * j;
        if (m >= a.Mr) continue;
        float y[4];
        int keep = 15;
        if constexpr (OP == TILE_MASKED) keep = mask[m * a.ldm + (n >> 3)] >> (n & 4);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          y[v] = acc[i][j][v] + b[v];
          if constexpr (OP == TILE_LINEAR) y[v] = a.act == NM_ACT_GELU ? gelu_f32(y[v]) : y[v];
          if constexpr (OP == TILE_MASKED) y[v] = (keep >> v & 1) ? y[v] : 0.f;   // a select: NaN is masked too
        }
        store4<OUT>(C, m * a.ldc + n, y, left, vec);
      }
    }
  }
#endif
}

template <int ET, int OP, int OUT, int BM, int BN, int WM, int WN>
hipError_t launch_tile_cfg(TileArgs a, hipStream_t s) {
  constexpr int BNO = OP == TILE_GLU ? BN / 2 : BN;
  a.mt = (int)((a.Mr + BM - 1) / BM);
  a.nt = (int)((a.Nr + BNO - 1) / BNO);
  const int64_t total = (int64_t)a.mt * a.nt * a.split * a.batch;
  const int64_t grid = (total + 7) / 8 * 8;
  const int gm = a.mt < 8 ? a.mt : 8;
  hipLaunchKernelGGL((tile_kernel<ET, OP, OUT, BM, BN, WM, WN>), dim3((unsigned)grid), dim3(WM * WN * 64), 0, s, a,
                     gm);
  return hipGetLastError();
}

// Tile choice: 256 x 256 where its tiles fill the chip, 128 x 128 (two
// workgroups share a CU) for fewer.
template <int ET, int OP, int OUT>
hipError_t launch_tile_op(const TileArgs& a, hipStream_t s) {
  constexpr int BNO = OP == TILE_GLU ? 128 : 256;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) dev = 0;
  const int64_t big = ((a.Mr + 255) / 256) * ((a.Nr + BNO - 1) / BNO) * a.batch * a.split;
  if (big >= cu_count(dev) * 3 / 4) return launch_tile_cfg<ET, OP, OUT, 256, 256, 4, 2>(a, s);
  return launch_tile_cfg<ET, OP, OUT, 128, 128, 2, 2>(a, s);
}

template <int ET>
hipError_t launch_tile(TileOp op, int ydt, const TileArgs& a, hipStream_t s) {
  constexpr int W16 = ET == TILE_BF16 ? NM_BF16 : NM_F16;
  if constexpr (ET == TILE_MX) {
    if (op == TILE_GLU) {
      if (ydt == NM_F16) return launch_tile_op<ET, TILE_GLU, NM_F16>(a, s);
      if (ydt == NM_BF16) return launch_tile_op<ET, TILE_GLU, NM_BF16>(a, s);
      return launch_tile_op<ET, TILE_GLU, NM_F32>(a, s);
    }
    if (op != TILE_LINEAR) return hipErrorInvalidValue;
    if (ydt == NM_F16) return launch_tile_op<ET, TILE_LINEAR, NM_F16>(a, s);
    if (ydt == NM_BF16) return launch_tile_op<ET, TILE_LINEAR, NM_BF16>(a, s);
    return launch_tile_op<ET, TILE_LINEAR, NM_F32>(a, s);
  } else {
    switch (op) {
      case TILE_GLU: return launch_tile_op<ET, TILE_GLU, W16>(a, s);
      case TILE_MASKED: return launch_tile_op<ET, TILE_MASKED, W16>(a, s);
      default:
        return ydt == NM_F32 ? launch_tile_op<ET, TILE_LINEAR, NM_F32>(a, s)
                             : launch_tile_op<ET, TILE_LINEAR, W16>(a, s);
    }
  }
}

}  // namespace

}  // namespace nm
