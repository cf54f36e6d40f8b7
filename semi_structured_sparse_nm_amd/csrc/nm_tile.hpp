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
// Persistent workgroups walk a list of BM x BN tiles as one stream of slabs:
// slab s of both operands sits in one of NS LDS stages, filled by
// direct-to-LDS loads issued NS - 1 slabs ahead, across tile borders too, so
// a tile's first slabs arrive while the tile before is finished and its
// outputs leave.  A stage row is 128 bytes, its 16-byte piece c at position
// c ^ (row % 8) (no bank conflicts, by counter).  B rows are the
// instruction's first operand (D rows), so a lane ends up with four
// consecutive n of one m: outputs and the kept bits of a group of four are
// consecutive in memory.
//
// Rows past Mr / Nr repeat the last row (their results are not stored);
// 16-byte pieces past ka / kb read as zeros, so the reduction's tail adds
// nothing.  Every slab has a piece inside ka and one inside kb, so no load has
// all its lanes outside its operand: such a load would return ahead of older
// ones, and a count of outstanding loads could pass too early.  TILE_GLU: half of a wave's B rows are gate
// rows, the other half the up rows of the same outputs, so g and u of one
// output meet in one lane and the activation and product need no exchange.
// TILE_BACK: the input's and both weights' gradients are items of one launch.
//
// bf16, 2048 tokens, two 11008 x 4096 weights: gated 285 us (1.3 PFLOP/s), both
// gradients 675 (1.09); 4 bits, 1900 tokens, gated 96 (3.6).  By counters the
// matrix cores are busy 59%, 46% and 39% of that (2048 of some 3500 to 5300 cycles
// a slab of the 256 x 256 shape), and LDS is read for 1536 cycles a slab, without
// bank conflicts.  Power is a part of it only: on operands of zeros, the same
// instructions, the gated products take 12% and 18% less (fp16 with its copies
// 327 -> 289, 4 bits 95 -> 78), the gradients 1%.  (A full last round of the
// gradients' items changed nothing at 2048 tokens.)
#pragma once

#include "nm_tile_common.hpp"

namespace nm {

namespace {

#if defined(__HIP_DEVICE_COMPILE__)
template <int OA, int OB>
__device__ __forceinline__ v4f mfma_mx_op(v4i a, v4i b, v4f c, int sa, int sb) {
  // 4-bit operands take the first four registers; the rest stays undefined
  const v8i a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const v8i b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, OA, sa, OB, sb);
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

template <int ET, int OP, int OUT, int BM, int BN, int WM, int WN, int NS>
__global__ void __launch_bounds__(WM * WN * 64) __attribute__((amdgpu_waves_per_eu(2, 2)))
tile_kernel(TileArgs a, TileList list, TileList list2) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;   // 16 x 16 tiles of a wave
  constexpr bool MX = ET == TILE_MX;
  constexpr bool GLU = OP == TILE_GLU;
  constexpr bool BACK = OP == TILE_BACK;
  constexpr int ROWS = BM + BN;
  constexpr int DATA = ROWS * 128;
  constexpr int STAGE = DATA + (MX ? ROWS * 8 : 0);
  constexpr int NL = ROWS / 8 / NW;                     // 1 KB loads of a wave per slab
  constexpr int NLA = BM / 8 / NW;                      // of them A rows
  constexpr int NU = MX ? ROWS / 32 : 0;                // scale units per slab
  constexpr int NLT = NL + (NU + NW - 1) / NW;          // loads of a wave per slab
  constexpr int BNO = GLU ? BN / 2 : BN;                // outputs per tile
  constexpr int HB = BN / WN / 2;                       // TILE_GLU: rows per half
  constexpr int RJ = 8 * NW;                            // rows one load of every wave covers
  static_assert(BM % RJ == 0 && BN % RJ == 0, "every load of one operand");
  static_assert(!GLU || HB % RJ == 0 || RJ % (2 * HB) == 0, "a wave's load has rows of one weight");
  static_assert(NS * STAGE <= 160 * 1024, "LDS");
  static_assert(!MX || !GLU || HB % 32 == 0, "whole scale units per half");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * STAGE];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wm = wave % WM, wn = wave / WM;

  const TileWalk<BACK> walk(list, list2, a.w.lead);
  if (walk.count <= 0) return;

  // ---- operand loads: load d fills LDS rows 8 d .. 8 d + 7, lane l row
  // 8 d + l / 8, position l % 8 = piece (l % 8) ^ (l / 8); wave w issues
  // d = w + NW j
  const int piece = (lane & 7) ^ (lane >> 3);
  // TILE_GLU with the RJ rows of a load spanning both halves: a wave's rows are all gate or all up rows
  constexpr bool SPAN = GLU && HB % RJ != 0;
  const bool wave_up = SPAN && (8 * wave / HB & 1);
  // row of the tile (A: of BM, B: of BNO outputs) that load j brings this lane
  auto load_row = [&](auto jc) {
    constexpr int j = decltype(jc)::value;
    int row = 8 * wave + (lane >> 3) + RJ * j;
    if constexpr (j >= NLA) {
      row -= BM;
      if constexpr (GLU) row = row / (2 * HB) * HB + row % HB;
    }
    return row;
  };
  // pieces past the end of a row, in the last slab: an offset no resource holds
  // (TILE_BACK: rows of whole slabs)
  const int cut_a = !BACK && (a.ka & 7) && piece >= (a.ka & 7) ? (int)0x80000000 : 0;
  const int cut_b = !BACK && (a.kb & 7) && piece >= (a.kb & 7) ? (int)0x80000000 : 0;

  // the load cursor: work item, its resources, next slab
  int ck = 0, cs, ce, voff[NL];
  v4i ra, rb0, rb1, rsc[MX ? (NU + NW - 1) / NW : 1];
  // (always inlined: a call would keep the cursor, and what it refers to, in memory)
  auto cursor_item = [&](int k) __attribute__((always_inline)) {
    const TileItem it = walk.item(k);
    const int64_t m0 = (int64_t)it.m * BM, n0 = (int64_t)it.n * BNO;
    auto tile_rsrc = [&](const uint8_t* p, int64_t row0, int64_t ld) {
      const v4i r = make_rsrc(p + row0 * ld, 0x7fffffff);
      return v4i{scalar(r[0]), scalar(r[1]), r[2], r[3]};
    };
    const bool grad = BACK && it.batch;                 // a weight gradient
    const int64_t Mr = grad ? a.w.Mr : a.Mr, Nr = grad ? a.w.Nr : a.Nr;
    const int64_t lda = grad ? a.w.ld : a.lda, ldb = grad ? a.w.ld : a.ldb;
    const int mlast = (int)min(Mr - m0, (int64_t)BM) - 1, nlast = (int)min(Nr - n0, (int64_t)BNO) - 1;
    static_for<0, NL>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      voff[j] = j < NLA ? min(load_row(jc), mlast) * (int)lda + 16 * piece
                        : min(load_row(jc), nlast) * (int)ldb + 16 * piece;
    });
    ra = tile_rsrc(grad ? (it.batch > 1 ? a.w.A[1] : a.w.A[0]) : a.A, m0, lda);
    rb0 = tile_rsrc(grad ? a.w.B : wave_up ? a.B[1] : a.B[0], n0, ldb);
    if constexpr (GLU && !SPAN) rb1 = tile_rsrc(a.B[1], n0, ldb);
    if constexpr (MX) {
      // unit u of a stage: LDS rows 32 u ..; row groups past the end repeat the last one
      static_for<0, (NU + NW - 1) / NW>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        const int u = min(wave + NW * j, NU - 1);
        const uint8_t* base = a.As;
        int64_t g32 = min(m0 / 32 + u, (a.Mr - 1) / 32);
        if (u >= BM / 32) {
          int row = 32 * u - BM;
          base = a.Bs[0];
          if constexpr (GLU) {
            if (row / HB & 1) base = a.Bs[1];
            row = row / (2 * HB) * HB + row % HB;
          }
          g32 = min((n0 + row) / 32, (a.Nr - 1) / 32);
        }
        const v4i r = make_rsrc(base + g32 * a.nslab * 256, 0);
        rsc[j] = v4i{scalar(r[0]), scalar(r[1]), scalar(a.nslab * 256), r[3]};
      });
    }
    cs = it.s0;
    ce = it.s1;
  };
  auto issue_one = [&](auto jc, int st, int ca, int cb) {
    constexpr int j = decltype(jc)::value;
    uint8_t* sp = lds + st * STAGE;
    if constexpr (j < NL) {
      const int so = scalar(cs * 128);
      const uint32_t dst = lds_addr(sp + 1024 * (wave + NW * j));
      constexpr bool UP = GLU && !SPAN && ((RJ * j - BM) / HB & 1);
      lds_dma16(j < NLA ? ra : (UP ? rb1 : rb0), dst, voff[j] | (j < NLA ? ca : cb), so);
    } else {
      // (a wave without a unit of its own repeats the last one: no branch among the products)
      const int u = min(wave + NW * (j - NL), NU - 1);
      lds_dma4(rsc[j - NL], lds_addr(sp + DATA + 256 * u), 4 * lane, cs * 256);
    }
  };
  // part p of NP of the cursor slab's loads into stage st
  auto issue_part = [&](auto pc, auto npc, int st) {
    constexpr int P = decltype(pc)::value, NP = decltype(npc)::value;
    const int ca = BACK || cs + 1 < a.nslab ? 0 : cut_a, cb = BACK || cs + 1 < a.nslab ? 0 : cut_b;
    static_for<NLT * P / NP, NLT * (P + 1) / NP>([&](auto jc) { issue_one(jc, st, ca, cb); });
  };
  // past the last work item the cursor stays on its last slab: the loads fill
  // a stage nobody reads
  auto advance = [&]() __attribute__((always_inline)) {
    if (__builtin_expect(cs + 1 < ce, 1)) {
      ++cs;
    } else if (ck + 1 < walk.count) {
      asm volatile("" ::: "memory");                    // a branch, not selects around it
      cursor_item(++ck);
    }
  };

  v4f acc[TN][TM];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  };
  clear();

  // fragment addresses: row li of a 16-row tile, piece 4 kk + lq
  const int arow = (wm * TM * 16 + li) * 128;
  const int brow = (BM + wn * TN * 16 + li) * 128;
  const int pos0 = 16 * (lq ^ (li & 7)), pos1 = 16 * ((4 + lq) ^ (li & 7));
  struct Frag {
    v4i a[TM], b[TN];
  };
  constexpr int NF = TM + TN;
  auto read_one = [&](Frag& f, auto xc, int st, int pos) {
    constexpr int X = decltype(xc)::value;
    const uint8_t* sp = lds + st * STAGE + pos;
    if constexpr (X < TM)
      f.a[X] = *reinterpret_cast<const v4i*>(sp + arow + X * 2048);
    else
      f.b[X - TM] = *reinterpret_cast<const v4i*>(sp + brow + (X - TM) * 2048);
  };
  struct Scales {
    int a[MX ? TM / 2 : 1], b[MX ? TN / 2 : 1];
  };
  auto read_scales = [&](Scales& f, int st) {
    if constexpr (MX) {
      const uint8_t* sp = lds + st * STAGE + DATA + 4 * lane;
#pragma unroll
      for (int j = 0; j < TM / 2; ++j) f.a[j] = *reinterpret_cast<const int*>(sp + (wm * TM / 2 + j) * 256);
#pragma unroll
      for (int i = 0; i < TN / 2; ++i) f.b[i] = *reinterpret_cast<const int*>(sp + (BM / 32 + wn * TN / 2 + i) * 256);
    }
  };
  auto mul_row = [&](auto ic_, auto kc, const Frag& f, const Scales& c) {
    constexpr int i = decltype(ic_)::value, kk = decltype(kc)::value;
    // back and forth: one operand stays at the turn too (what changes at the
    // matrix cores' inputs costs power: 2-4% of the forward products)
#pragma unroll
    for (int q = 0; q < TM; ++q) {
      const int j = i & 1 ? TM - 1 - q : q;
      if constexpr (MX)
        acc[i][j] = mfma_mx(f.b[i], f.a[j], acc[i][j], c.b[i / 2], 2 * (i & 1) + kk, c.a[j / 2], 2 * (j & 1) + kk);
      else
        acc[i][j] = mfma_16<ET>(f.b[i], f.a[j], acc[i][j]);
    }
  };

  // Slab s: its second half's fragments are read between the products of the
  // first half; then, with slab s + 1 landed and every wave done reading slab
  // s, the first fragments of slab s + 1 are read and the loads of slab
  // s + NS go out into s's stage between the products of the second half.
  cursor_item(0);
  static_for<0, NS - 1>([&](auto k) {
    issue_part(ic<0>(), ic<1>(), decltype(k)::value);
    advance();
  });
  constexpr int AHEAD = NLT * (NS - 2);                 // loads that may be outstanding once the next slab is in
  static_assert(AHEAD < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt(waitcnt(AHEAD, 15));
  barrier_nofence();
  issue_part(ic<0>(), ic<1>(), NS - 1);
  advance();
  Frag f0, f1;
  Scales c0, c1;
  static_for<0, NF>([&](auto x) { read_one(f0, x, 0, pos0); });
  read_scales(c0, 0);
  int st = 0;
  for (int k = 0; k < walk.count; ++k) {
    const TileItem it = walk.item(k);
    for (int s = it.s0; s < it.s1; ++s) {
      static_for<0, TN>([&](auto i) {
        constexpr int I = decltype(i)::value;
        static_for<NF * I / TN, NF * (I + 1) / TN>([&](auto x) { read_one(f1, x, st, pos1); });
        __builtin_amdgcn_sched_barrier(0);
        mul_row(i, ic<0>(), f0, c0);
        __builtin_amdgcn_sched_barrier(0);
      });
      __builtin_amdgcn_s_waitcnt(waitcnt(AHEAD, 0));
      barrier_nofence();
      const int nx = st + 1 == NS ? 0 : st + 1;
      read_scales(c1, nx);
      static_for<0, TN>([&](auto i) {
        constexpr int I = decltype(i)::value;
        static_for<NF * I / TN, NF * (I + 1) / TN>([&](auto x) { read_one(f0, x, nx, pos0); });
        issue_part(i, ic<TN>(), st);
        __builtin_amdgcn_sched_barrier(0);
        mul_row(i, ic<1>(), f1, c0);
        __builtin_amdgcn_sched_barrier(0);
      });
      // the products stay above the cursor's branch (sunk below it they would
      // keep every fragment of the slab alive)
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) asm volatile("" : "+v"(acc[i][j]));
      advance();
      c0 = c1;
      st = nx;
    }
    tile_epilogue<OP, OUT, TM, TN>(a, it, (int64_t)it.m * BM + wm * TM * 16, (int64_t)it.n * BNO + wn * (BNO / WN), acc);
    clear();
  }
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 15));           // nothing lands in LDS after this
#endif
}

template <int ET, int OP, int OUT, int BM, int BN, int WM, int WN, int NS>
hipError_t launch_tile_cfg(const TileArgs& a, hipStream_t s) {
  constexpr int BNO = OP == TILE_GLU ? BN / 2 : BN;
  const bool back = OP == TILE_BACK;
  const TileList list = tile_list(a.Mr, a.Nr, BM, BNO, a.split, a.sps, a.nslab, back && !a.C ? 0 : 1);
  const TileList list2 = tile_list(a.w.Mr, a.w.Nr, BM, BNO, 1, a.w.nslab, a.w.nslab, back && a.w.C[0] ? 2 : 0);
  const int grid = 8 * tile_slots(list.per + list2.per);
  hipLaunchKernelGGL((tile_kernel<ET, OP, OUT, BM, BN, WM, WN, NS>), dim3((unsigned)grid), dim3(WM * WN * 64), 0, s,
                     a, list, list2);
  return hipGetLastError();
}

template <int ET, int OP, int OUT>
hipError_t launch_tile_op(const TileArgs& a, hipStream_t s) {
  switch (a.shape) {
    // wave tiles of 128 tokens x 64 rows of B keep one operand for eight
    // products (22016 x 4096 x 2048, bf16: 290 us against 341 for 64 x 128);
    // the microscaled kernel would spill in that form
    case 0:
      if constexpr (ET == TILE_MX) return launch_tile_cfg<ET, OP, OUT, 256, 256, 4, 2, 2>(a, s);
      else return launch_tile_cfg<ET, OP, OUT, 256, 256, 2, 4, 2>(a, s);
    case 1: return launch_tile_cfg<ET, OP, OUT, 128, 256, 2, 4, 3>(a, s);
    case 2:
      if constexpr (OP == TILE_GLU) return launch_tile_cfg<ET, OP, OUT, 128, 128, 4, 2, 4>(a, s);
      else return launch_tile_cfg<ET, OP, OUT, 128, 128, 2, 4, 4>(a, s);
    default:
      if constexpr (OP == TILE_GLU && ET == TILE_MX) return launch_tile_cfg<ET, OP, OUT, 64, 128, 2, 2, 6>(a, s);
      else if constexpr (OP == TILE_GLU) return launch_tile_cfg<ET, OP, OUT, 64, 128, 4, 2, 6>(a, s);
      else return launch_tile_cfg<ET, OP, OUT, 64, 128, 2, 4, 6>(a, s);
  }
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
    if (ydt != W16) return hipErrorInvalidValue;
    if (op == TILE_GLU) return launch_tile_op<ET, TILE_GLU, W16>(a, s);
    if (op == TILE_BACK) return launch_tile_op<ET, TILE_BACK, W16>(a, s);
    return hipErrorInvalidValue;
  }
}

}  // namespace

}  // namespace nm
