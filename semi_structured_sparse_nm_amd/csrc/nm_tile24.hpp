// Products with 2:4 packed weights, more than a few tokens: the gated block, and
// products of rows grouped by expert (16-bit and 8-bit).  The packed blocks go to
// the sparse matrix instruction (v_smfmac_f32_16x16x64) as they are, so neither a
// dense copy of the weights nor the products with pruned ones exist.
//
// The structure is the dense tile product's (nm_tile.hpp): persistent
// workgroups, one stream of slabs through NS LDS stages, loads and fragment
// reads between the products.  A slab is 64 columns: BM token rows of 128
// bytes, and for 128 outputs the 16-row blocks of both weights, 1 KB of values
// and 128 bytes of positions each.  Half the products of the dense form, and
// 50 KB instead of 64 KB a slab at BM = 256.  2048 tokens, 11008 x 4096: 198 to 212
// us (1.8 PFLOP/s of the dense product, which takes 285 by dense tiles); 256
// tokens 36 us.  By counters the matrix cores are busy 75 us of it (1024 cycles a
// slab, and LDS is read for as many); a quarter is power (151 us on operands of
// zeros, the same instructions), and the last of three rounds is 69% full.
//
// A stage holds the tokens (16-byte piece c of row r at position c ^ (r % 8)),
// the sixteen value blocks (piece c of row r at c ^ (r / 2 % 4)) and their
// positions.  A wave multiplies its gate blocks first, then its up blocks;
// while the up products run, each token tile's registers are refilled with the
// next slab's as soon as its last product is issued.
//
// Grouped rows (TILE_ROWS): the "up" blocks are the row blocks behind a wave's
// "gate" ones of the same weight, so a tile has twice the outputs.
//
// Operand layout of the instruction (as in the [K][T] kernels): lane (row i,
// group g) of the first operand holds the 16 bytes at 16 g of its packed row
// and that run's 16 position bits; of the second operand columns 8 g .. + 7
// and 32 + 8 g .. + 7 of its token.  8-bit: a slab is 128 columns, the same
// 128 bytes of a token and 1 KB of a block's values, and 256 bytes of
// positions, 32 bits a run.
#pragma once

#include <algorithm>

#include "nm_tile_common.hpp"

namespace nm {

namespace {

typedef _Float16 v16h_t __attribute__((ext_vector_type(16)));
typedef __bf16 v16bf_t __attribute__((ext_vector_type(16)));

#if defined(__HIP_DEVICE_COMPILE__)
template <int WT>
__device__ __forceinline__ auto smfmac_tile(v4i a, v4i b0, v4i b1,
                                            typename std::conditional<WT == NM_I8, v4i, v4f>::type c, int idx) {
  const v8i b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
  if constexpr (WT == NM_I8)
    return __builtin_amdgcn_smfmac_i32_16x16x128_i8(a, b, c, idx, 0, 0);
  else if constexpr (WT == NM_F16)
    return __builtin_amdgcn_smfmac_f32_16x16x64_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v16h_t, b), c, idx,
                                                    0, 0);
  else
    return __builtin_amdgcn_smfmac_f32_16x16x64_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v16bf_t, b), c,
                                                     idx, 0, 0);
}
#endif

struct Tile24Args : TileArgs { // A, lda, Mr, Nr, ka, nslab, outputs, act
  const uint8_t* values[2];    // gate, up
  const uint8_t* meta[2];
};

template <int OP>
using tile24_args = typename std::conditional<OP == TILE_ROWS, RowsTile, Tile24Args>::type;

// Boundaries the table of grouped rows holds: the 8-bit shapes that leave 4 KB
// of LDS take half as many.
template <int WT, int TM, int H, int NS>
constexpr int rows24_table = NS * (64 * TM * 128 + 4 * H * (WT == NM_I8 ? 1280 : 1152)) + 8 * kRowsTable <= 160 * 1024
                                 ? kRowsTable
                                 : kRowsTable / 2;

// TM: 16-token tiles of a wave, H: its 16-output tiles; four waves along the
// tokens, two along the outputs
template <int WT, int OP, int OUT, int TM, int H, int NS>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
tile24_kernel(tile24_args<OP> p, TileList list) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool EROWS = OP == TILE_ROWS, I8 = WT == NM_I8;
  typedef typename std::conditional<I8, v4i, v4f>::type Acc;
  constexpr int NW = 8, BM = 64 * TM, TN = 2 * H, BNO = EROWS ? 64 * H : 32 * H;
  constexpr int NB = 4 * H;                             // blocks of a stage: per wave column H gate, then H up
  constexpr int MK = I8 ? 256 : 128;                    // bytes of a block's positions
  constexpr int XB = BM * 128, VB = NB * 1024, MB = NB * MK;
  constexpr int STAGE = XB + VB + MB;
  constexpr int NLX = BM / 8 / NW;                      // token loads of a wave per slab
  constexpr int NLV = NB / NW;                          // value blocks of a wave
  constexpr int NLT = NLX + NLV + (I8 ? NLV : 1);       // and their positions, or a pair of position blocks
  constexpr int TAB = rows24_table<WT, TM, H, NS>, TABLE = rows_table_bytes(EROWS, TAB);
  static_assert(NB % NW == 0 && NB >= 8, "whole blocks per wave");
  constexpr int AHEAD = NLT * (NS - 2);
  static_assert(NS * STAGE + TABLE <= 160 * 1024 && AHEAD < 64, "LDS, vmcnt");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * STAGE + TABLE];

  const TileArgs& a = p;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wm = wave & 3, wn = wave >> 2;
  const int nKB = a.nslab;
  const int64_t nRB = (a.Nr + 15) / 16;

  const auto walk = [&]() {
    if constexpr (EROWS) return RowsWalk<BM, false, TAB>(p, 0, list.nt, reinterpret_cast<int*>(lds + NS * STAGE));
    else return TileWalk<false>(list, list, 0);
  }();
  if constexpr (EROWS) zero_other_rows<OUT>(p, walk.row_at);
  if (walk.count <= 0) return;

  // ---- loads.  Tokens: load d = w + 8 j fills LDS rows 8 d .. + 7.  Block b
  // of a stage: wave column b / (2 H), weight b % (2 H) / H, row block b % H of
  // that column's H (EROWS: row block b).  Wave w brings value blocks NLV w ..
  // and position blocks 2 p, 2 p + 1, p = w modulo the pairs there are (8 bits:
  // its value blocks' ones).
  const int piece = (lane & 7) ^ (lane >> 3);
  const int cut = (a.ka & 7) && piece >= (a.ka & 7) ? (int)0x80000000 : 0;
  const int bv = NLV * wave, bm = 2 * (wave % (NB / 2));
  auto weight_of = [](int b) { return EROWS ? 0 : b % (2 * H) / H; };
  auto row_of = [](int b) { return EROWS ? b : b / (2 * H) * H + b % H; };
  const int voff_v = (lane >> 2) * 64 + 16 * ((lane & 3) ^ ((lane >> 3) & 3));
  int ck = 0, cs, ce, voff[NLX], voff_m, so_v[NLV];
  v4i ra, rv, rm;
  auto cursor_item = [&](int k) __attribute__((always_inline)) {
    const TileItem it = walk.item(k);
    const int64_t m0 = EROWS ? (int64_t)it.row : (int64_t)it.m * BM, rb0 = (int64_t)it.n * (BNO / 16);
    auto rsrc = [&](const uint8_t* b, int64_t off) {
      const v4i r = make_rsrc(b + off, 0x7fffffff);
      return v4i{scalar(r[0]), scalar(r[1]), r[2], r[3]};
    };
    const int mlast = (int)min((EROWS ? (int64_t)it.end : a.Mr) - m0, (int64_t)BM) - 1;
    static_for<0, NLX>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      voff[j] = min(8 * (wave + NW * j) + (lane >> 3), mlast) * (int)a.lda + 16 * piece;
    });
    ra = rsrc(a.A, m0 * a.lda);
    if constexpr (EROWS) {
      rv = rsrc(p.B[0], (it.batch * nRB + rb0) * nKB * 1024);
      rm = rsrc(p.meta, (it.batch * nRB + rb0) * nKB * MK);
    } else {
      rv = rsrc(weight_of(bv) ? p.values[1] : p.values[0], rb0 * nKB * 1024);
      rm = rsrc(weight_of(bm) ? p.meta[1] : p.meta[0], rb0 * nKB * MK);
    }
    // row blocks past the weights' end repeat the last one (their results are not stored)
    const int blast = (int)min(nRB - rb0, (int64_t)(BNO / 16)) - 1;
    static_for<0, NLV>([&](auto q) {
      so_v[decltype(q)::value] = scalar(min(row_of(bv + decltype(q)::value), blast) * nKB * 1024);
    });
    if constexpr (I8) voff_m = 4 * lane;
    else voff_m = min(row_of(bm + (lane >> 5)), blast) * nKB * 128 + 4 * (lane & 31);
    cs = it.s0;
    ce = it.s1;
  };
  auto issue_one = [&](auto jc, int st) {
    constexpr int j = decltype(jc)::value;
    uint8_t* sp = lds + st * STAGE;
    if constexpr (j < NLX) {
      const int c = cs + 1 < a.nslab ? 0 : cut;
      lds_dma16(ra, lds_addr(sp + 1024 * (wave + NW * j)), voff[j] | c, cs * 128);
    } else if constexpr (j < NLX + NLV) {
      lds_dma16(rv, lds_addr(sp + XB + 1024 * (bv + j - NLX)), voff_v, so_v[j - NLX] + cs * 1024);
    } else if constexpr (I8) {
      constexpr int q = j - NLX - NLV;                  // (four bytes of positions for 16 of values)
      lds_dma4(rm, lds_addr(sp + XB + VB + MK * (bv + q)), voff_m, (so_v[q] >> 2) + cs * MK);
    } else {
      lds_dma4(rm, lds_addr(sp + XB + VB + MK * bm), voff_m, cs * MK);
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {
    if (__builtin_expect(cs + 1 < ce, 1)) {
      ++cs;
    } else if (ck + 1 < walk.count) {
      asm volatile("" ::: "memory");                    // a branch, not selects around it
      cursor_item(++ck);
    }
  };

  Acc acc[TN][TM];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = Acc{0, 0, 0, 0};
  };
  clear();

  // ---- fragments
  const int xrow = (wm * TM * 16 + li) * 128;
  const int xp0 = xrow + 16 * (lq ^ (li & 7)), xp1 = xrow + 16 * ((4 + lq) ^ (li & 7));
  const int vpos = XB + wn * TN * 1024 + li * 64 + 16 * (lq ^ ((li >> 1) & 3));
  const int mpos = XB + VB + wn * TN * MK + (I8 ? li * 16 + 4 * lq : li * 8 + 2 * lq);
  v4i x0[TM], x1[TM];
  struct Blocks {
    v4i v[H];
    int idx[H];
  };
  auto read_x = [&](auto jc, int st) {
    constexpr int j = decltype(jc)::value;
    const uint8_t* sp = lds + st * STAGE + j * 2048;
    x0[j] = *reinterpret_cast<const v4i*>(sp + xp0);
    x1[j] = *reinterpret_cast<const v4i*>(sp + xp1);
  };
  auto read_block = [&](Blocks& b, auto ic_, int half, int st) {
    constexpr int i = decltype(ic_)::value;
    const uint8_t* sp = lds + st * STAGE;
    b.v[i] = *reinterpret_cast<const v4i*>(sp + vpos + (half * H + i) * 1024);
    if constexpr (I8) b.idx[i] = *reinterpret_cast<const int*>(sp + mpos + (half * H + i) * MK);
    else b.idx[i] = *reinterpret_cast<const uint16_t*>(sp + mpos + (half * H + i) * MK);
  };

  cursor_item(0);
  static_for<0, NS - 1>([&](auto k) {
    static_for<0, NLT>([&](auto j) { issue_one(j, decltype(k)::value); });
    advance();
  });
  __builtin_amdgcn_s_waitcnt(waitcnt(AHEAD, 15));
  barrier_nofence();
  static_for<0, NLT>([&](auto j) { issue_one(j, NS - 1); });
  advance();
  Blocks bg, bu;
  static_for<0, TM>([&](auto j) { read_x(j, 0); });
  static_for<0, H>([&](auto i) { read_block(bg, i, 0, 0); });
  int st = 0;
  for (int k = 0; k < walk.count; ++k) {
    const TileItem it = walk.item(k);
    for (int s = it.s0; s < it.s1; ++s) {
      // gate products; the up blocks are read between them
      static_for<0, TM>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        static_for<H * j / TM, H * (j + 1) / TM>([&](auto i) { read_block(bu, i, 1, st); });
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < H; ++i) acc[i][j] = smfmac_tile<WT>(bg.v[i], x0[j], x1[j], acc[i][j], bg.idx[i]);
        __builtin_amdgcn_sched_barrier(0);
      });
      // slab s + 1 has landed, and every wave is done reading slab s
      __builtin_amdgcn_s_waitcnt(waitcnt(AHEAD, 0));
      barrier_nofence();
      const int nx = st + 1 == NS ? 0 : st + 1;
      // up products; loads of slab s + NS into s's stage, next slab's gate
      // blocks and, behind their last product, its tokens
      static_for<0, TM>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        static_for<NLT * j / TM, NLT * (j + 1) / TM>([&](auto q) { issue_one(q, st); });
        static_for<H * j / TM, H * (j + 1) / TM>([&](auto i) { read_block(bg, i, 0, nx); });
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < H; ++i)
          acc[H + i][j] = smfmac_tile<WT>(bu.v[i], x0[j], x1[j], acc[H + i][j], bu.idx[i]);
        __builtin_amdgcn_sched_barrier(0);
        read_x(jc, nx);
      });
      // the products stay above the cursor's branch
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) asm volatile("" : "+v"(acc[i][j]));
      advance();
      st = nx;
    }
    if constexpr (EROWS)
      rows_epilogue<OUT, TM, TN>(p, it, it.row + wm * TM * 16, (int64_t)it.n * BNO + wn * TN * 16, acc);
    else
      tile_epilogue<TILE_GLU, WT, TM, TN>(a, it, (int64_t)it.m * BM + wm * TM * 16, (int64_t)it.n * BNO + wn * H * 16,
                                          acc);
    clear();
  }
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 15));           // nothing lands in LDS after this
#endif
}

template <int WT, int TM, int H, int NS>
hipError_t launch_tile24_cfg(const Tile24Args& p, hipStream_t s) {
  const TileList list = tile_list(p.Mr, p.Nr, 64 * TM, 32 * H, 1, p.nslab, p.nslab, 1);
  hipLaunchKernelGGL((tile24_kernel<WT, TILE_GLU, WT, TM, H, NS>), dim3((unsigned)(8 * tile_slots(list.per))),
                     dim3(512), 0, s, p, list);
  return hipGetLastError();
}

template <int WT, int OUT, int TM, int H, int NS>
hipError_t launch_rows24_cfg(const RowsTile& p, hipStream_t s) {
  if (p.rows.E >= rows24_table<WT, TM, H, NS>) return hipErrorInvalidValue;
  TileList l{};
  l.nt = (int)((p.Nr + 64 * H - 1) / (64 * H));
  const int64_t most = units_most(p.rows.T, p.rows.E, 64 * TM) * l.nt;
  const int grid = 8 * tile_slots((int)std::min<int64_t>((most + 7) / 8, 1 << 20));
  hipLaunchKernelGGL((tile24_kernel<WT, TILE_ROWS, OUT, TM, H, NS>), dim3((unsigned)grid), dim3(512), 0, s, p, l);
  return hipGetLastError();
}

}  // namespace

}  // namespace nm
