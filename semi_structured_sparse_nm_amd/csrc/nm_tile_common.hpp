// What the tile kernels share: the list of work items, the epilogue.
#pragma once

#include <type_traits>

#include "nm_rows.hpp"

namespace nm {

namespace {

template <int I, int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(ic<I>());
    static_for<I + 1, N>(f);
  }
}

// a wave-uniform value made visibly so (integer divisions run on the vector
// unit: buffer resources chosen by their results must be in scalar registers)
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Work items: mt x nt tiles, split slices of the reduction, batch products.
// XCD x (blockIdx % 8) takes a contiguous run of the list, in groups of gm row
// tiles, row tile fastest inside a group: the workgroups of an XCD that run
// together share both operands' slabs through its L2.
struct TileList {
  int mt, nt, gm, split, sps, nslab, total, per;
};

inline TileList tile_list(int64_t Mr, int64_t Nr, int bm, int bno, int split, int sps, int nslab, int batch) {
  TileList l;
  l.mt = (int)((Mr + bm - 1) / bm);
  l.nt = (int)((Nr + bno - 1) / bno);
  l.gm = l.mt < 8 ? l.mt : 8;
  l.split = split;
  l.sps = sps;
  l.nslab = nslab;
  l.total = l.mt * l.nt * split * batch;
  l.per = (l.total + 7) / 8;
  return l;
}
// workgroups of an XCD for `per` items: at most one a CU
inline int tile_slots(int per) {
  const int slots = (device_cu_count() + 7) / 8;
  return per < slots ? per : slots;
}

struct TileItem {
  int m, n;        // tile
  int batch, ks;   // product, slice of the reduction
  int s0, s1;      // its slabs
  int row, end;    // grouped rows: the tile's first row, its expert's end
};

// Bytes of LDS a kernel of grouped rows keeps its table of boundaries in.
constexpr int rows_table_bytes(bool grouped, int entries) { return grouped ? 8 * entries : 0; }

#if defined(__HIP_DEVICE_COMPILE__)
// The items of one workgroup of a product of grouped rows, from the table of
// the experts' rows that it builds in LDS (`table`, 2 * TAB words): the row
// tiles of BM rows of every expert times the column tiles, expert by expert
// (an XCD's run of the list meets few experts' weights), dealt as TileWalk
// does.  COLS: every expert's mt x nt tiles, its slabs of 64 rows the reduction.
// They last as long as the expert has rows, so every XCD takes an eighth of each
// expert's, side by side.  bf16, eight experts of 2048 x 4096 with 4096 rows together,
// a call for the weights' gradients alone, in us: rows even, by a router, or all of one
// expert 128, 128, 356 where each XCD has an eighth of the list (an expert of its own),
// 124, 110, 130 where the XCDs take runs of one tile a workgroup in turn, 125, 106, 116
// so; four times the rows 298, 350, 1376; 291, 292, 428; 287, 292, 396.  With the rows'
// gradients as well 205, 230, 393; 200, 205, 180; 200, 206, 168.  (32 experts of 1536 x
// 2048, 4096 rows, both: 210, 245, 300; 202, 239, 150; 213, 251, 143: runs in turn are
// 5% better there.)
template <int BM, bool COLS, int TAB>
struct RowsWalk {
  const int* row_at;
  const int* unit_at;
  int E, mt, nt, x, j, step, per, count, more, nslab;
  int q, lead, ahead, chunk;                            // COLS: as in TileWalk, and items of a chunk
  __device__ __forceinline__ RowsWalk(const RowsTile& a, int mt_, int nt_, int* table, int first = 0) {
    int* rows = table;
    int* units = table + TAB;
    if (threadIdx.x < 64) {
      row_boundaries<BM>(a.rows, [&](int i, int, int at, int u, int) {
        if (i <= a.rows.E) {
          rows[i] = at;
          units[i] = u;
        }
        return false;
      });
    }
    __syncthreads();
    row_at = rows;
    unit_at = units;
    E = a.rows.E;
    mt = mt_;
    nt = nt_;
    nslab = a.nslab;
    x = blockIdx.x & 7;
    j = blockIdx.x >> 3;
    step = gridDim.x >> 3;
    const int total = COLS ? E * mt * nt : scalar(unit_at[E]) * nt;
    per = (total + 7) / 8;
    auto rounds = [](int n, int every) { return n > 0 ? scalar((n + every - 1) / every) : 0; };
    if constexpr (COLS) {
      // the XCD's items: every eighth chunk
      chunk = min(max(mt * nt / 8, 1), step);
      const int chunks = scalar(total / chunk);
      const int n = (chunks + 7 - x) / 8 * chunk + ((chunks & 7) == x ? total - chunks * chunk : 0);
      q = first;
      lead = a.w.lead;
      ahead = lead * (step - q);
      count = rounds(n - ahead - j, step);
      if (j >= q) count += min(lead, rounds(n - (j - q), step - q));
    } else {
      const int n = min(per, total - x * per);
      more = n > 0 ? scalar(n - n / step * step) : 0;
      count = rounds(n - j, step);
    }
  }
  __device__ __forceinline__ TileItem item(int k) const {
    int L = x * per + j + k * step;
    if constexpr (COLS) {
      if (j < q) k += lead;
      const int i = k < lead ? k * (step - q) + j - q : ahead + (k - lead) * step + j;
      const int c = scalar(i / chunk);
      L = (8 * c + x) * chunk + i - c * chunk;
    }
    TileItem t;
    int e, rows_m;
    if constexpr (COLS) {
      e = scalar(L / (mt * nt));
      L -= e * mt * nt;
      rows_m = mt;
    } else {
      // the last expert whose first unit is not behind the item's
      const int unit = scalar(L / nt), lane = threadIdx.x & 63;
      e = -1;
      for (int c = 0; c <= E; c += 64)
        e += __popcll(__ballot(c + lane <= E && unit_at[min(c + lane, E)] <= unit));
      e = scalar(e);
      const int first = scalar(unit_at[e]);
      L -= first * nt;
      rows_m = scalar(unit_at[e + 1]) - first;
    }
    const int gm = min(rows_m, 8);
    const int grp = scalar(L / (gm * nt));
    const int in = L - grp * gm * nt;
    const int rows = min(gm, rows_m - grp * gm);
    t.batch = e;
    t.ks = 0;
    t.n = scalar(in / rows);
    t.m = grp * gm + in - t.n * rows;
    t.end = scalar(row_at[e + 1]);
    t.row = scalar(row_at[e]) + (COLS ? 0 : t.m * BM);
    t.s0 = 0;
    t.s1 = COLS ? max((t.end - t.row + 63) / 64, 1) : nslab;
    return t;
  }
};

// zeros in the rows of C that belong to no expert, by all workgroups
template <int OUT>
__device__ __forceinline__ void zero_other_rows(const RowsTile& a, const int* row_at) {
  if (!a.zero_rest) return;
  const int first = scalar(row_at[0]), last = scalar(row_at[a.rows.E]);
  const int rest = first + (int)a.rows.T - last;
  for (int i = blockIdx.x; i < rest; i += gridDim.x) {
    const int64_t o = (int64_t)(i < first ? i : last + (i - first)) * a.ldc;
    for (int64_t n = threadIdx.x; n < a.Nr; n += blockDim.x) {
      if constexpr (OUT == NM_F32) static_cast<float*>(a.C)[o + n] = 0.f;
      else static_cast<uint16_t*>(a.C)[o + n] = 0;
    }
  }
}

// The items of one workgroup, of `step` on its XCD: every step-th of the XCD's
// run.  TWO: of list l, then of l2 (their products count from 1).  Where l
// leaves q workgroups one item more than the others, those others take `lead`
// items of l2 each ahead of the rest, which goes to all in turn.
template <bool TWO>
struct TileWalk {
  const TileList& l;
  const TileList& l2;
  int x, j, step, n0, q, lead, ahead, count;
  static __device__ __forceinline__ int rounds(int n, int step) { return n > 0 ? scalar((n + step - 1) / step) : 0; }
  __device__ __forceinline__ TileWalk(const TileList& list, const TileList& list2, int lead_) : l(list), l2(list2) {
    x = blockIdx.x & 7;
    j = blockIdx.x >> 3;
    step = gridDim.x >> 3;
    count = n0 = rounds(min(l.per, l.total - x * l.per) - j, step);
    if constexpr (TWO) {
      const int len = min(l2.per, l2.total - x * l2.per);
      q = l.per - scalar(l.per / step) * step;
      lead = lead_;
      ahead = lead * (step - q);
      if (j >= q) count += min(lead, rounds(len - (j - q), step - q));
      count += rounds(len - ahead - j, step);
    }
  }
  __device__ __forceinline__ TileItem item(int k) const {
    const bool second = TWO && k >= n0;
    int L = x * l.per + j + k * step;
    if (second) {
      k -= n0;
      if (j < q) k += lead;
      L = x * l2.per + (k < lead ? k * (step - q) + j - q : ahead + (k - lead) * step + j);
    }
    const int mt = second ? l2.mt : l.mt, nt = second ? l2.nt : l.nt, gm = second ? l2.gm : l.gm;
    const int split = second ? l2.split : l.split, sps = second ? l2.sps : l.sps;
    const int nslab = second ? l2.nslab : l.nslab;
    const int z = scalar(L / (mt * nt));
    L -= z * mt * nt;
    TileItem t;
    t.batch = scalar(z / split);
    t.ks = z - t.batch * split;
    const int grp = scalar(L / (gm * nt));
    const int in = L - grp * gm * nt;
    const int rows = min(gm, mt - grp * gm);
    t.n = scalar(in / rows);
    t.m = grp * gm + in - t.n * rows;
    t.s0 = t.ks * sps;
    t.s1 = min(t.s0 + sps, nslab);
    if (second) ++t.batch;
    return t;
  }
};

// Outputs of one row m: per pair of 16-column tiles i, i + 1 lane group lq
// holds columns 4 lq .. + 3 of each.  Two lane exchanges leave it with columns
// 8 lq .. + 7 of the pair's 32, so a 16-bit row leaves in 64-byte pieces: past
// the caches where rows are whole pieces, through them where they start
// anywhere (past them 2048 x 4098 outputs at 4 bits, K 4096, take 39 us against 32).
// y0, y1: the lane's four values of each tile; n: first column of the pair.
template <int OUT>
__device__ __forceinline__ v4i pair_of(const float* y0, const float* y1) {
  uint32_t a0 = pack_16x2<OUT>(y0[0], y0[1]), a1 = pack_16x2<OUT>(y0[2], y0[3]);
  uint32_t b0 = pack_16x2<OUT>(y1[0], y1[1]), b1 = pack_16x2<OUT>(y1[2], y1[3]);
  // lane groups of a: 0 1 2 3, of b: 4 5 6 7 -> (0 1 | 4 5), (2 3 | 6 7) -> (0 2 4 6), (1 3 5 7)
  auto swap = [](uint32_t& x, uint32_t& y) {
    auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    auto q = __builtin_amdgcn_permlane16_swap(r[0], r[1], false, false);
    x = q[0];
    y = q[1];
  };
  swap(a0, b0);
  swap(a1, b1);
  return v4i{(int)a0, (int)a1, (int)b0, (int)b1};
}
template <int OUT>
__device__ __forceinline__ void store_pair(void* C, int64_t row, int64_t n, int64_t N, int lq, const float* y0,
                                           const float* y1, bool whole) {
  if constexpr (OUT != NM_F32) {
    if (n + 32 <= N) {
      const v4i v = pair_of<OUT>(y0, y1);
      uint16_t* p = static_cast<uint16_t*>(C) + row + n + 8 * lq;
      if (whole) __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(p));
      else *reinterpret_cast<v4i_any*>(p) = v;
      return;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t c = n + 16 * h + 4 * lq;
    const int left = (int)min(N - c, (int64_t)4);
    if (left > 0) store4<OUT>(C, row + c, h ? y1 : y0, left);
  }
}

// whether rows of ld 16-bit elements from p are whole 16-byte pieces
__device__ __forceinline__ bool whole_pieces(const void* p, int64_t ld) { return ld % 8 == 0 && (uintptr_t)p % 16 == 0; }

// One wave's TN x TM tiles of 16 x 16 as rows of C [Mr][ldc]: lane (li, lq)
// holds n = n0 + 16 i + 4 lq + v of row m0 + 16 j + li.  MASKED: zero where
// the mask has no bit; else act(C + bias).
template <bool MASKED, int OUT, int TM, int TN>
__device__ __forceinline__ void tile_rows(void* C, int64_t ldc, int64_t Mr, int64_t Nr, const float* bias, int act,
                                          const uint8_t* mask, int64_t ldm, int64_t m0, int64_t n0,
                                          const v4f (&acc)[TN][TM]) {
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const bool whole = whole_pieces(C, ldc);
  // the kept bits of every row and column pair (32 columns, one word: rows of
  // the mask are padded to 64), in flight together before the first use
  uint32_t keep[MASKED ? TN / 2 : 1][TM];
  if constexpr (MASKED) {
#pragma unroll
    for (int i = 0; i < TN / 2; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int64_t m = m0 + 16 * j + li, n = n0 + 32 * i;
        keep[i][j] = m < Mr && n < Nr ? *reinterpret_cast<const uint32_t*>(mask + m * ldm + n / 8) >> (4 * lq) : 0;
      }
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = 0; i < TN; i += 2) {
    float b[2][4];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t n = n0 + 16 * (i + e) + 4 * lq + v;
        b[e][v] = !MASKED && bias && n < Nr ? bias[n] : 0.f;
      }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t m = m0 + 16 * j + li;
      float y[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if constexpr (MASKED) {
            y[e][v] = keep[i / 2][j] >> (16 * e + v) & 1 ? acc[i + e][j][v] : 0.f;   // a select: NaN is masked too
          } else {
            y[e][v] = acc[i + e][j][v] + b[e][v];
            y[e][v] = act == NM_ACT_GELU ? gelu_f32(y[e][v]) : y[e][v];
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);                // one output's temporaries at a time
      if (m < Mr) store_pair<OUT>(C, m * ldc, n0 + 16 * i, Nr, lq, y[0], y[1], whole);
    }
  }
}

// One wave's tiles of 8-bit products as rows of C: integer sums, converted once,
// times the row's scale, times the channel's, each product rounded to binary32
// (bias, activation and the rounding to the output's type follow).
template <int OUT, int TM, int TN>
__device__ __forceinline__ void tile_rows_i8(void* C, int64_t ldc, int64_t Mr, int64_t Nr, const float* xscale,
                                             const float* wscale, const float* bias, int act, int64_t m0, int64_t n0,
                                             const v4i (&acc)[TN][TM]) {
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  const bool whole = whole_pieces(C, ldc);
  float sx[TM];
#pragma unroll
  for (int j = 0; j < TM; ++j) sx[j] = xscale[min(m0 + 16 * j + li, Mr - 1)];
#pragma unroll
  for (int i = 0; i < TN; i += 2) {
    float sw[2][4], b[2][4];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t n = n0 + 16 * (i + e) + 4 * lq + v;
        sw[e][v] = n < Nr ? wscale[n] : 0.f;
        b[e][v] = bias && n < Nr ? bias[n] : 0.f;
      }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t m = m0 + 16 * j + li;
      float y[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          y[e][v] = (float)acc[i + e][j][v] * sx[j] * sw[e][v] + b[e][v];
          y[e][v] = act == NM_ACT_GELU ? gelu_f32(y[e][v]) : y[e][v];
        }
      __builtin_amdgcn_sched_barrier(0);                // one output's temporaries at a time
      if (m < Mr) store_pair<OUT>(C, m * ldc, n0 + 16 * i, Nr, lq, y[0], y[1], whole);
    }
  }
}

// One wave's tiles of a weight gradient; kept: its bits (one 16-byte load a lane,
// asked for before the item's products; read row by row in the epilogue they cost
// 3 us a tile of 256 x 256).
template <int OUT, int TM, int TN>
__device__ __forceinline__ void tile_cols(const RowsTile& a, const TileItem& it, int64_t m0, int64_t n0, v4i kept,
                                          const v4f (&acc)[TN][TM]) {
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  uint16_t* C = static_cast<uint16_t*>(a.C) + it.batch * a.es;
  const bool whole = whole_pieces(a.C, a.ldc) && a.es % 8 == 0;
  const int i0 = (int)(n0 >> 4) & 3, j0 = (int)(m0 >> 4) & 7;
#pragma unroll
  for (int i = 0; i < TN; i += 2)
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int bits = (TM == 8 ? kept[j >> 1] : kept[(j0 + j) >> 1]) >> (16 * (j & 1) + 4 * (i0 + i));
      const int64_t m = m0 + 16 * j + li;
      float y[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          y[e][v] = bits >> (4 * e + v) & 1 ? acc[i + e][j][v] : 0.f;   // a select: NaN is masked too
      __builtin_amdgcn_sched_barrier(0);                // one output's temporaries at a time
      if (m < a.Mr) store_pair<OUT>(C, m * a.ldc, n0 + 16 * i, a.Nr, lq, y[0], y[1], whole);
    }
}

// Epilogue of one wave's tiles of grouped rows.
template <int OUT, int TM, int TN, class Acc>
__device__ __forceinline__ void rows_epilogue(const RowsTile& a, const TileItem& it, int64_t m0, int64_t n0,
                                              const Acc (&acc)[TN][TM]) {
  if constexpr (std::is_same<Acc, v4i>::value)
    tile_rows_i8<OUT, TM, TN>(a.C, a.ldc, it.end, a.Nr, a.xscale, a.wscale + it.batch * a.Nr,
                              a.bias ? a.bias + it.batch * a.Nr : nullptr, a.act, m0, n0, acc);
  else
    tile_rows<false, OUT, TM, TN>(a.C, a.ldc, it.end, a.Nr, nullptr, NM_ACT_NONE, nullptr, 0, m0, n0, acc);
}

// Epilogue of one wave's tiles.  TILE_GLU: tiles i < TN / 2 are gate, the
// others up columns of the same outputs.
template <int OP, int OUT, int TM, int TN>
__device__ __forceinline__ void tile_epilogue(const TileArgs& a, const TileItem& it, int64_t m0, int64_t n0,
                                              const v4f (&acc)[TN][TM]) {
  if constexpr (OP == TILE_GLU) {
    const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
    constexpr int H = TN / 2;
    const bool whole = whole_pieces(a.C, a.ldc);
    const bool kept = whole_pieces(a.P[0], a.ldp) && whole_pieces(a.P[1], a.ldp);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t m = m0 + 16 * j + li;
#pragma unroll
      for (int i = 0; i < H; i += 2) {
        float g[2][4], u[2][4], h[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            g[e][v] = acc[i + e][j][v];
            u[e][v] = acc[i + e + H][j][v];
            h[e][v] = glu_act(a.act, g[e][v]) * u[e][v];
          }
        __builtin_amdgcn_sched_barrier(0);              // one output's temporaries at a time
        if (m < a.Mr) {
          store_pair<OUT>(a.C, m * a.ldc, n0 + 16 * i, a.Nr, lq, h[0], h[1], whole);
          if (a.P[0] && a.p32) {
            store_pair<NM_F32>(a.P[0], m * a.ldp, n0 + 16 * i, a.Nr, lq, g[0], g[1], false);
            store_pair<NM_F32>(a.P[1], m * a.ldp, n0 + 16 * i, a.Nr, lq, u[0], u[1], false);
          } else if (a.P[0]) {
            store_pair<OUT>(a.P[0], m * a.ldp, n0 + 16 * i, a.Nr, lq, g[0], g[1], kept);
            store_pair<OUT>(a.P[1], m * a.ldp, n0 + 16 * i, a.Nr, lq, u[0], u[1], kept);
          }
        }
      }
    }
  } else if constexpr (OP == TILE_LINEAR) {
    void* C = static_cast<uint8_t*>(a.C) + (int64_t)it.ks * a.cs * (OUT == NM_F32 ? 4 : 2);
    tile_rows<false, OUT, TM, TN>(C, a.ldc, a.Mr, a.Nr, a.bias, a.act, nullptr, 0, m0, n0, acc);
  } else if (it.batch) {
    const bool up = it.batch > 1;
    tile_rows<true, OUT, TM, TN>(up ? a.w.C[1] : a.w.C[0], a.w.ldc, a.w.Mr, a.w.Nr, nullptr, NM_ACT_NONE,
                                 up ? a.w.mask[1] : a.w.mask[0], a.w.ldm, m0, n0, acc);
  } else if (a.split > 1) {
    tile_rows<false, NM_F32, TM, TN>(static_cast<float*>(a.C) + (int64_t)it.ks * a.cs, a.ldc, a.Mr, a.Nr, nullptr,
                                     NM_ACT_NONE, nullptr, 0, m0, n0, acc);
  } else {
    tile_rows<false, OUT, TM, TN>(a.C, a.ldc, a.Mr, a.Nr, nullptr, NM_ACT_NONE, nullptr, 0, m0, n0, acc);
  }
}
#endif

}  // namespace

}  // namespace nm
