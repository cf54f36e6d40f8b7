// What the tile kernels share: the list of work items, the epilogue.
#pragma once

#include "nm_ffn.hpp"

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

// Work items: mt x nt tiles, a.split slices of the reduction, a.batch
// products.  XCD x (blockIdx % 8) takes a contiguous run of the list, in
// groups of gm row tiles, row tile fastest inside a group: the workgroups of
// an XCD that run together share both operands' slabs through its L2.
struct TileList {
  int mt, nt, gm, batch, split, sps, nslab, total, per, grid;
};

inline TileList tile_list(const TileArgs& a, int bm, int bno) {
  TileList l;
  l.mt = (int)((a.Mr + bm - 1) / bm);
  l.nt = (int)((a.Nr + bno - 1) / bno);
  l.gm = l.mt < 8 ? l.mt : 8;
  l.batch = a.batch;
  l.split = a.split;
  l.sps = a.sps;
  l.nslab = a.nslab;
  l.total = l.mt * l.nt * a.split * a.batch;
  l.per = (l.total + 7) / 8;
  const int slots = (device_cu_count() + 7) / 8;   // workgroups of an XCD (one a CU)
  l.grid = 8 * (l.per < slots ? l.per : slots);
  return l;
}

struct TileItem {
  int m, n;        // tile
  int batch, ks;   // product, slice of the reduction
  int s0, s1;      // its slabs
};

#if defined(__HIP_DEVICE_COMPILE__)
// the items of one workgroup: every (workgroups of an XCD)-th of its XCD's run
struct TileWalk {
  const TileList& l;
  int first, step, count;
  __device__ __forceinline__ explicit TileWalk(const TileList& list) : l(list) {
    const int x = blockIdx.x & 7, j = blockIdx.x >> 3;
    step = l.grid >> 3;
    first = x * l.per + j;
    const int end = min((x + 1) * l.per, l.total);
    count = first < end ? scalar((end - first + step - 1) / step) : 0;
  }
  __device__ __forceinline__ TileItem item(int k) const {
    int L = first + k * step;
    const int ntile = l.mt * l.nt;
    const int z = scalar(L / ntile);
    L -= z * ntile;
    TileItem t;
    t.batch = scalar(z / l.split);
    t.ks = z - t.batch * l.split;
    const int grp = scalar(L / (l.gm * l.nt));
    const int in = L - grp * l.gm * l.nt;
    const int rows = min(l.gm, l.mt - grp * l.gm);
    t.n = scalar(in / rows);
    t.m = grp * l.gm + in - t.n * rows;
    t.s0 = t.ks * l.sps;
    t.s1 = min(t.s0 + l.sps, l.nslab);
    return t;
  }
};

// Outputs of one row m: per pair of 16-column tiles i, i + 1 lane group lq
// holds columns 4 lq .. + 3 of each.  Where rows allow 16-byte stores, two
// lane exchanges leave it with columns 8 lq .. + 7 of the pair's 32, so a row
// leaves in 64-byte pieces.
// y0, y1: the lane's four values of each tile; n: first column of the pair.
template <int OUT>
__device__ __forceinline__ void store_pair(void* C, int64_t row, int64_t n, int64_t N, int lq, const float* y0,
                                           const float* y1, bool vec8, bool vec4) {
  if constexpr (OUT != NM_F32) {
    if (vec8 && n + 32 <= N) {
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
      const v4i v = {(int)a0, (int)a1, (int)b0, (int)b1};
      __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(static_cast<uint16_t*>(C) + row + n + 8 * lq));
      return;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t c = n + 16 * h + 4 * lq;
    const int left = (int)min(N - c, (int64_t)4);
    if (left > 0) store4<OUT>(C, row + c, h ? y1 : y0, left, vec4);
  }
}

// Epilogue of one wave's TN x TM tiles of 16 x 16: lane (li, lq) holds n = n0
// + 16 i + 4 lq + v of row m0 + 16 j + li.  TILE_GLU: tiles i < TN / 2 are
// gate, the others up columns of the same outputs.
template <int OP, int OUT, int TM, int TN>
__device__ __forceinline__ void tile_epilogue(const TileArgs& a, const TileItem& it, int64_t m0, int64_t n0,
                                              const v4f (&acc)[TN][TM]) {
  const int lane = threadIdx.x & 63, li = lane & 15, lq = lane >> 4;
  constexpr int EB = OUT == NM_F32 ? 4 : 2;
  uint8_t* C = static_cast<uint8_t*>(OP == TILE_MASKED && it.batch ? a.C[1] : a.C[0]) + (int64_t)it.ks * a.cs * EB;
  auto vec = [](const void* p, int64_t ld, int n) { return ld % n == 0 && (uintptr_t)p % (n * EB) == 0; };
  const bool v8 = vec(C, a.ldc, 8), v4 = vec(C, a.ldc, 4);
  if constexpr (OP == TILE_GLU) {
    constexpr int H = TN / 2;
    const bool p8 = a.P[0] && vec(a.P[0], a.ldp, 8) && vec(a.P[1], a.ldp, 8);
    const bool p4 = a.P[0] && vec(a.P[0], a.ldp, 4) && vec(a.P[1], a.ldp, 4);
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
          store_pair<OUT>(C, m * a.ldc, n0 + 16 * i, a.Nr, lq, h[0], h[1], v8, v4);
          if (a.P[0]) {
            store_pair<OUT>(a.P[0], m * a.ldp, n0 + 16 * i, a.Nr, lq, g[0], g[1], p8, p4);
            store_pair<OUT>(a.P[1], m * a.ldp, n0 + 16 * i, a.Nr, lq, u[0], u[1], p8, p4);
          }
        }
      }
    }
  } else {
    // the kept bits of every row and column pair (32 columns, one word: rows
    // of the mask are padded to 64), in flight together before the first use
    uint32_t keep[TN / 2][TM];
    if constexpr (OP == TILE_MASKED) {
      const uint8_t* mask = it.batch ? a.mask[1] : a.mask[0];
#pragma unroll
      for (int i = 0; i < TN / 2; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          const int64_t m = m0 + 16 * j + li, n = n0 + 32 * i;
          keep[i][j] = m < a.Mr && n < a.Nr ? *reinterpret_cast<const uint32_t*>(mask + m * a.ldm + n / 8) >> (4 * lq) : 0;
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
          b[e][v] = OP == TILE_LINEAR && a.bias && n < a.Nr ? a.bias[n] : 0.f;
        }
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int64_t m = m0 + 16 * j + li;
        float y[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            y[e][v] = acc[i + e][j][v] + b[e][v];
            if constexpr (OP == TILE_LINEAR) y[e][v] = a.act == NM_ACT_GELU ? gelu_f32(y[e][v]) : y[e][v];
            if constexpr (OP == TILE_MASKED) y[e][v] = keep[i / 2][j] >> (16 * e + v) & 1 ? y[e][v] : 0.f;   // a select: NaN is masked too
          }
        }
        __builtin_amdgcn_sched_barrier(0);              // one output's temporaries at a time
        if (m < a.Mr) store_pair<OUT>(C, m * a.ldc, n0 + 16 * i, a.Nr, lq, y[0], y[1], v8, v4);
      }
    }
  }
}
#endif

}  // namespace

}  // namespace nm
