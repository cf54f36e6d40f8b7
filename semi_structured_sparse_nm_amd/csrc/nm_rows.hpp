// Shared definitions of the products of rows grouped by expert (16-bit and
// 8-bit packed weights, one weight being one expert) and of the 8-bit row
// format.  Internal; the public surface is include/nm_sparse.h.
#pragma once

#include "nm_ffn.hpp"

namespace nm {

// Most experts: each workgroup keeps a table of their rows in LDS.
constexpr int kMaxExperts = 1023;

// 8-bit rows: K elements and zeros up to a multiple of 128, one matrix
// instruction's reduction of the sparse product.
inline int64_t i8_kp(int64_t K) { return (K + 127) / 128 * 128; }

// The rows of each expert: at[e] .. at[e + 1] - 1, `at` of E + 1 whole numbers
// in device memory.  Read defensively, since the host does not see them: each
// is taken into [0, T] and as at least the one before it, so whatever they
// hold, experts' rows are disjoint and inside the call's.  Null: one expert,
// all rows.
struct RowGroups {
  const void* at;
  int wide;                  // 64-bit, else 32-bit
  int E;
  int64_t T;
};

// Y[s][r] = act(sum_k X[s][k] W_e[r][k] (x scale[s] x wscale[e][r]) + bias[e][r])
struct RowsArgs {
  Geometry g;                // of one expert's weight
  int wdt;
  const uint8_t* values;     // of expert 0; the others follow
  const uint8_t* meta;
  RowGroups rows;
  const void* X;             // 16-bit values, or 8-bit elements
  int64_t ldx;
  const float* xscale;       // 8 bits: [T]
  int xdt;                   // NM_I8, or (streamed, rows_decode_quantizes) the type the rows are quantised from
  const float* wscale;       // 8 bits: [E][R]
  const float* bias;         // 8 bits: [E][R] or nullptr
  int act;
  void* Y;
  int64_t ldy;
  int ydt;
  bool zero_rest;            // rows of no expert: zeros, else left as they are
};

// Units of `u` rows that T rows of E experts make at most, each expert's
// counted for itself.
inline int64_t units_most(int64_t T, int64_t E, int64_t u) {
  const int64_t some = T < E ? T : E;
  return (T + some * (u - 1)) / u;
}

// How a product multiplies.
enum RowsPath {
  ROWS_STREAM,   // few rows an expert: the packed weights streamed past each 16 to 64 of them
  ROWS_WIDE,     // more: past each 64 or 128, shared by a workgroup's waves
  ROWS_SPARSE,   // 2:4: the sparse tile product
  ROWS_REPACK,   // 1:4, 1:8, 2:8: re-packed to 2:4 in the workspace, then the same
  ROWS_DENSE     // others: dense blocks (in the workspace where N < M), the dense tile product
};
struct RowsPlan {
  RowsPath path;
  int shape;                 // tile shape; ROWS_WIDE: 16-row tiles of a workgroup
  int64_t cut = 0;           // tiles: outputs from here on, if any, in a launch of their own
  int rest = 0;              // and in this shape
};
// For T rows of E experts, by time models; g: one expert's weight.
RowsPlan rows_plan(const Geometry& g, int64_t T, int64_t E, int cus);
// that of the gradients (16 bits), and how many of the weights' tiles take the time
// of one of the rows' (0: no rows')
int grads_tile_shape(const Geometry& g, int64_t T, int64_t E, bool dx, bool dw, int cus, int* lead);

// few rows an expert: the packed weights streamed once per unit of 16 rows or more
hipError_t launch_rows_decode(const RowsArgs& a, hipStream_t s);
// Its launch: 16-row tiles of a workgroup, waves along K, and workgroups.
void rows_decode_plan(const Geometry& g, int64_t T, int64_t E, int* nt, int* ks, int64_t* workgroups);
// Whether the streamed 8-bit product quantises T rows of E experts itself: what
// a workgroup keeps of them fits its LDS, and they are so few that quantising
// them in every workgroup takes less than a launch.  (One row, 11008 x 4096: 13.3
// us with a launch for it, 9.7 without; sixteen rows of one expert's 4096
// columns would take each workgroup 5 us, the launch takes 4.)
inline bool rows_decode_quantizes(int64_t T, int64_t E, int64_t K) {
  const int64_t Kp = i8_kp(K), some = T < E ? T : E;
  return T <= 16 && T * (Kp + 16) <= 48 * 1024 && (T + some - 1) / some * Kp <= 16 * 1024;
}
hipError_t launch_rows_decode_i8(const RowsArgs& a, hipStream_t s);
hipError_t launch_rows_decode_f16(const RowsArgs& a, hipStream_t s);
hipError_t launch_rows_decode_bf16(const RowsArgs& a, hipStream_t s);

// more rows an expert: the packed weights streamed once per 64 or 128 rows, which
// the workgroup's waves share (tm: 4 or 8 tiles of 16)
hipError_t launch_rows_wide(const RowsArgs& a, int tm, hipStream_t s);
hipError_t launch_rows_wide_i8(const RowsArgs& a, int tm, hipStream_t s);
hipError_t launch_rows_wide_f16(const RowsArgs& a, int tm, hipStream_t s);
hipError_t launch_rows_wide_bf16(const RowsArgs& a, int tm, hipStream_t s);

// Tile products of grouped rows.
//   TILE_ROWS  C[s][n] = sum_k A[s][k] B_e[n][k] for expert e's rows s (8 bits:
//              scaled, with bias and activation).  A [T] rows of lda bytes; B
//              in blocks of 16 rows x 128 bytes (sparse: packed 2:4 blocks of
//              64, with positions), nslab of them side by side, the blocks of
//              an expert's ceil(Nr / 16) x nslab one after another, then the
//              next expert's.
//   TILE_COLS  C_e[m][n] = keep (.) sum over expert e's rows t of A[t][m] B[t][n]:
//              rows of lda and ldb bytes, of which ka and kb 16-byte pieces count.
struct RowsTile : TileArgs {
  RowGroups rows;
  const uint8_t* meta;       // sparse TILE_ROWS
  const float* xscale;       // 8 bits: [T], [E][Nr]; bias [E][Nr] or nullptr
  const float* wscale;
  bool zero_rest;            // TILE_ROWS: rows of no expert become zeros
  int64_t es;                // TILE_COLS: elements between experts' outputs
  const uint8_t* mask;       // and kept bits, one block for 128 rows x 64 columns
  int64_t ldm;               // blocks along a row
};
// Kept bits as the weight gradients' lanes need them, 1 KB a block of 128 rows x
// 64 columns: 16 bytes of lane 16 lq + li, 16 bits a row tile j of them: bits 4 i + v
// of row 16 j + li, columns 16 i + 4 lq + v.
inline int64_t kept_blocks(int64_t R, int64_t nKB) { return (R + 127) / 128 * nKB; }
// TILE_ROWS; et: TILE_F16, TILE_BF16 (outputs of that type) or TILE_I8
hipError_t launch_rows_tile(int et, int ydt, const RowsTile& a, hipStream_t s);
// TILE_ROWS (x) and TILE_COLS (w), one launch in tiles of `shape`; C null: not that one
hipError_t launch_rows_grads(int et, const RowsTile& x, const RowsTile& w, int shape, hipStream_t s);
// TILE_ROWS on 2:4 weights
hipError_t launch_rows_tile24(int wdt, int ydt, const RowsTile& a, hipStream_t s);
constexpr int kRowsTable = 1024;   // boundaries (E + 1) a workgroup's table holds

// Packed weights -> the same blocks with every column (dense blocks of 16 rows
// x 128 bytes), for experts that have rows.
hipError_t launch_rows_dense(const Geometry& g, const uint8_t* values, const uint8_t* meta, const RowGroups& rows,
                             uint8_t* dense, hipStream_t s);

// Operands of the gradients (16-bit): each expert's weight transposed, in
// blocks as above (wt: K rows, Rp = R rounded up to 64 columns) where it has
// rows; its kept bits, mask [E][kept_blocks]; X and dY in rows of whole slabs of
// 64 columns, the last filled with zeros (xp, yp).  Null outputs are left out.
struct RowsPrepareArgs {
  Geometry g;
  RowGroups rows;
  const uint8_t* values;
  const uint8_t* meta;
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* dY;
  int64_t lddy;
  uint16_t* wt;
  uint8_t* mask;
  uint16_t* xp;
  uint16_t* yp;
};
hipError_t launch_rows_prepare(const RowsPrepareArgs& a, hipStream_t s);

// X [rows][ldx] of xdt -> elements [rows][i8_kp(K)] and scales [rows]; back
hipError_t launch_i8_quantize(const void* X, int64_t ldx, int xdt, int64_t rows, int64_t K, int8_t* codes,
                              float* scales, hipStream_t s);
hipError_t launch_i8_dequantize(const int8_t* codes, const float* scales, int64_t rows, int64_t K, void* Y,
                                int64_t ldy, int ydt, hipStream_t s);

// ---------------------------------------------------------------- device
#if defined(__HIP_DEVICE_COMPILE__)
// at[i], taken into [0, T]
__device__ __forceinline__ int row_bound(const RowGroups& o, int i) {
  if (!o.at) return i ? (int)o.T : 0;
  const int64_t v = o.wide ? static_cast<const int64_t*>(o.at)[i] : (int64_t)static_cast<const int32_t*>(o.at)[i];
  return (int)min(max(v, (int64_t)0), o.T);
}
// Inclusive scans over a wave by the vector unit's own lane moves (inside rows of
// 16 lanes, then a row's last lane to the next one, then lane 31 to the upper
// half); values are not negative.  By LDS exchanges a scan takes about 700 cycles.
template <class F>
__device__ __forceinline__ int wave_scan(int v, F&& op) {
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
  return op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
}
__device__ __forceinline__ int wave_scan_max(int v) {
  return wave_scan(v, [](int x, int y) { return max(x, y); });
}
__device__ __forceinline__ int wave_scan_add(int v) {
  return wave_scan(v, [](int x, int y) { return x + y; });
}

// Experts' first rows and first units (of U rows), a wave's lanes 64 boundaries at
// a time: f(i, from, at, unit, n) for the lane's boundary i: the expert in front of
// it has the rows from .. at - 1 and the units unit - n .. unit - 1 (i = 0 and i > E:
// none).  f returns whether to stop, the same in every lane.
template <int U, class F>
__device__ __forceinline__ void row_boundaries(const RowGroups& o, F&& f) {
  const int lane = threadIdx.x & 63;
  int last = 0, units = 0;                              // of the boundaries before this chunk
  for (int c = 0; c <= o.E; c += 64) {
    const int i = c + lane;
    int v = i <= o.E ? row_bound(o, i) : 0;
    v = max(wave_scan_max(v), last);
    int p = __builtin_amdgcn_update_dpp(0, v, 0x138, 0xf, 0xf, false);   // the lane before
    if (lane == 0) p = c ? last : v;
    int n = (v - p + U - 1) / U;
    if (i == 0 || i > o.E) n = 0;
    const int u = wave_scan_add(n) + units;
    if (f(i, p, v, u, n)) return;
    last = __builtin_amdgcn_readlane(v, 63);
    units = __builtin_amdgcn_readlane(u, 63);
  }
}

// Item L of the units of all experts times nt column tiles, expert by expert,
// an expert's units first (called by whole waves): the expert, the unit's first
// row, the expert's first row and end, the column tile; e < 0 where there are
// fewer items.
struct RowUnit {
  int e, row, begin, end, n;
};
template <int U>
__device__ __forceinline__ RowUnit find_unit(const RowGroups& o, int L, int nt = 1) {
  RowUnit r = {-1, 0, 0, 0, 0};
  if (!o.at) {
    const int units = (int)((o.T + U - 1) / U);
    r.n = __builtin_amdgcn_readfirstlane(L / units);
    r.row = (L - r.n * units) * U;
    r.end = (int)o.T;
    r.e = r.n < nt ? 0 : -1;
    return r;
  }
  row_boundaries<U>(o, [&](int i, int from, int at, int u, int n) {
    const uint64_t hit = __ballot(u * nt > L && (u - n) * nt <= L);
    if (!hit) return false;
    const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
    const int units = __builtin_amdgcn_readlane(n, l);
    const int in = L - __builtin_amdgcn_readlane(u - n, l) * nt;
    r.e = __builtin_amdgcn_readlane(i, l) - 1;
    r.begin = __builtin_amdgcn_readlane(from, l);
    r.end = __builtin_amdgcn_readlane(at, l);
    r.n = __builtin_amdgcn_readfirstlane(in / units);
    r.row = r.begin + (in - r.n * units) * U;
    return true;
  });
  return r;
}

// Units of all rows (called by whole waves).
template <int U>
__device__ __forceinline__ int count_units(const RowGroups& o) {
  if (!o.at) return (int)((o.T + U - 1) / U);
  int n = 0;
  row_boundaries<U>(o, [&](int, int, int, int u, int) {
    n = __builtin_amdgcn_readlane(u, 63);
    return false;
  });
  return n;
}

// The rows of no expert are those before `first` and from `last` on.
__device__ __forceinline__ void rows_taken(const RowGroups& o, int& first, int& last) {
  first = 0;
  last = (int)o.T;
  if (!o.at) return;
  first = row_bound(o, 0);
  last = first;
  for (int i = threadIdx.x & 63; i <= o.E; i += 64) last = max(last, row_bound(o, i));
  last = __builtin_amdgcn_readlane(wave_scan_max(last), 63);
}
#endif

}  // namespace nm
