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
// ones, and a count of outstanding loads could pass too early (TILE_COLS: while a
// slab that ends inside is on its way, all loads are waited for).  TILE_GLU: half of
// a wave's B rows are gate rows, the other half the up rows of the same outputs, so
// g and u of one output meet in one lane and the activation and product need no
// exchange.  TILE_BACK: the input's and both weights' gradients are items of one
// launch; those of grouped rows are TILE_ROWS, then TILE_COLS items of one.
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

#include <algorithm>

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

constexpr bool grouped_op(int op) { return op == TILE_ROWS || op == TILE_COLS; }
template <int OP>
using tile_args = typename std::conditional<grouped_op(OP), RowsTile, TileArgs>::type;

// Bytes of LDS.
template <int ET, int OP, int BM, int BN, int NS>
constexpr int tile_lds() {
  return NS * ((BM + BN) * (ET == TILE_MX ? 136 : 128)) + rows_table_bytes(grouped_op(OP), kRowsTable);
}

#if defined(__HIP_DEVICE_COMPILE__)
// The kernel's body as a function, for the kernel that runs two operations.  (Not for
// the others: as a function's arguments those of TILE_BACK, which chooses between
// fields, pass through scratch memory, and resources from there are in vector
// registers, which the loads do not take.)
template <int ET, int OP, int OUT, int BM, int BN, int WM, int WN, int NS>
__device__ __forceinline__ int tile_items(const tile_args<OP>& a, const TileList& list, const TileList& list2,
                                          uint8_t* lds, int first) {
#define TILE_RETURN return more
#include "nm_tile_body.hpp"
#undef TILE_RETURN
  return more;
}
#endif

template <int ET, int OP, int OUT, int BM, int BN, int WM, int WN, int NS>
__global__ void __launch_bounds__(WM * WN * 64) __attribute__((amdgpu_waves_per_eu(2, 2)))
tile_kernel(tile_args<OP> a, TileList list, TileList list2) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) uint8_t lds[tile_lds<ET, OP, BM, BN, NS>()];
  constexpr int first = 0;
#define TILE_RETURN return
#include "nm_tile_body.hpp"
#undef TILE_RETURN
#endif
}

// Gradients of grouped rows: the rows' (x), then the weights' (w), of which those
// workgroups get more that had an item less of x's.  Either's C may be null.
template <int ET, int OUT, int BM, int BN, int WM, int WN, int NS>
__global__ void __launch_bounds__(WM * WN * 64) __attribute__((amdgpu_waves_per_eu(2, 2)))
tile_grads_kernel(RowsTile x, RowsTile w, TileList lx, TileList lw) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) uint8_t lds[tile_lds<ET, TILE_ROWS, BM, BN, NS>()];
  int more = 0;
  if (x.C) {
    more = tile_items<ET, TILE_ROWS, OUT, BM, BN, WM, WN, NS>(x, lx, lx, lds, 0);
    __syncthreads();
  }
  if (w.C) tile_items<ET, TILE_COLS, OUT, BM, BN, WM, WN, NS>(w, lw, lw, lds, more);
#endif
}

// The list of a product of grouped rows: as many items as there could be (the host
// does not know the experts' rows).
template <int OP, int BM, int BN>
TileList rows_list(const RowsTile& a) {
  TileList l{};
  if (!a.C) return l;
  l.mt = (int)((a.Mr + BM - 1) / BM);
  l.nt = (int)((a.Nr + BN - 1) / BN);
  const int64_t most = (OP == TILE_COLS ? (int64_t)l.mt * a.rows.E : units_most(a.rows.T, a.rows.E, BM)) * l.nt;
  l.per = (int)std::min<int64_t>((most + 7) / 8, 1 << 20);
  return l;
}

template <int ET, int OP, int OUT, int BM, int BN, int WM, int WN, int NS>
hipError_t launch_tile_cfg(const tile_args<OP>& a, hipStream_t s) {
  constexpr int BNO = OP == TILE_GLU ? BN / 2 : BN;
  if constexpr (OP == TILE_ROWS) {
    const TileList l = rows_list<OP, BM, BN>(a);
    hipLaunchKernelGGL((tile_kernel<ET, OP, OUT, BM, BN, WM, WN, NS>), dim3(8u * tile_slots(l.per)),
                       dim3(WM * WN * 64), 0, s, a, l, l);
    return hipGetLastError();
  } else {
    const bool back = OP == TILE_BACK;
    const TileList list = tile_list(a.Mr, a.Nr, BM, BNO, a.split, a.sps, a.nslab, back && !a.C ? 0 : 1);
    const TileList list2 = tile_list(a.w.Mr, a.w.Nr, BM, BNO, 1, a.w.nslab, a.w.nslab, back && a.w.C[0] ? 2 : 0);
    const int grid = 8 * tile_slots(list.per + list2.per);
    hipLaunchKernelGGL((tile_kernel<ET, OP, OUT, BM, BN, WM, WN, NS>), dim3((unsigned)grid), dim3(WM * WN * 64), 0, s,
                       a, list, list2);
    return hipGetLastError();
  }
}

template <int ET, int OUT, int BM, int BN, int WM, int WN, int NS>
hipError_t launch_grads_cfg(const RowsTile& x, const RowsTile& w, hipStream_t s) {
  const TileList lx = rows_list<TILE_ROWS, BM, BN>(x), lw = rows_list<TILE_COLS, BM, BN>(w);
  hipLaunchKernelGGL((tile_grads_kernel<ET, OUT, BM, BN, WM, WN, NS>), dim3(8u * tile_slots(lx.per + lw.per)),
                     dim3(WM * WN * 64), 0, s, x, w, lx, lw);
  return hipGetLastError();
}
template <int ET, int OUT>
hipError_t launch_grads(const RowsTile& x, const RowsTile& w, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch_grads_cfg<ET, OUT, 256, 256, 2, 4, 2>(x, w, s);
    case 1: return launch_grads_cfg<ET, OUT, 128, 256, 2, 4, 3>(x, w, s);
    case 2: return launch_grads_cfg<ET, OUT, 128, 128, 2, 4, 4>(x, w, s);
    default: return launch_grads_cfg<ET, OUT, 64, 128, 2, 4, 6>(x, w, s);
  }
}

template <int ET, int OP, int OUT>
hipError_t launch_tile_op(const tile_args<OP>& a, hipStream_t s) {
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
