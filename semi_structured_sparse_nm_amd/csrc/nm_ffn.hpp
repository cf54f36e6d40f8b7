// Shared definitions of the feed-forward operators (gated block on N:M packed
// weights and its backward pass; the microscaled 4-bit format, its product
// and its gated block).  Internal; the public surface is include/nm_sparse.h.
#pragma once

#include "nm_common.hpp"

namespace nm {

// a packed weight's descriptor, checked as nm_spmm checks it (nm_api.hip)
nm_status check_packed(const nm_packed* w, Geometry* g);

// ---------------------------------------------------------------- microscaled 4-bit layout
// rows x K values in blocks of 32 along K.  codes: row r at r * ldc bytes,
// ldc = Kp / 2, Kp = K rounded up to 256, element k in bits 4 (k % 2) .. of
// byte k / 2.  scales: one 256-byte unit for 32 rows x 256 columns, unit
// (r / 32) * (Kp / 256) + k / 256; inside it the block of row r, column k at
// byte 4 (16 (b % 4) + r % 16) + 2 ((r % 32) / 16) + b / 4, b = (k % 256) / 32:
// dword l of a unit holds the four scales that lane l of a wave needs for two
// 16-row tiles x two matrix instructions of 128 columns.
constexpr int kMxSlab = 256;                 // elements of K a unit covers
inline int64_t mx_kp(int64_t K) { return (K + kMxSlab - 1) / kMxSlab * kMxSlab; }
inline int64_t mx_codes_bytes(int64_t rows, int64_t K) { return rows * (mx_kp(K) / 2); }
inline int64_t mx_scales_bytes(int64_t rows, int64_t K) { return (rows + 31) / 32 * (mx_kp(K) / kMxSlab) * 256; }

// ---------------------------------------------------------------- tile product
// C[m][n] = sum_k A[m][k] B[n][k]: A the activations (rows = tokens, or
// weight rows in the weight gradient), B the weights, both with the reduction
// contiguous; a "slab" is 128 bytes of the reduction.
//   TILE_LINEAR  act(C + bias)
//   TILE_GLU     act(C0) * C1 over two weights
//   TILE_BACK    the gradients of the gated block in one launch: A B^T of the
//                fields below (16-bit, or binary32 slices where split > 1), and
//                A B^T of `w`, twice, where kept
enum TileOp { TILE_LINEAR = 0, TILE_GLU = 1, TILE_BACK = 2 };

struct TileGradArgs {
  const uint8_t* A[2];       // transposed dG, dU: [Mr] rows of ld bytes
  const uint8_t* B;          // X transposed: [Nr] rows of ld bytes
  int64_t ld, Mr, Nr;
  int nslab;
  void* C[2];                // nullptr: not computed
  int64_t ldc;
  const uint8_t* mask[2];    // bit k % 8 of byte k / 8 of row m says the weight is kept
  int64_t ldm;               // bytes
  int lead;                  // from plan_back
};

struct TileArgs {
  const uint8_t* A;          // lda bytes between rows
  const uint8_t* B[2];       // TILE_GLU: gate and up weights; else the first
  const uint8_t* As;         // scales (microscaled operands), unit layout above
  const uint8_t* Bs[2];
  int64_t lda, ldb;          // bytes
  int64_t Mr, Nr;            // rows of A, rows of B (of one of the two weights)
  int ka, kb;                // valid 16-byte pieces of an A row, of a B row
  int nslab;                 // slabs of the reduction
  void* C;                   // output, ldc elements between rows (TILE_BACK: nullptr, not computed)
  int64_t ldc;
  void* P[2];                // TILE_GLU: the two products (nullptr: not kept), ldp elements between rows
  int64_t ldp;
  bool p32;                  // in binary32, else the output's type
  const float* bias;         // [Nr] or nullptr
  int act;                   // NM_ACT_NONE / NM_ACT_GELU / NM_ACT_SILU
  int shape;                 // tile shape, from plan_tile or plan_back
  // split of the reduction (TILE_LINEAR, TILE_BACK): slice s covers slabs
  // s * sps .., raw sums to C + s * cs elements of binary32
  int split, sps;
  int64_t cs;
  TileGradArgs w;            // TILE_BACK
};

// Element types of the tile kernel's operands.
enum { TILE_F16 = 0, TILE_BF16 = 1, TILE_MX = 2 };

// Tile shape (0: 256 x 256, 1: 128 x 256, 2: 128 x 128, 3: 64 x 128) and slices
// of the reduction for one product, by a model of its time.
struct TilePlan {
  int shape, split, sps, lead;
  double time;               // microseconds, by the model
};
TilePlan plan_tile(TileOp op, bool mx, int64_t Mr, int64_t Nr, int nslab, int cus);
// The same for TILE_BACK's products of T tokens: T x K over 2 R and, twice, R x
// K over T, in slabs; lead: products of the second kind that a workgroup with
// one product less of the first takes ahead of the others.
TilePlan plan_back(int64_t T, int64_t R, int64_t K, int nslab_x, int nslab_w, bool dx, bool dw, int cus);
int device_cu_count();
// Workgroups of `block` threads for n items, at most 2^22 (a launch has fewer
// than 2^32 threads): kernels launched so loop over the rest.
inline unsigned grid_1d(int64_t n, int block) {
  const int64_t b = (n + block - 1) / block;
  return (unsigned)(b < (1 << 22) ? b : 1 << 22);
}
bool ffn_tile_override(const char* kind, int* shape, int* split);
// C[t][r] = act(sum over the slices + bias[r]), part [split][T][R] binary32
hipError_t launch_tile_reduce(const float* part, int split, int64_t T, int64_t R, const float* bias, int act, void* C,
                              int64_t ldc, int ydt, hipStream_t s);

hipError_t launch_tile_f16(TileOp op, int ydt, const TileArgs& a, hipStream_t s);
hipError_t launch_tile_bf16(TileOp op, int ydt, const TileArgs& a, hipStream_t s);
hipError_t launch_tile_mx(TileOp op, int ydt, const TileArgs& a, hipStream_t s);

// ---------------------------------------------------------------- other launches
struct GluArgs {
  Geometry g;                // both weights
  int wdt;
  const uint8_t* values[2];
  const uint8_t* meta[2];
  const void* X;
  int64_t ldx, T;
  void* H;
  int64_t ldh;
  void* P[2];                // the two products, as in TileArgs
  int64_t ldp;
  bool p32;
  int act;
};

// Tiles of 16 tokens (1, 2 or 4) that a workgroup of a streamed product takes:
// as many as there are, but fewer where the workgroups would leave half the
// compute units idle.
int stream_tiles(int64_t blocks, int64_t T);
// few tokens: the packed weights streamed once per token tile
hipError_t launch_glu_decode(const GluArgs& a, hipStream_t s);
// more tokens, both weights 2:4: the sparse tile product
hipError_t launch_glu_tile24(const GluArgs& a, hipStream_t s);
// its time in microseconds by the model its tile shape is chosen with
double glu_tile24_time(int64_t T, int64_t R, int64_t nslab, int cus, int* shape);

// Both packed weights -> dense [R][Kp] (Kp = K rounded up to 64, zero filled).
struct DenseArgs {
  const uint8_t* values[2];
  const uint8_t* meta[2];
  uint16_t* dense[2];
};
hipError_t launch_expand_dense(const Geometry& g, const DenseArgs& a, hipStream_t s);

// The backward pass's operands (16-bit): from G and U, in the weights' type or
// binary32 (p32), and dH, dG = dH u act'(g) and dU = dH act(g) as rows d [T][2 Rp]
// (gate at column 0, up at Rp, zeros from R to Rp) and transposed dt [2][R][Tp];
// both weights transposed, wt [K][2 Rp]; their kept bits, mask[w] [R][Kp / 8]; X
// transposed, xt [K][Tp].  Rp, Tp, Kp: R, T, K rounded up to 64, zero filled.  Null
// outputs are left out.  parts = 2 (with p32): what the rounding of dG and dU
// left, rounded too, follows them along the reductions, d [T][4 Rp] and dt
// [2][R][2 Tp], and the other operands come twice, wt [K][4 Rp] and xt [K][2 Tp]:
// the same products add both.
struct PrepareArgs {
  Geometry g;
  const uint8_t* values[2];
  const uint8_t* meta[2];
  const uint16_t* X;
  int64_t ldx, T;
  const void* G;
  const void* U;
  int64_t ldp;
  bool p32;
  const uint16_t* dH;
  int64_t lddh;
  int act;
  int64_t Rp, Tp;
  int parts;
  uint16_t* d;
  uint16_t* dt;
  uint16_t* wt;
  uint16_t* xt;
  uint8_t* mask[2];
};
hipError_t launch_glu_prepare(const PrepareArgs& a, int wdt, hipStream_t s);
// copy of X [T][ldx] with rows of Kp elements, zeros past K
hipError_t launch_pad_rows(const void* X, int64_t ldx, int64_t T, int64_t K, void* Y, int64_t Kp, hipStream_t s);

hipError_t launch_mx_quantize(const void* X, int64_t ldx, int xdt, int64_t rows, int64_t K, uint8_t* codes,
                              uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* Y,
                                int64_t ldy, int ydt, hipStream_t s);

struct MxDecodeArgs {
  const uint8_t* codes[2];   // one weight, or gate and up
  const uint8_t* scales[2];
  int64_t R, K;
  const void* X;             // 16- or 32-bit activations, quantised in registers ...
  int64_t ldx;
  int xdt;
  const uint8_t* xcodes;     // ... or (X null) already quantised
  const uint8_t* xscales;
  int64_t T;
  void* Y;
  int64_t ldy;
  int ydt;
  const float* bias;
  int act;
  bool glu;
};
hipError_t launch_mx_decode(const MxDecodeArgs& a, hipStream_t s);

// ---------------------------------------------------------------- device
// SiLU(x) = x / (1 + exp(-x)), binary32: exp2 and reciprocal of the
// transcendental unit (1 ulp each); exp's rounded argument adds 2^-24 |x|
// relative, so the error stays below 2^-22 (1 + |x|) |SiLU(x)|, far below
// half a 16-bit step.  With q = exp(-|x| / 2), r = 1 / (1 + q^2) and p = q for
// negative x, else 1, the sigmoid is p^2 r: multiplied in this order nothing
// leaves binary32's range before the result does (x / (1 + exp(-x)) as it stands
// is 0 below x = -88.7, where SiLU is a normal number down to -91.8; gated
// block of 2048 tokens, 11008 x 4096: 212 us, 209 with it as it stands, 211 with
// a branch for the far values).
__device__ __forceinline__ void sigmoid_parts(float x, float& p, float& r) {
  const float q = __builtin_amdgcn_exp2f(__builtin_fabsf(x) * -0.72134752044448170368f);
  r = __builtin_amdgcn_rcpf(__builtin_fmaf(q, q, 1.0f));
  p = x < 0.0f ? q : 1.0f;
}
__device__ __forceinline__ float silu_f32(float x) {
  float p, r;
  sigmoid_parts(x, p, r);
  return (x * p) * (p * r);
}

// act(x) and act'(x) of the gated block (NM_ACT_GELU or NM_ACT_SILU)
__device__ __forceinline__ float glu_act(int act, float x) { return act == NM_ACT_SILU ? silu_f32(x) : gelu_f32(x); }
__device__ __forceinline__ void glu_act_slope(int act, float x, float& y, float& dy) {
  if (act == NM_ACT_SILU) {
    float p, r;
    sigmoid_parts(x, p, r);
    y = (x * p) * (p * r);
    const float s = p * (p * r);
    dy = s * (1.0f + x * (1.0f - s));
  } else {
    const float cdf = 0.5f * (1.0f + erf_as(x * 0.70710678118654752440f));
    y = x * cdf;
    // x phi(x), phi the normal density
    dy = cdf + x * 0.39894228040143267794f * __builtin_amdgcn_exp2f(-0.5f * 1.44269504088896341f * x * x);
  }
}

// two binary32 -> packed 16-bit floats, round to nearest even
typedef float v2f_ __attribute__((ext_vector_type(2)));
typedef _Float16 v2h_ __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf_ __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ uint32_t pack_16x2(float lo, float hi) {
  if constexpr (DT == NM_F16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f_{lo, hi}), v2h_));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f_{lo, hi}), v2bf_));
}
// infinities as the 16-bit type's largest value of their sign (NaN stays)
template <int DT>
__device__ __forceinline__ float finite_16(float x) {
  constexpr float top = DT == NM_F16 ? 65504.f : 0x1.FEp127f;
  return __builtin_fabsf(x) > top ? __builtin_copysignf(top, x) : x;
}
template <int DT>
__device__ __forceinline__ float from_16(uint32_t bits) {
  if constexpr (DT == NM_F16)
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  else
    return __builtin_bit_cast(float, bits << 16);
}

// 16 and 8 bytes of a row that starts at any element: global memory takes wide
// accesses at any address (the product of 1508 x 1602 x 2304 at 4 bits: 14.8 us
// with rows written element by element, 10.6 so).
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));
typedef int v2i_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ v4i load16(const void* p) { return *static_cast<const v4i_any*>(p); }

// Eight 16-bit values without their first n (zeros follow), by dwords and then
// half a dword.  No 64-bit shifts: one whose amount is in a wave's last vector
// register (v15 of 16, as the compiler placed it here) now and then shifts by
// another amount on this chip.
__device__ __forceinline__ v4i shift_out(v4i x, int n) {
  if (n & 4) x = v4i{x[2], x[3], 0, 0};
  if (n & 2) x = v4i{x[1], x[2], x[3], 0};
  if (n & 1)
    x = v4i{(int)((uint32_t)x[0] >> 16 | (uint32_t)x[1] << 16), (int)((uint32_t)x[1] >> 16 | (uint32_t)x[2] << 16),
            (int)((uint32_t)x[2] >> 16 | (uint32_t)x[3] << 16), (int)((uint32_t)x[3] >> 16)};
  return x;
}
// Eight 16-bit elements i .. i + 7 of a row of n, zeros past its end (i < n): a
// short last piece is read as the row's last eight and shifted.
__device__ __forceinline__ v4i load_piece(const uint16_t* row, int64_t i, int64_t n) {
  if (i + 8 <= n) return load16(row + i);
  if (n >= 8) return shift_out(load16(row + n - 8), (int)(i + 8 - n));
  v4i x = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) x[e >> 1] |= (int)((uint32_t)row[e] << (16 * (e & 1)));
  return x;
}

// Four consecutive outputs y[0..3] of a row at element offset o; `n` of them
// (1..4) exist.
template <int DT>
__device__ __forceinline__ void store4(void* Y, int64_t o, const float* y, int n) {
  if constexpr (DT == NM_F32) {
    float* p = static_cast<float*>(Y) + o;
    if (n == 4) {
      *reinterpret_cast<v4f_any*>(p) = v4f_any{y[0], y[1], y[2], y[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = y[i];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(Y) + o;
    const uint32_t a = pack_16x2<DT>(y[0], y[1]), b = pack_16x2<DT>(y[2], y[3]);
    if (n == 4) {
      *reinterpret_cast<v2i_any*>(p) = v2i_any{(int)a, (int)b};
    } else {
      p[0] = (uint16_t)a;
      if (n > 1) p[1] = (uint16_t)(a >> 16);
      if (n > 2) p[2] = (uint16_t)b;
    }
  }
}

}  // namespace nm
