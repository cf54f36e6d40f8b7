// C ABI of the 8-bit rows, their product, and the products of rows grouped by
// expert (include/nm_sparse.h): host-side validation, choice of the path per
// shape, launches.  Stateless and thread-safe.
#include <algorithm>

#include "nm_rows.hpp"

using nm::Geometry;
using nm::RowGroups;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t up64(int64_t n) { return (n + 63) / 64 * 64; }
// rows the tile kernels address with 32-bit offsets: 256 of them within 2^31 bytes
constexpr int64_t kMaxStride = 1ll << 23;
bool row_ok(int64_t row_bytes) { return row_bytes < kMaxStride; }
bool float_dtype(int32_t dt) { return dt == NM_F16 || dt == NM_BF16 || dt == NM_F32; }

constexpr int64_t kMaxLen = 1ll << 25;      // rows
constexpr int64_t kMaxOut = 1ll << 22;      // outputs R
constexpr int64_t kMaxGrid = 1ll << 24;     // workgroups: a launch has fewer than 2^32 threads
constexpr int64_t kMaxK8 = 131071;          // 2^31 / 128^2 products of 8-bit numbers

// ---------------------------------------------------------------- descriptors
nm_status check_i8(const nm_i8* q) {
  if (!q || q->rows < 1 || q->K < 1 || !q->codes || !q->scales) return NM_EINVAL;
  if (q->K > kMaxK8 || q->rows > (1ll << 40) / q->K) return NM_EUNSUPPORTED;
  if ((int64_t)q->codes_bytes != q->rows * nm::i8_kp(q->K) || (int64_t)q->scales_bytes != q->rows * 4) return NM_EINVAL;
  if (!aligned(q->codes, 16) || !aligned(q->scales, 4)) return NM_EUNSUPPORTED;
  return NM_OK;
}

// the weights of a call: one packed weight, or one an expert
struct Weights {
  Geometry g;                // of one expert
  int dtype;
  const uint8_t* values;
  const uint8_t* meta;
  int64_t E;
};

nm_status weights_of(const nm_packed* w, Weights* o) {
  const nm_status st = nm::check_packed(w, &o->g);
  if (st != NM_OK) return st;
  if (w->format_version != NM_FORMAT_VERSION) return NM_EINVAL;
  o->dtype = w->dtype;
  o->values = static_cast<const uint8_t*>(w->values);
  o->meta = static_cast<const uint8_t*>(w->meta);
  o->E = 1;
  return NM_OK;
}

// (version 0 is a weight not packed yet)
nm_status weights_of(const nm_experts* w, Weights* o, bool packed = true) {
  if (!w || w->experts < 1) return NM_EINVAL;
  if (w->experts > nm::kMaxExperts) return NM_EUNSUPPORTED;
  const int64_t E = w->experts;
  if (w->values_bytes % E || w->meta_bytes % E) return NM_EINVAL;
  nm_packed p{w->rows, w->K,      w->N,    w->M, w->dtype, w->format_version, w->values, w->values_bytes / E,
              w->meta, w->meta_bytes / E};
  const nm_status st = nm::check_packed(&p, &o->g);
  if (st != NM_OK) return st;
  if (packed && w->format_version != NM_FORMAT_VERSION) return NM_EINVAL;
  o->dtype = w->dtype;
  o->values = static_cast<const uint8_t*>(w->values);
  o->meta = static_cast<const uint8_t*>(w->meta);
  o->E = E;
  return NM_OK;
}

nm_status check_sizes(const Weights& w, int64_t T) {
  if (T < 1) return NM_EINVAL;
  const Geometry& g = w.g;
  if (T > kMaxLen || g.R > kMaxOut || !row_ok(g.nKB * 128)) return NM_EUNSUPPORTED;
  if (w.dtype == NM_I8 && g.K > kMaxK8) return NM_EUNSUPPORTED;
  // the smallest tiles of a launch, counted in 32 bits; a copy's threads
  if ((double)nm::units_most(T, w.E, 64) * (double)((g.R + 127) / 128) >= 2e9) return NM_EUNSUPPORTED;
  if (w.E * g.nRB * g.nKB >= (1ll << 31)) return NM_EUNSUPPORTED;
  return NM_OK;
}

// ---------------------------------------------------------------- paths
using nm::ROWS_DENSE;
using nm::ROWS_REPACK;
using nm::ROWS_STREAM;
using nm::ROWS_WIDE;
using nm::RowsPath;
using nm::RowsPlan;

Geometry geometry24(const Geometry& g) { return Geometry::make(g.R, g.K, 2, 4, g.eb); }
RowsPlan plan_of(const Weights& w, int64_t T) { return nm::rows_plan(w.g, T, w.E, nm::device_cu_count()); }

int tile_type(int dt) { return dt == NM_I8 ? nm::TILE_I8 : dt == NM_F16 ? nm::TILE_F16 : nm::TILE_BF16; }

// Whether a 16-bit path's kernel reads X's rows as they are.  Streamed: any rows
// of at least one 16-byte piece, wide: of whole ones; tiles: 16-byte pieces, none of which crosses
// the end of a row, and 32-bit offsets.
bool rows_direct(RowsPath path, const void* X, int64_t ldx, int64_t K) {
  if (path == ROWS_STREAM) return K >= 8;
  if (path == ROWS_WIDE) return K % 8 == 0 && row_ok(ldx * 2);
  return aligned(X, 16) && ldx % 8 == 0 && K % 8 == 0 && row_ok(ldx * 2);
}
size_t padded_bytes(int64_t T, int64_t K) { return up256((size_t)(T * up64(K) * 2)); }

size_t repacked_values(const Weights& w) { return up256((size_t)w.E * geometry24(w.g).values_bytes()); }
size_t copies_bytes(const Weights& w, RowsPath path) {
  if (path == ROWS_REPACK) return repacked_values(w) + up256((size_t)w.E * geometry24(w.g).meta_bytes());
  if (path == ROWS_DENSE && w.g.N != w.g.M) return up256((size_t)(w.E * w.g.nRB * w.g.nKB * 2048));
  return 0;
}
size_t codes_bytes(int64_t T, int64_t K) { return up256((size_t)(T * nm::i8_kp(K))); }
size_t quantized_bytes(int64_t T, int64_t K) { return codes_bytes(T, K) + up256((size_t)T * 4); }

// The product of rows already in the kernels' form (a.X, a.ldx; ka: valid
// 16-byte pieces of a row); `ws`: copies_bytes of workspace.
hipError_t multiply(const Weights& w, const RowsPlan& plan, const nm::RowsArgs& a, int ka, uint8_t* ws, hipStream_t s) {
  const Geometry& g = w.g;
  const RowsPath path = plan.path;
  if (path == ROWS_STREAM) return nm::launch_rows_decode(a, s);
  if (path == ROWS_WIDE) return nm::launch_rows_wide(a, plan.shape, s);
  nm::RowsTile t{};
  t.rows = a.rows;
  t.A = static_cast<const uint8_t*>(a.X);
  t.lda = a.ldx * g.eb;
  t.ka = ka;
  t.B[0] = w.values;
  t.meta = w.meta;
  t.Mr = a.rows.T;
  t.Nr = g.R;
  t.nslab = (int)g.nKB;
  t.C = a.Y;
  t.ldc = a.ldy;
  t.xscale = a.xscale;
  t.wscale = a.wscale;
  t.bias = a.bias;
  t.act = a.act;
  t.zero_rest = a.zero_rest;
  t.shape = plan.shape;
  hipError_t e = hipSuccess;
  if (path == ROWS_REPACK) {
    // the blocks of all experts as one weight's
    const Geometry from = Geometry::make(w.E * g.nRB * 16, g.K, g.N, g.M, g.eb);
    uint8_t* meta = ws + repacked_values(w);
    e = nm::launch_repack24(from, w.values, w.meta, geometry24(from), ws, meta, s);
    t.B[0] = ws;
    t.meta = meta;
  } else if (path == ROWS_DENSE && g.N != g.M) {
    e = nm::launch_rows_dense(g, w.values, w.meta, a.rows, ws, s);
    t.B[0] = ws;
  }
  if (e != hipSuccess) return e;
  auto launch = [&] {
    return path == ROWS_DENSE ? nm::launch_rows_tile(tile_type(w.dtype), a.ydt, t, s)
                              : nm::launch_rows_tile24(w.dtype, a.ydt, t, s);
  };
  if (!plan.cut) return launch();
  t.Nr = plan.cut;
  e = launch();
  if (e != hipSuccess) return e;
  const int64_t blocks = plan.cut / 16 * g.nKB;
  const Geometry tg = path == ROWS_DENSE ? g : geometry24(g);
  t.B[0] += blocks * (path == ROWS_DENSE ? 2048 : tg.vblk);
  if (path != ROWS_DENSE) t.meta += blocks * tg.mblk;
  t.C = static_cast<uint8_t*>(t.C) + plan.cut * nm::dtype_bytes(a.ydt);
  if (t.wscale) t.wscale += plan.cut;
  if (t.bias) t.bias += plan.cut;
  t.Nr = g.R - plan.cut;
  t.shape = plan.rest;
  return launch();
}

// ---------------------------------------------------------------- 8-bit products
bool quantizes_inside(const Weights& w, RowsPath path, int64_t T) {
  return path == ROWS_STREAM && nm::rows_decode_quantizes(T, w.E, w.g.K);
}

nm_status i8_workspace(const Weights& w, const nm_i8* xq, int64_t T, size_t* bytes) {
  if (!bytes) return NM_EINVAL;
  if (w.dtype != NM_I8) return NM_EUNSUPPORTED;
  const nm_status st = check_sizes(w, T);
  if (st != NM_OK) return st;
  const RowsPath path = plan_of(w, T).path;
  *bytes = (xq || quantizes_inside(w, path, T) ? 0 : quantized_bytes(T, w.g.K)) + copies_bytes(w, path);
  return NM_OK;
}

nm_status i8_product(const Weights& w, const float* w_scale, const nm_i8* xq, const void* X, int64_t ldx, int32_t xdt,
                     int64_t T, const RowGroups& rows, void* Y, int64_t ldy, int32_t ydt, const float* bias,
                     int32_t act, bool zero_rest, void* workspace, size_t ws_bytes, void* stream) {
  if (w.dtype != NM_I8) return NM_EUNSUPPORTED;
  nm_status st = check_sizes(w, T);
  if (st != NM_OK) return st;
  const Geometry& g = w.g;
  if (!w_scale || !Y || ldy < g.R) return NM_EINVAL;
  if (!float_dtype(ydt) || (act != NM_ACT_NONE && act != NM_ACT_GELU)) return NM_EUNSUPPORTED;
  if (!aligned(Y, (size_t)nm::dtype_bytes(ydt)) || !aligned(w_scale, 4) || (bias && !aligned(bias, 4)))
    return NM_EUNSUPPORTED;
  if (xq) {
    st = check_i8(xq);
    if (st != NM_OK) return st;
    if (xq->format_version != NM_FORMAT_VERSION || xq->rows != T || xq->K != g.K) return NM_EINVAL;
  } else {
    if (!X || ldx < g.K) return NM_EINVAL;
    if (!float_dtype(xdt) || !aligned(X, (size_t)nm::dtype_bytes(xdt))) return NM_EUNSUPPORTED;
  }
  const RowsPlan plan = plan_of(w, T);
  const bool inside = !xq && quantizes_inside(w, plan.path, T);
  const size_t quant = xq || inside ? 0 : quantized_bytes(T, g.K), need = quant + copies_bytes(w, plan.path);
  if (need && (!workspace || ws_bytes < need)) return NM_EINVAL;
  if (need && !aligned(workspace, 256)) return NM_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  const int64_t Kp = nm::i8_kp(g.K);
  nm::RowsArgs a{};
  a.g = g;
  a.xdt = NM_I8;
  a.ldx = Kp;
  if (inside) {
    a.X = X;
    a.ldx = ldx;
    a.xdt = xdt;
  } else if (xq) {
    a.X = xq->codes;
    a.xscale = static_cast<const float*>(xq->scales);
  } else {
    float* scales = reinterpret_cast<float*>(ws + codes_bytes(T, g.K));
    if (nm::launch_i8_quantize(X, ldx, xdt, T, g.K, reinterpret_cast<int8_t*>(ws), scales, s) != hipSuccess)
      return NM_EHIP;
    a.X = ws;
    a.xscale = scales;
  }
  if (!inside) a.g.K = Kp;                              // a row's zeros may be read
  a.wdt = NM_I8;
  a.values = w.values;
  a.meta = w.meta;
  a.rows = rows;
  a.wscale = w_scale;
  a.bias = bias;
  a.act = act;
  a.Y = Y;
  a.ldy = ldy;
  a.ydt = ydt;
  a.zero_rest = zero_rest;
  return multiply(w, plan, a, (int)(Kp / 16), ws + quant, s) == hipSuccess ? NM_OK : NM_EHIP;
}

nm_status check_offsets(const void* offsets, int32_t dtype) {
  if (!offsets) return NM_EINVAL;
  if (dtype != NM_OFFSETS_I32 && dtype != NM_OFFSETS_I64) return NM_EUNSUPPORTED;
  return aligned(offsets, dtype == NM_OFFSETS_I64 ? 8 : 4) ? NM_OK : NM_EUNSUPPORTED;
}
RowGroups groups_of(const void* offsets, int32_t dtype, int64_t E, int64_t T) {
  return RowGroups{offsets, dtype == NM_OFFSETS_I64, (int)E, T};
}

// ---------------------------------------------------------------- gradients
struct BackwardPlan {
  size_t wt, mask, xp, yp, total;            // bytes of each part
  BackwardPlan(const Weights& w, int64_t T, bool dx, bool dw, bool pad_x, bool pad_y) {
    const Geometry& g = w.g;
    wt = dx ? up256((size_t)(w.E * ((g.K + 15) / 16) * (up64(g.R) / 64) * 2048)) : 0;
    mask = dw ? (size_t)(w.E * nm::kept_blocks(g.R, g.nKB) * 1024) : 0;
    xp = dw && pad_x ? padded_bytes(T, g.K) : 0;
    yp = pad_y ? padded_bytes(T, g.R) : 0;
    total = wt + mask + xp + yp;
  }
};

// that of a call with these rows
BackwardPlan backward_plan(const Weights& w, const void* X, int64_t ldx, int64_t T, const void* dY, int64_t lddy,
                           bool dx, bool dw) {
  return BackwardPlan(w, T, dx, dw, !rows_direct(ROWS_DENSE, X, ldx, w.g.K), !rows_direct(ROWS_DENSE, dY, lddy, w.g.R));
}

nm_status check_backward(const Weights& w, int64_t T) {
  if (w.dtype == NM_I8) return NM_EUNSUPPORTED;
  const nm_status st = check_sizes(w, T);
  if (st != NM_OK) return st;
  const Geometry& g = w.g;
  if (!row_ok(up64(g.R) * 2)) return NM_EUNSUPPORTED;
  if (w.E * nm::kept_blocks(g.R, g.nKB) + 2 * 4096 >= kMaxGrid) return NM_EUNSUPPORTED;
  return NM_OK;
}

}  // namespace

extern "C" {

nm_status nm_i8_size(int64_t rows, int64_t K, size_t* codes_bytes, size_t* scales_bytes) {
  if (!codes_bytes || !scales_bytes || rows < 1 || K < 1) return NM_EINVAL;
  if (K > kMaxK8 || rows > (1ll << 40) / K) return NM_EUNSUPPORTED;
  *codes_bytes = (size_t)(rows * nm::i8_kp(K));
  *scales_bytes = (size_t)rows * 4;
  return NM_OK;
}

nm_status nm_i8_quantize(const void* X, int64_t ldx, int32_t x_dtype, nm_i8* q, void* stream) {
  const nm_status st = check_i8(q);
  if (st != NM_OK) return st;
  if (!X || ldx < q->K) return NM_EINVAL;
  if (!float_dtype(x_dtype) || !aligned(X, (size_t)nm::dtype_bytes(x_dtype))) return NM_EUNSUPPORTED;
  if (nm::launch_i8_quantize(X, ldx, x_dtype, q->rows, q->K, static_cast<int8_t*>(q->codes),
                             static_cast<float*>(q->scales), static_cast<hipStream_t>(stream)) != hipSuccess)
    return NM_EHIP;
  q->format_version = NM_FORMAT_VERSION;
  q->reserved = 0;
  return NM_OK;
}

nm_status nm_i8_dequantize(const nm_i8* q, void* Y, int64_t ldy, int32_t y_dtype, void* stream) {
  const nm_status st = check_i8(q);
  if (st != NM_OK) return st;
  if (q->format_version != NM_FORMAT_VERSION || !Y || ldy < q->K) return NM_EINVAL;
  if (!float_dtype(y_dtype) || !aligned(Y, (size_t)nm::dtype_bytes(y_dtype))) return NM_EUNSUPPORTED;
  return nm::launch_i8_dequantize(static_cast<const int8_t*>(q->codes), static_cast<const float*>(q->scales), q->rows,
                                  q->K, Y, ldy, y_dtype, static_cast<hipStream_t>(stream)) == hipSuccess
             ? NM_OK
             : NM_EHIP;
}

nm_status nm_i8_linear_workspace_size(const nm_packed* w, const nm_i8* xq, int64_t T, size_t* bytes) {
  Weights ww;
  const nm_status st = weights_of(w, &ww);
  return st != NM_OK ? st : i8_workspace(ww, xq, T, bytes);
}

nm_status nm_i8_linear(const nm_packed* w, const float* w_scale, const nm_i8* xq, const void* Xt, int64_t ldx,
                       int32_t x_dtype, int64_t T, void* Yt, int64_t ldy, int32_t y_dtype, const float* bias,
                       int32_t act, void* workspace, size_t workspace_bytes, void* stream) {
  Weights ww;
  const nm_status st = weights_of(w, &ww);
  if (st != NM_OK) return st;
  return i8_product(ww, w_scale, xq, Xt, ldx, x_dtype, T, RowGroups{nullptr, 0, 1, T}, Yt, ldy, y_dtype, bias, act,
                    false, workspace, workspace_bytes, stream);
}

nm_status nm_experts_size(int64_t experts, int64_t rows, int64_t K, int32_t N, int32_t M, int32_t dtype,
                          size_t* values_bytes, size_t* meta_bytes) {
  if (experts < 1) return NM_EINVAL;
  if (experts > nm::kMaxExperts) return NM_EUNSUPPORTED;
  const nm_status st = nm_pack_size(rows, K, N, M, dtype, values_bytes, meta_bytes);
  if (st != NM_OK) return st;
  *values_bytes *= (size_t)experts;
  *meta_bytes *= (size_t)experts;
  return NM_OK;
}

nm_status nm_experts_pack(const void* W, int64_t lde, int64_t ldw, nm_experts* w, void* stream) {
  Weights ww;
  const nm_status st = weights_of(w, &ww, false);
  if (st != NM_OK) return st;
  if (!W || ldw < w->K || lde < 0) return NM_EINVAL;
  const size_t vb = w->values_bytes / ww.E, mb = w->meta_bytes / ww.E;
  for (int64_t e = 0; e < ww.E; ++e) {
    nm_packed p{w->rows, w->K, w->N, w->M, w->dtype, 0, static_cast<uint8_t*>(w->values) + e * vb, vb,
                w->meta ? static_cast<uint8_t*>(w->meta) + e * mb : nullptr, mb};
    const nm_status se = nm_pack(static_cast<const uint8_t*>(W) + e * lde * ww.g.eb, ldw, &p, stream);
    if (se != NM_OK) return se;
  }
  w->format_version = NM_FORMAT_VERSION;
  return NM_OK;
}

nm_status nm_expert_linear_workspace_size(const nm_experts* w, const void* Xt, int64_t ldx, int64_t T, size_t* bytes) {
  Weights ww;
  nm_status st = weights_of(w, &ww);
  if (st != NM_OK) return st;
  if (!bytes) return NM_EINVAL;
  if (ww.dtype == NM_I8) return NM_EUNSUPPORTED;
  st = check_sizes(ww, T);
  if (st != NM_OK) return st;
  if (Xt && ldx < ww.g.K) return NM_EINVAL;
  const RowsPath path = plan_of(ww, T).path;
  // NULL: the worst rows, at an odd address and farther apart than 32-bit offsets reach
  const bool direct = Xt ? rows_direct(path, Xt, ldx, ww.g.K)
                         : rows_direct(path, reinterpret_cast<const void*>(2), kMaxStride, ww.g.K);
  *bytes = (direct ? 0 : padded_bytes(T, ww.g.K)) + copies_bytes(ww, path);
  return NM_OK;
}

nm_status nm_expert_linear(const nm_experts* w, const void* Xt, int64_t ldx, int64_t T, const void* offsets,
                           int32_t offsets_dtype, void* Yt, int64_t ldy, int32_t zero_rest, void* workspace,
                           size_t workspace_bytes, void* stream) {
  Weights ww;
  nm_status st = weights_of(w, &ww);
  if (st != NM_OK) return st;
  if (ww.dtype == NM_I8) return NM_EUNSUPPORTED;
  st = check_sizes(ww, T);
  if (st != NM_OK) return st;
  const Geometry& g = ww.g;
  if (!Xt || !Yt || ldx < g.K || ldy < g.R) return NM_EINVAL;
  st = check_offsets(offsets, offsets_dtype);
  if (st != NM_OK) return st;
  if (!aligned(Xt, 2) || !aligned(Yt, 2)) return NM_EUNSUPPORTED;
  const RowsPlan plan = plan_of(ww, T);
  const bool direct = rows_direct(plan.path, Xt, ldx, g.K);
  const size_t pad = direct ? 0 : padded_bytes(T, g.K), need = pad + copies_bytes(ww, plan.path);
  if (need && (!workspace || workspace_bytes < need)) return NM_EINVAL;
  if (need && !aligned(workspace, 256)) return NM_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  nm::RowsArgs a{};
  a.g = g;
  a.X = Xt;
  a.ldx = ldx;
  if (!direct) {
    a.ldx = up64(g.K);
    if (nm::launch_pad_rows(Xt, ldx, T, g.K, ws, a.ldx, s) != hipSuccess) return NM_EHIP;
    a.X = ws;
    a.g.K = a.ldx;                                      // a padded row's zeros may be read
  }
  a.wdt = ww.dtype;
  a.values = ww.values;
  a.meta = ww.meta;
  a.rows = groups_of(offsets, offsets_dtype, ww.E, T);
  a.Y = Yt;
  a.ldy = ldy;
  a.ydt = ww.dtype;
  a.zero_rest = zero_rest != 0;
  return multiply(ww, plan, a, (int)(a.g.K / 8), ws + pad, s) == hipSuccess ? NM_OK : NM_EHIP;
}

nm_status nm_expert_linear_backward_workspace_size(const nm_experts* w, int64_t T, size_t* bytes) {
  Weights ww;
  nm_status st = weights_of(w, &ww);
  if (st != NM_OK) return st;
  if (!bytes) return NM_EINVAL;
  st = check_backward(ww, T);
  if (st != NM_OK) return st;
  *bytes = BackwardPlan(ww, T, true, true, true, true).total;
  return NM_OK;
}

nm_status nm_expert_linear_backward_workspace_size_for(const nm_experts* w, const void* Xt, int64_t ldx, int64_t T,
                                                       const void* dY, int64_t lddy, int32_t dx, int32_t dw,
                                                       size_t* bytes) {
  Weights ww;
  nm_status st = weights_of(w, &ww);
  if (st != NM_OK) return st;
  st = check_backward(ww, T);
  if (st != NM_OK) return st;
  if (!bytes || !Xt || !dY || ldx < ww.g.K || lddy < ww.g.R || (!dx && !dw)) return NM_EINVAL;
  *bytes = backward_plan(ww, Xt, ldx, T, dY, lddy, dx != 0, dw != 0).total;
  return NM_OK;
}

nm_status nm_expert_linear_backward(const nm_experts* w, const void* Xt, int64_t ldx, int64_t T, const void* offsets,
                                    int32_t offsets_dtype, const void* dY, int64_t lddy, void* dX, int64_t lddx,
                                    int32_t zero_rest, void* dW, int64_t lddw, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  Weights ww;
  nm_status st = weights_of(w, &ww);
  if (st != NM_OK) return st;
  st = check_backward(ww, T);
  if (st != NM_OK) return st;
  const Geometry& g = ww.g;
  if (!Xt || !dY || ldx < g.K || lddy < g.R || (!dX && !dW)) return NM_EINVAL;
  if ((dX && lddx < g.K) || (dW && lddw < g.K)) return NM_EINVAL;
  st = check_offsets(offsets, offsets_dtype);
  if (st != NM_OK) return st;
  if (!aligned(Xt, 2) || !aligned(dY, 2) || !aligned(dX, 2) || !aligned(dW, 2)) return NM_EUNSUPPORTED;
  const BackwardPlan p = backward_plan(ww, Xt, ldx, T, dY, lddy, dX != nullptr, dW != nullptr);
  const bool pad_x = p.xp != 0, pad_y = p.yp != 0;
  if (!workspace || workspace_bytes < p.total) return NM_EINVAL;
  if (!aligned(workspace, 256)) return NM_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* wt = static_cast<uint8_t*>(workspace);
  uint8_t* mask = wt + p.wt;
  uint8_t* xp = mask + p.mask;
  uint8_t* yp = xp + p.xp;
  const RowGroups rows = groups_of(offsets, offsets_dtype, ww.E, T);

  nm::RowsPrepareArgs q{};
  q.g = g;
  q.rows = rows;
  q.values = ww.values;
  q.meta = ww.meta;
  q.X = static_cast<const uint16_t*>(Xt);
  q.ldx = ldx;
  q.dY = static_cast<const uint16_t*>(dY);
  q.lddy = lddy;
  q.wt = dX ? reinterpret_cast<uint16_t*>(wt) : nullptr;
  q.mask = dW ? mask : nullptr;
  q.xp = pad_x ? reinterpret_cast<uint16_t*>(xp) : nullptr;
  q.yp = pad_y ? reinterpret_cast<uint16_t*>(yp) : nullptr;
  if (nm::launch_rows_prepare(q, s) != hipSuccess) return NM_EHIP;
  const int64_t Rp = up64(g.R), Kp = up64(g.K);
  nm::RowsTile tx{}, tw{};
  tx.rows = tw.rows = rows;
  tx.A = tw.A = pad_y ? yp : static_cast<const uint8_t*>(dY);
  tx.lda = tw.lda = pad_y ? Rp * 2 : lddy * 2;
  tx.ka = tw.ka = (int)((pad_y ? Rp : g.R) / 8);
  // dX[s][k] = sum_r dY[s][r] W_e[r][k]
  tx.B[0] = wt;
  tx.Mr = T;
  tx.Nr = g.K;
  tx.nslab = (int)(Rp / 64);
  tx.C = dX;
  tx.ldc = lddx;
  tx.zero_rest = zero_rest != 0;
  // dW_e[r][k] = sum over e's rows of dY[s][r] X[s][k]
  tw.B[0] = pad_x ? xp : static_cast<const uint8_t*>(Xt);
  tw.ldb = pad_x ? Kp * 2 : ldx * 2;
  tw.kb = (int)((pad_x ? Kp : g.K) / 8);
  tw.Mr = g.R;
  tw.Nr = g.K;
  tw.C = dW;
  tw.ldc = lddw;
  tw.es = g.R * lddw;
  tw.mask = mask;
  tw.ldm = g.nKB;
  const int shape = nm::grads_tile_shape(g, T, ww.E, dX != nullptr, dW != nullptr, nm::device_cu_count(), &tw.w.lead);
  return nm::launch_rows_grads(tile_type(ww.dtype), tx, tw, shape, s) == hipSuccess ? NM_OK : NM_EHIP;
}

nm_status nm_i8_expert_linear_workspace_size(const nm_experts* w, const nm_i8* xq, int64_t T, size_t* bytes) {
  Weights ww;
  const nm_status st = weights_of(w, &ww);
  return st != NM_OK ? st : i8_workspace(ww, xq, T, bytes);
}

nm_status nm_i8_expert_linear(const nm_experts* w, const float* w_scale, const nm_i8* xq, const void* Xt, int64_t ldx,
                              int32_t x_dtype, int64_t T, const void* offsets, int32_t offsets_dtype, void* Yt,
                              int64_t ldy, int32_t y_dtype, const float* bias, int32_t act, int32_t zero_rest,
                              void* workspace, size_t workspace_bytes, void* stream) {
  Weights ww;
  nm_status st = weights_of(w, &ww);
  if (st != NM_OK) return st;
  st = check_offsets(offsets, offsets_dtype);
  if (st != NM_OK) return st;
  return i8_product(ww, w_scale, xq, Xt, ldx, x_dtype, T, groups_of(offsets, offsets_dtype, ww.E, T), Yt, ldy, y_dtype,
                    bias, act, zero_rest != 0, workspace, workspace_bytes, stream);
}

}  // extern "C"
