// C ABI of the feed-forward operators (include/nm_sparse.h): host-side
// validation, choice of the path per shape, launches.  Stateless and
// thread-safe.
#include <algorithm>

#include "nm_ffn.hpp"

using nm::Geometry;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t up64(int64_t n) { return (n + 63) / 64 * 64; }

// rows the tile kernel addresses with 32-bit offsets: 256 of them within 2^31 bytes
bool row_ok(int64_t row_bytes) { return row_bytes < (1ll << 23); }

// Up to the first number of tokens (one tile of the matrix instruction) weights
// are streamed always, up to the second where that is faster; beyond, the tile
// product shares them.
constexpr int64_t kStreamOnly = 16, kStreamTokens = 1024;

// -1, or what the environment forces: 1 streamed weights, 0 tiles
int stream_forced() {
  int v;
  if (nm::ffn_tile_override("stream", &v, nullptr)) return v != 0;
  return nm::ffn_tile_override("tile", &v, nullptr) || nm::ffn_tile_override("tile24", &v, nullptr) ? 0 : -1;
}

// A product whose weights are streamed runs in whole rounds of workgroups, one
// to a compute unit: the row blocks (16 outputs) of an XCD times the groups of
// tokens, over its compute units.
struct StreamRounds {
  int64_t rounds;
  int nt;                    // 16-token tiles of a workgroup
  StreamRounds(int64_t blocks, int64_t T, int cus) : nt(nm::stream_tiles(blocks, T)) {
    const int64_t slots = (cus + 7) / 8;
    rounds = ((blocks + 7) / 8 * ((T + 16 * nt - 1) / (16 * nt)) + slots - 1) / slots;
  }
  // Microseconds.  passes: of the workgroup's eight waves along K; weight: what
  // a pass costs for its weights, and 0.2 for each token tile; `bytes` of weights
  // at 5.4 TB/s at least.  Fitted to 960 products of every pattern and of 4 bits,
  // 17 to 1024 tokens, 160 to 131072 outputs, K 256 to 8192: 7% off as a root mean
  // square, 30% at most; the choice costs 0.3% against the faster way as a mean
  // over them.  For example 2:4, 600 x 4096: 384 tokens 12.5 us (one round), 512
  // 21.1 and 768 22.6 (two), 1024 33.4 (three).
  double time(double passes, double weight, double bytes) const {
    return 2.7 + std::max(rounds * (0.3 + 0.25 * nt + passes * (weight + 0.2 * nt)), bytes / 5.4e6);
  }
};

// Longest dimension taken, and most workgroups of 256 threads: a launch has
// fewer than 2^32 threads.
constexpr int64_t kMaxLen = 1ll << 25;
constexpr int64_t kMaxGrid = 1ll << 24;

// One tile product of elements `et` (TILE_*), with its plan; a split's slices
// go to `part` (plan.split * Mr * Nr binary32) and are added afterwards.
hipError_t run_tile(int et, nm::TileOp op, int ydt, nm::TileArgs a, const nm::TilePlan& plan, float* part,
                    hipStream_t s) {
  auto launch = et == nm::TILE_F16 ? nm::launch_tile_f16 : et == nm::TILE_BF16 ? nm::launch_tile_bf16 : nm::launch_tile_mx;
  a.shape = plan.shape;
  a.split = plan.split;
  a.sps = plan.sps;
  a.w.lead = plan.lead;
  if (plan.split == 1 || !a.C) return launch(op, ydt, a, s);
  nm::TileArgs p = a;
  p.C = part;
  p.ldc = a.Nr;
  p.cs = a.Mr * a.Nr;
  p.bias = nullptr;
  p.act = NM_ACT_NONE;
  const hipError_t e = launch(op, op == nm::TILE_LINEAR ? NM_F32 : ydt, p, s);
  if (e != hipSuccess) return e;
  return nm::launch_tile_reduce(part, plan.split, a.Mr, a.Nr, a.bias, a.act, a.C, a.ldc, ydt, s);
}

size_t part_bytes(const nm::TilePlan& p, int64_t Mr, int64_t Nr) {
  return p.split > 1 ? up256((size_t)(p.split * Mr * Nr * 4)) : 0;
}

int tile_type(int wdt) { return wdt == NM_F16 ? nm::TILE_F16 : nm::TILE_BF16; }

// ---------------------------------------------------------------- gated block, N:M weights
nm_status check_pair(const nm_packed* gate, const nm_packed* up, Geometry* g) {
  Geometry gu;
  nm_status st = nm::check_packed(gate, g);
  if (st != NM_OK) return st;
  st = nm::check_packed(up, &gu);
  if (st != NM_OK) return st;
  if (gate->rows != up->rows || gate->K != up->K || gate->N != up->N || gate->M != up->M || gate->dtype != up->dtype)
    return NM_EINVAL;
  if (gate->dtype != NM_F16 && gate->dtype != NM_BF16) return NM_EUNSUPPORTED;
  // dense rows of K within the tile kernel's offsets; launches along R
  if (!row_ok(up64(g->K) * 2) || g->R > (1ll << 22)) return NM_EUNSUPPORTED;
  return NM_OK;
}

bool glu_act_ok(int32_t act) { return act == NM_ACT_SILU || act == NM_ACT_GELU; }
bool kept_type_ok(int32_t p_dtype, int32_t wdt) { return p_dtype == wdt || p_dtype == NM_F32; }

// How a call multiplies.
enum GluPath {
  GLU_STREAM,   // few tokens: the packed weights streamed past each 16 to 64 of them
  GLU_SPARSE,   // 2:4: the sparse tile product
  GLU_REPACK,   // 1:4, 1:8, 2:8: re-packed to 2:4 in the workspace, then the same
  GLU_DENSE     // others: dense copies in the workspace, the dense tile product
};

Geometry geometry24(const Geometry& g) { return Geometry::make(g.R, g.K, 2, 4, g.eb); }

// Weights of one round are streamed: measured, streamed and tiles, 2:4 of 600 x
// 4096 12.5 and 20.7 us (384 tokens), 4:4 of 600 x 8192 28 and 46, 7:8 43 and 54.
// More rounds by models of both times: StreamRounds; the tile product's own, and
// the copies at 5 TB/s.  Measured, streamed and tiles: 11008 x 4096, 2:4 21.4 and
// 21.3 us (32 tokens), 31 and 22 (64); 4:8 33 and 93 (64), 98 and 112 (256), 149
// and 133 (384); 131072 x 256, 2:4 42 and 27 (32); 600 x 4096, 2:4 22.6 and 20.9
// (768), 4:8 23.5 and 30.7.
GluPath glu_path(const Geometry& g, int64_t T) {
  const GluPath tiles = g.N == 2 && g.M == 4 ? GLU_SPARSE : nm::repack24_supported(g) ? GLU_REPACK : GLU_DENSE;
  if (T > kStreamTokens) return tiles;
  const int forced = stream_forced();
  if (forced >= 0) return forced ? GLU_STREAM : tiles;
  if (T <= kStreamOnly) return GLU_STREAM;
  const int cus = nm::device_cu_count();
  const StreamRounds r(g.nRB, T, cus);
  if (r.rounds == 1) return GLU_STREAM;
  // what 512 columns of both weights' 16 rows cost a wave: sparse as they are or
  // by the selector table, and expanded by shifts (3:4, 5:8 to 7:8)
  static const double weight[2][8] = {{0.10, 0.17, 0.43, 0.63}, {0.22, 0.24, 0.27, 0.34, 1.06, 1.2, 1.67, 0.63}};
  const double packed = 2.0 * (double)(g.values_bytes() + g.meta_bytes());
  const double stream = r.time((double)g.K / 512, weight[g.M == 8][g.N - 1], packed);
  double other;
  if (tiles == GLU_DENSE) {
    const int64_t Kp = up64(g.K);
    // (odd N of 8: kept values read one at a time)
    other = 5.0 + ((g.M == 8 && g.N % 2 ? 3.0 : 1.0) * packed + 4.0 * g.R * Kp) / 5e6 +
            nm::plan_tile(nm::TILE_GLU, false, T, g.R, (int)(Kp / 64), cus).time;
  } else {
    other = nm::glu_tile24_time(T, g.R, g.nKB, cus, nullptr);
    if (tiles == GLU_REPACK) {
      const Geometry d = geometry24(g);
      other += 8.0 + (packed + 2.0 * (double)(d.values_bytes() + d.meta_bytes())) / 5e6;
    }
  }
  return stream <= other ? GLU_STREAM : tiles;
}

// Whether the path's kernel reads X's rows as they are.  Streamed: any rows of
// at least one 16-byte piece; tiles: 16-byte pieces, none of which crosses the
// end of a row, and 32-bit offsets.
bool rows_direct(GluPath path, const void* X, int64_t ldx, int64_t K) {
  if (path == GLU_STREAM) return K >= 8;
  return aligned(X, 16) && ldx % 8 == 0 && K % 8 == 0 && row_ok(ldx * 2);
}

// a weight re-packed to 2:4: values, then positions
size_t repacked_bytes(const Geometry& g) {
  const Geometry d = geometry24(g);
  return up256(d.values_bytes()) + up256(d.meta_bytes());
}

size_t padded_bytes(const Geometry& g, int64_t T) { return up256((size_t)(T * up64(g.K) * 2)); }
size_t dense_bytes(const Geometry& g) { return up256((size_t)(g.R * up64(g.K) * 2)); }
// workspace for both weights' copies
size_t weights_bytes(const Geometry& g, GluPath path) {
  return path == GLU_DENSE ? 2 * dense_bytes(g) : path == GLU_REPACK ? 2 * repacked_bytes(g) : 0;
}

// transposed rows of T, and rows of both dG and dU, within the tile kernel's
// offsets; the operands' tiles within one launch
bool backward_ok(const Geometry& g, int64_t T) {
  return row_ok(up64(T) * 2) && row_ok(up64(g.R) * 4) &&
         up64(T) / 64 * (up64(g.R) / 64 + g.nKB) + 2 * ((g.R + 127) / 128) * g.nKB < kMaxGrid;
}

// With kept products in binary32, up to this many multiply-adds a product: dG and
// dU in two 16-bit parts.  One part's rounding makes the gradients' distance from
// 64-bit ones 1.41 times the output rounding's, but where few of them meet up to
// 1.7 times (over 1.5 in 41 of 390 products of random sizes, in 1 of those beyond
// this limit); two parts leave the output's rounding alone.  They double
// reductions that are short here: 64 tokens, 256 x 256 10.2 -> 12.6 us, 16, 1000 x
// 768 15.4 -> 18.8, 128, 512 x 512 13.3 -> 18.1; beyond, 197, 2048 x 2048 34 -> 43.
constexpr double kTwoPartWork = 1 << 26;

struct BackwardPlan {
  int64_t Rp, Tp, Kp;
  int parts;
  size_t d, dt, xt, wt, mask, part, total;   // bytes of each part (mask: of one weight)
  nm::TilePlan plan;
  BackwardPlan(const Geometry& g, int64_t T, bool dx, bool dw, bool p32) {
    Rp = up64(g.R);
    Tp = up64(T);
    Kp = up64(g.K);
    parts = p32 && (double)T * (double)g.R * (double)g.K <= kTwoPartWork && row_ok(Tp * 4) && row_ok(Rp * 8) ? 2 : 1;
    d = up256((size_t)(T * 2 * Rp * parts * 2));
    dt = up256((size_t)(2 * g.R * Tp * parts * 2));
    xt = up256((size_t)(g.K * Tp * parts * 2));
    wt = up256((size_t)(g.K * 2 * Rp * parts * 2));
    mask = up256((size_t)(g.R * Kp / 8));
    plan = nm::plan_back(T, g.R, g.K, (int)(parts * 2 * Rp / 64), (int)(parts * Tp / 64), dx, dw,
                         nm::device_cu_count());
    part = dx ? part_bytes(plan, T, g.K) : 0;
    total = d + dt + xt + wt + 2 * mask + part;
  }
};

// ---------------------------------------------------------------- microscaled format
nm_status check_mx(const nm_mx* m) {
  if (!m || m->rows < 1 || m->K < 1 || !m->codes || !m->scales) return NM_EINVAL;
  if (m->K > kMaxLen || m->rows > kMaxLen) return NM_EUNSUPPORTED;
  if ((int64_t)m->codes_bytes != nm::mx_codes_bytes(m->rows, m->K)) return NM_EINVAL;
  if ((int64_t)m->scales_bytes != nm::mx_scales_bytes(m->rows, m->K)) return NM_EINVAL;
  if (!aligned(m->codes, 16) || !aligned(m->scales, 16)) return NM_EUNSUPPORTED;
  if ((m->rows + 31) / 32 * (nm::mx_kp(m->K) / nm::kMxSlab) >= kMaxGrid) return NM_EUNSUPPORTED;
  return NM_OK;
}

bool float_dtype(int32_t dt) { return dt == NM_F16 || dt == NM_BF16 || dt == NM_F32; }

size_t mx_ws_codes(int64_t T, int64_t K) { return up256((size_t)nm::mx_codes_bytes(T, K)); }
size_t mx_ws(int64_t T, int64_t K) { return mx_ws_codes(T, K) + up256((size_t)nm::mx_scales_bytes(T, K)); }
// up to 16 tokens are quantised inside the product (in pieces of eight columns)
bool mx_inside(int64_t T, int64_t K) { return T <= 16 && K >= 8; }
// How a product of T tokens is computed: the weights streamed for every 64 of
// them (always where that is one round), or the tile product with its plan, by
// models of both times.  Measured, streamed and tiles: gated block of 11008 x
// 4096 14.6 and 14.3 us (64 tokens), 23 and 20 (128); of 4096 x 11008 22 and 26
// (128), 37 and 27 (256); product of 1000 x 3000 5.5 and 12 (256), 7.2 and 12
// (512); of 131072 x 256 22 and 11 (32).
struct MxPath {
  bool stream;
  nm::TilePlan plan;
};
MxPath mx_path(bool glu, int64_t T, int64_t R, int64_t K) {
  MxPath p{};
  const int forced = stream_forced();
  if (T <= kStreamTokens && (forced >= 0 ? forced : T <= kStreamOnly)) {
    p.stream = true;
    return p;
  }
  const int cus = nm::device_cu_count();
  const StreamRounds r((R + 15) / 16, T, cus);
  if (T <= kStreamTokens && forced < 0 && r.rounds == 1) return MxPath{true, {}};
  p.plan = nm::plan_tile(glu ? nm::TILE_GLU : nm::TILE_LINEAR, true, T, R, (int)(nm::mx_kp(K) / nm::kMxSlab), cus);
  if (T > kStreamTokens || forced == 0) return p;
  const double w = (glu ? 2.0 : 1.0) * (double)(R * nm::mx_kp(K)) * 17 / 32;
  // (2.5: the launch, which the 4-bit tiles' model leaves out)
  if (r.time((double)nm::mx_kp(K) / 2048, glu ? 0.7 : 0.35, w) <= p.plan.time + 2.5) p = MxPath{true, {}};
  return p;
}

nm_status mx_product(const nm_mx* w0, const nm_mx* w1, const nm_mx* xq, const void* X, int64_t ldx, int32_t xdt,
                     int64_t T, void* Y, int64_t ldy, int32_t ydt, const float* bias, int32_t act, void* ws,
                     size_t ws_bytes, void* stream) {
  const bool glu = w1 != nullptr;
  nm_status st = check_mx(w0);
  if (st != NM_OK) return st;
  if (w0->format_version != NM_FORMAT_VERSION) return NM_EINVAL;
  const int64_t R = w0->rows, K = w0->K, Kp = nm::mx_kp(K);
  if (glu) {
    st = check_mx(w1);
    if (st != NM_OK) return st;
    if (w1->format_version != NM_FORMAT_VERSION || w1->rows != R || w1->K != K) return NM_EINVAL;
  }
  if (!Y || T < 1 || ldy < R) return NM_EINVAL;
  if (!float_dtype(ydt) || T > kMaxLen) return NM_EUNSUPPORTED;
  if (glu ? !glu_act_ok(act) : (act != NM_ACT_NONE && act != NM_ACT_GELU)) return NM_EUNSUPPORTED;
  if (!aligned(Y, (size_t)nm::dtype_bytes(ydt)) || (bias && !aligned(bias, 4))) return NM_EUNSUPPORTED;
  if (!row_ok(Kp / 2)) return NM_EUNSUPPORTED;
  if (xq) {
    st = check_mx(xq);
    if (st != NM_OK) return st;
    if (xq->format_version != NM_FORMAT_VERSION || xq->rows != T || xq->K != K) return NM_EINVAL;
  } else {
    if (!X || ldx < K) return NM_EINVAL;
    if (!float_dtype(xdt) || !aligned(X, (size_t)nm::dtype_bytes(xdt))) return NM_EUNSUPPORTED;
    if ((T + 31) / 32 * (Kp / nm::kMxSlab) >= kMaxGrid) return NM_EUNSUPPORTED;
  }
  const bool inside = !xq && mx_inside(T, K);
  const MxPath path = inside ? MxPath{true, {}} : mx_path(glu, T, R, K);
  const size_t quant = xq || inside ? 0 : mx_ws(T, K);
  const size_t need = quant + part_bytes(path.plan, T, R);
  if (need && (!ws || ws_bytes < need)) return NM_EINVAL;
  if (need && !aligned(ws, 256)) return NM_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);

  const uint8_t* xcodes = xq ? static_cast<const uint8_t*>(xq->codes) : nullptr;
  const uint8_t* xscales = xq ? static_cast<const uint8_t*>(xq->scales) : nullptr;
  if (quant) {
    uint8_t* c = static_cast<uint8_t*>(ws);
    uint8_t* sc = c + mx_ws_codes(T, K);
    if (nm::launch_mx_quantize(X, ldx, xdt, T, K, c, sc, s) != hipSuccess) return NM_EHIP;
    xcodes = c;
    xscales = sc;
  }
  const nm_mx* ws2[2] = {w0, glu ? w1 : w0};
  if (path.stream) {
    nm::MxDecodeArgs a{};
    for (int i = 0; i < 2; ++i) {
      a.codes[i] = static_cast<const uint8_t*>(ws2[i]->codes);
      a.scales[i] = static_cast<const uint8_t*>(ws2[i]->scales);
    }
    a.R = R;
    a.K = K;
    a.X = inside ? X : nullptr;
    a.ldx = ldx;
    a.xdt = xdt;
    a.xcodes = xcodes;
    a.xscales = xscales;
    a.T = T;
    a.Y = Y;
    a.ldy = ldy;
    a.ydt = ydt;
    a.bias = bias;
    a.act = act;
    a.glu = glu;
    return nm::launch_mx_decode(a, s) == hipSuccess ? NM_OK : NM_EHIP;
  }
  nm::TileArgs a{};
  a.A = xcodes;
  a.As = xscales;
  for (int i = 0; i < 2; ++i) {
    a.B[i] = static_cast<const uint8_t*>(ws2[i]->codes);
    a.Bs[i] = static_cast<const uint8_t*>(ws2[i]->scales);
  }
  a.lda = a.ldb = Kp / 2;
  a.Mr = T;
  a.Nr = R;
  a.ka = a.kb = (int)(Kp / 32);
  a.nslab = (int)(Kp / nm::kMxSlab);
  a.C = Y;
  a.ldc = ldy;
  a.bias = bias;
  a.act = act;
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + quant);
  return run_tile(nm::TILE_MX, glu ? nm::TILE_GLU : nm::TILE_LINEAR, ydt, a, path.plan, part, s) == hipSuccess
             ? NM_OK
             : NM_EHIP;
}

}  // namespace

extern "C" {

nm_status nm_glu_workspace_size(const nm_packed* gate, const nm_packed* up, const void* Xt, int64_t ldx, int64_t T,
                                size_t* bytes) {
  if (!bytes || T < 1) return NM_EINVAL;
  Geometry g;
  const nm_status st = check_pair(gate, up, &g);
  if (st != NM_OK) return st;
  if (T > kMaxLen) return NM_EUNSUPPORTED;
  if (Xt && ldx < g.K) return NM_EINVAL;
  const GluPath path = glu_path(g, T);
  // (NULL: the worst rows)
  *bytes = (rows_direct(path, Xt ? Xt : reinterpret_cast<const void*>(2), ldx, g.K) ? 0 : padded_bytes(g, T)) +
           weights_bytes(g, path);
  return NM_OK;
}

nm_status nm_glu(const nm_packed* gate, const nm_packed* up, const void* Xt, int64_t ldx, int64_t T, void* Ht,
                 int64_t ldh, int32_t act, void* G, void* U, int64_t ldp, void* workspace, size_t workspace_bytes,
                 void* stream) {
  return nm_glu_kept(gate, up, Xt, ldx, T, Ht, ldh, act, G, U, ldp, gate ? gate->dtype : 0, workspace,
                     workspace_bytes, stream);
}

nm_status nm_glu_kept(const nm_packed* gate, const nm_packed* up, const void* Xt, int64_t ldx, int64_t T, void* Ht,
                      int64_t ldh, int32_t act, void* G, void* U, int64_t ldp, int32_t p_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  Geometry g;
  const nm_status st = check_pair(gate, up, &g);
  if (st != NM_OK) return st;
  if (T > kMaxLen) return NM_EUNSUPPORTED;
  if (gate->format_version != NM_FORMAT_VERSION || up->format_version != NM_FORMAT_VERSION) return NM_EINVAL;
  if (!Xt || !Ht || T < 1 || ldx < g.K || ldh < g.R) return NM_EINVAL;
  if ((G == nullptr) != (U == nullptr) || (G && ldp < g.R)) return NM_EINVAL;
  if (!glu_act_ok(act) || (G && !kept_type_ok(p_dtype, gate->dtype))) return NM_EUNSUPPORTED;
  const size_t pb = p_dtype == NM_F32 ? 4 : 2;
  if (!aligned(Xt, 2) || !aligned(Ht, 2) || (G && (!aligned(G, pb) || !aligned(U, pb)))) return NM_EUNSUPPORTED;
  const GluPath path = glu_path(g, T);
  const bool direct = rows_direct(path, Xt, ldx, g.K);
  const size_t pad = direct ? 0 : padded_bytes(g, T);
  const size_t need = pad + weights_bytes(g, path);
  if (need && (!workspace || workspace_bytes < need)) return NM_EINVAL;
  if (need && !aligned(workspace, 256)) return NM_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  const void* X = Xt;
  int64_t ld = ldx;
  if (!direct) {
    ld = up64(g.K);
    if (nm::launch_pad_rows(Xt, ldx, T, g.K, ws, ld, s) != hipSuccess) return NM_EHIP;
    X = ws;
  }
  const nm_packed* w[2] = {gate, up};
  if (path != GLU_DENSE) {
    nm::GluArgs a{};
    a.g = g;
    a.wdt = gate->dtype;
    for (int i = 0; i < 2; ++i) {
      a.values[i] = static_cast<const uint8_t*>(w[i]->values);
      a.meta[i] = g.w ? static_cast<const uint8_t*>(w[i]->meta) : nullptr;
    }
    a.X = X;
    a.ldx = ld;
    a.T = T;
    a.H = Ht;
    a.ldh = ldh;
    a.P[0] = G;
    a.P[1] = U;
    a.ldp = ldp;
    a.p32 = p_dtype == NM_F32;
    a.act = act;
    if (path == GLU_REPACK) {
      const Geometry d = geometry24(g);
      for (int i = 0; i < 2; ++i) {
        uint8_t* v = ws + pad + i * repacked_bytes(g);
        uint8_t* m = v + up256(d.values_bytes());
        if (nm::launch_repack24(g, a.values[i], a.meta[i], d, v, m, s) != hipSuccess) return NM_EHIP;
        a.values[i] = v;
        a.meta[i] = m;
      }
      a.g = d;
    }
    // a padded row is all 16-byte pieces: its zeros may be read
    if (!direct) a.g.K = ld;
    return (path == GLU_STREAM ? nm::launch_glu_decode(a, s) : nm::launch_glu_tile24(a, s)) == hipSuccess ? NM_OK
                                                                                                          : NM_EHIP;
  }
  nm::TileArgs a{};
  const int64_t Kp = up64(g.K);
  nm::DenseArgs e{};
  for (int i = 0; i < 2; ++i) {
    uint8_t* d = ws + pad + i * dense_bytes(g);
    e.values[i] = static_cast<const uint8_t*>(w[i]->values);
    e.meta[i] = static_cast<const uint8_t*>(w[i]->meta);
    e.dense[i] = reinterpret_cast<uint16_t*>(d);
    a.B[i] = d;
  }
  a.A = static_cast<const uint8_t*>(X);
  if (nm::launch_expand_dense(g, e, s) != hipSuccess) return NM_EHIP;
  a.lda = ld * 2;
  a.ldb = Kp * 2;
  a.Mr = T;
  a.Nr = g.R;
  a.ka = (int)((direct ? g.K : Kp) / 8);
  a.kb = (int)(Kp / 8);
  a.nslab = (int)(Kp / 64);
  a.C = Ht;
  a.ldc = ldh;
  a.P[0] = G;
  a.P[1] = U;
  a.ldp = ldp;
  a.p32 = p_dtype == NM_F32;
  a.act = act;
  const nm::TilePlan plan = nm::plan_tile(nm::TILE_GLU, false, T, g.R, a.nslab, nm::device_cu_count());
  return run_tile(tile_type(gate->dtype), nm::TILE_GLU, gate->dtype, a, plan, nullptr, s) == hipSuccess ? NM_OK
                                                                                                       : NM_EHIP;
}

nm_status nm_glu_backward_workspace_size(const nm_packed* gate, const nm_packed* up, int64_t T, size_t* bytes) {
  if (!bytes || T < 1) return NM_EINVAL;
  Geometry g;
  const nm_status st = check_pair(gate, up, &g);
  if (st != NM_OK) return st;
  if (T > kMaxLen) return NM_EUNSUPPORTED;
  if (!backward_ok(g, T)) return NM_EUNSUPPORTED;
  *bytes = 0;
  for (int i = 0; i < 4; ++i) *bytes = std::max(*bytes, BackwardPlan(g, T, true, i & 1, i & 2).total);
  return NM_OK;
}

nm_status nm_glu_backward(const nm_packed* gate, const nm_packed* up, const void* Xt, int64_t ldx, int64_t T,
                          const void* G, const void* U, int64_t ldp, const void* dH, int64_t lddh, int32_t act,
                          void* dX, int64_t lddx, void* dWg, void* dWu, int64_t lddw, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return nm_glu_backward_kept(gate, up, Xt, ldx, T, G, U, ldp, gate ? gate->dtype : 0, dH, lddh, act, dX, lddx, dWg,
                              dWu, lddw, workspace, workspace_bytes, stream);
}

nm_status nm_glu_backward_kept(const nm_packed* gate, const nm_packed* up, const void* Xt, int64_t ldx, int64_t T,
                               const void* G, const void* U, int64_t ldp, int32_t p_dtype, const void* dH,
                               int64_t lddh, int32_t act, void* dX, int64_t lddx, void* dWg, void* dWu, int64_t lddw,
                               void* workspace, size_t workspace_bytes, void* stream) {
  Geometry g;
  const nm_status st = check_pair(gate, up, &g);
  if (st != NM_OK) return st;
  if (T > kMaxLen) return NM_EUNSUPPORTED;
  if (gate->format_version != NM_FORMAT_VERSION || up->format_version != NM_FORMAT_VERSION) return NM_EINVAL;
  if (!Xt || !G || !U || !dH || T < 1 || ldx < g.K || ldp < g.R || lddh < g.R) return NM_EINVAL;
  if ((dWg == nullptr) != (dWu == nullptr) || (!dX && !dWg)) return NM_EINVAL;
  if ((dX && lddx < g.K) || (dWg && lddw < g.K)) return NM_EINVAL;
  if (!glu_act_ok(act) || !kept_type_ok(p_dtype, gate->dtype)) return NM_EUNSUPPORTED;
  const size_t pb = p_dtype == NM_F32 ? 4 : 2;
  if (!aligned(Xt, 2) || !aligned(G, pb) || !aligned(U, pb) || !aligned(dH, 2) || !aligned(dX, 2) || !aligned(dWg, 2) ||
      !aligned(dWu, 2))
    return NM_EUNSUPPORTED;
  if (!backward_ok(g, T)) return NM_EUNSUPPORTED;
  const BackwardPlan p(g, T, dX != nullptr, dWg != nullptr, p_dtype == NM_F32);
  if (!workspace || workspace_bytes < p.total) return NM_EINVAL;
  if (!aligned(workspace, 256)) return NM_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* d = static_cast<uint8_t*>(workspace);
  uint8_t* dt = d + p.d;
  uint8_t* xt = dt + p.dt;
  uint8_t* wt = xt + p.xt;
  uint8_t* mask = wt + p.wt;
  float* part = reinterpret_cast<float*>(mask + 2 * p.mask);
  const nm_packed* w[2] = {gate, up};

  nm::PrepareArgs q{};
  q.g = g;
  for (int i = 0; i < 2; ++i) {
    q.values[i] = static_cast<const uint8_t*>(w[i]->values);
    q.meta[i] = static_cast<const uint8_t*>(w[i]->meta);
    q.mask[i] = dWg ? mask + i * p.mask : nullptr;
  }
  q.X = static_cast<const uint16_t*>(Xt);
  q.ldx = ldx;
  q.T = T;
  q.G = G;
  q.U = U;
  q.ldp = ldp;
  q.p32 = p_dtype == NM_F32;
  q.dH = static_cast<const uint16_t*>(dH);
  q.lddh = lddh;
  q.act = act;
  q.Rp = p.Rp;
  q.Tp = p.Tp;
  q.parts = p.parts;
  q.d = dX ? reinterpret_cast<uint16_t*>(d) : nullptr;
  q.wt = dX ? reinterpret_cast<uint16_t*>(wt) : nullptr;
  q.dt = dWg ? reinterpret_cast<uint16_t*>(dt) : nullptr;
  q.xt = dWg ? reinterpret_cast<uint16_t*>(xt) : nullptr;
  if (nm::launch_glu_prepare(q, gate->dtype, s) != hipSuccess) return NM_EHIP;
  nm::TileArgs a{};
  // dX[t][k] = sum over both weights' rows of d[t][r] W[r][k]
  a.A = d;
  a.B[0] = wt;
  a.lda = a.ldb = 4 * p.Rp * p.parts;
  a.Mr = T;
  a.Nr = g.K;
  a.ka = a.kb = (int)(2 * p.Rp * p.parts / 8);
  a.nslab = (int)(2 * p.Rp * p.parts / 64);
  a.C = dX;
  a.ldc = lddx;
  // dW[r][k] = sum over t of d[t][r] X[t][k], both transposed
  a.w.B = xt;
  a.w.ld = 2 * p.Tp * p.parts;
  a.w.Mr = g.R;
  a.w.Nr = g.K;
  a.w.nslab = (int)(p.Tp * p.parts / 64);
  a.w.C[0] = dWg;
  a.w.C[1] = dWu;
  a.w.ldc = lddw;
  a.w.ldm = p.Kp / 8;
  for (int i = 0; i < 2; ++i) {
    a.w.A[i] = dt + (size_t)i * g.R * p.Tp * p.parts * 2;
    a.w.mask[i] = mask + i * p.mask;
  }
  return run_tile(tile_type(gate->dtype), nm::TILE_BACK, gate->dtype, a, p.plan, part, s) == hipSuccess ? NM_OK
                                                                                                       : NM_EHIP;
}

nm_status nm_mx_size(int64_t rows, int64_t K, size_t* codes_bytes, size_t* scales_bytes) {
  if (!codes_bytes || !scales_bytes || rows < 1 || K < 1) return NM_EINVAL;
  if (K > kMaxLen || rows > kMaxLen) return NM_EUNSUPPORTED;
  *codes_bytes = (size_t)nm::mx_codes_bytes(rows, K);
  *scales_bytes = (size_t)nm::mx_scales_bytes(rows, K);
  return NM_OK;
}

nm_status nm_mx_quantize(const void* X, int64_t ldx, int32_t x_dtype, nm_mx* m, void* stream) {
  const nm_status st = check_mx(m);
  if (st != NM_OK) return st;
  if (!X || ldx < m->K) return NM_EINVAL;
  if (!float_dtype(x_dtype) || !aligned(X, (size_t)nm::dtype_bytes(x_dtype))) return NM_EUNSUPPORTED;
  if (nm::launch_mx_quantize(X, ldx, x_dtype, m->rows, m->K, static_cast<uint8_t*>(m->codes),
                             static_cast<uint8_t*>(m->scales), static_cast<hipStream_t>(stream)) != hipSuccess)
    return NM_EHIP;
  m->format_version = NM_FORMAT_VERSION;
  m->reserved = 0;
  return NM_OK;
}

nm_status nm_mx_dequantize(const nm_mx* m, void* Y, int64_t ldy, int32_t y_dtype, void* stream) {
  const nm_status st = check_mx(m);
  if (st != NM_OK) return st;
  if (m->format_version != NM_FORMAT_VERSION || !Y || ldy < m->K) return NM_EINVAL;
  if (!float_dtype(y_dtype) || !aligned(Y, (size_t)nm::dtype_bytes(y_dtype))) return NM_EUNSUPPORTED;
  return nm::launch_mx_dequantize(static_cast<const uint8_t*>(m->codes), static_cast<const uint8_t*>(m->scales),
                                  m->rows, m->K, Y, ldy, y_dtype, static_cast<hipStream_t>(stream)) == hipSuccess
             ? NM_OK
             : NM_EHIP;
}

nm_status nm_mx_workspace_size(const nm_mx* w, const nm_mx* xq, int64_t T, int32_t glu, size_t* bytes) {
  if (!bytes || T < 1) return NM_EINVAL;
  const nm_status st = check_mx(w);
  if (st != NM_OK) return st;
  if (!row_ok(nm::mx_kp(w->K) / 2) || T > kMaxLen) return NM_EUNSUPPORTED;
  if ((T + 31) / 32 * (nm::mx_kp(w->K) / nm::kMxSlab) >= kMaxGrid) return NM_EUNSUPPORTED;
  const bool quant = !xq && !mx_inside(T, w->K);
  const size_t part = quant || xq ? part_bytes(mx_path(glu != 0, T, w->rows, w->K).plan, T, w->rows) : 0;
  *bytes = (quant ? mx_ws(T, w->K) : 0) + part;
  return NM_OK;
}

nm_status nm_mx_linear(const nm_mx* w, const nm_mx* xq, const void* Xt, int64_t ldx, int32_t x_dtype, int64_t T,
                       void* Yt, int64_t ldy, int32_t y_dtype, const float* bias, int32_t act, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return mx_product(w, nullptr, xq, Xt, ldx, x_dtype, T, Yt, ldy, y_dtype, bias, act, workspace, workspace_bytes,
                    stream);
}

nm_status nm_mx_glu(const nm_mx* gate, const nm_mx* up, const nm_mx* xq, const void* Xt, int64_t ldx,
                    int32_t x_dtype, int64_t T, void* Ht, int64_t ldh, int32_t h_dtype, int32_t act, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!up) return NM_EINVAL;
  return mx_product(gate, up, xq, Xt, ldx, x_dtype, T, Ht, ldh, h_dtype, nullptr, act, workspace, workspace_bytes,
                    stream);
}

}  // extern "C"
