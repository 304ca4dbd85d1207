// The dense operators' C interface (moe_linear_*, moe_gated_*): host-side validation, workspace carving
// and launches.  Nothing is enqueued when a call refuses its arguments or workspace; a backward pass whose later launch
// fails (MOE_EHIP) may have run its earlier ones.
#include "dense.hpp"

namespace moe {

DensePlan g_dense_plan = {MOE_DENSE_AUTO, 0, 0};

// Workspace: control words, the sums of split reductions, then for a backward pass dz (gated: dg, du) in the
// operands' type with rows padded to whole 16-byte chunks, and the bias gradients' partial sums.
struct DenseWs {
  size_t part, x, w[2], dz0, dz1, bias_part, total;
  int64_t ldz;
};

static size_t dense_align(size_t v) { return (v + 255) & ~(size_t)255; }

// Room for the sums of split reductions: what kMaxSplits splits of the largest product would take, up to a limit.
static size_t part_bytes(const moe_dense_dims* d, int64_t T, bool backward) {
  size_t n = split_bytes(kMaxSplits, 2, T, d->n_out);
  if (backward) {
    const size_t dx = split_bytes(kMaxSplits, 1, T, d->n_in), dw = split_bytes(kMaxSplits, 2, d->n_out, d->n_in);
    n = dx > dw ? dx : dw;
    if (n < split_bytes(kMaxSplits, 2, T, d->n_out)) n = split_bytes(kMaxSplits, 2, T, d->n_out);
  }
  return n < kDensePartBytes ? n : kDensePartBytes;
}

// Two matrices whatever the call (one size serves the linear and the gated block).
static DenseWs dense_ws(const moe_dense_dims* d, int64_t T, bool backward) {
  DenseWs L{};
  L.part = kCtrlBytes;
  size_t off = dense_align(L.part + part_bytes(d, T, backward));
  // copies of operands without whole 16-byte rows: x always (its stride is the caller's), the weights when n_in
  // says so
  const int64_t ld_in = ((int64_t)d->n_in + 7) / 8 * 8;
  if (T > MOE_DENSE_ROW_TOKENS || backward) {
    L.x = off;
    off = dense_align(off + 2 * (size_t)(T * ld_in));
    if (d->n_in % 8)
      for (int m = 0; m < 2; ++m) {
        L.w[m] = off;
        off = dense_align(off + 2 * (size_t)(d->n_out * ld_in));
      }
  }
  if (backward) {
    const int64_t most = grad_runs_most(d->n_out), runs = (T + 3) / 4 < most ? (T + 3) / 4 : most;
    L.ldz = ((int64_t)d->n_out + 7) / 8 * 8;
    L.dz0 = off;
    off = dense_align(off + 2 * (size_t)(T * L.ldz));
    L.dz1 = off;
    off = dense_align(off + 2 * (size_t)(T * L.ldz));
    L.bias_part = off;
    off = dense_align(off + sizeof(float) * 2 * (size_t)(runs * d->n_out));
  }
  L.total = off;
  return L;
}

static int check_dense(const moe_dense_dims* d) {
  if (!d || d->n_in < 1 || d->n_out < 1) return MOE_EINVAL;
  if (d->n_in > MOE_DENSE_MAX_WIDTH || d->n_out > MOE_DENSE_MAX_WIDTH) return MOE_EUNSUPPORTED;
  if (d->dtype != MOE_BF16 && d->dtype != MOE_F16) return MOE_EUNSUPPORTED;
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_SIGMOID) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

static int check_tokens(int32_t T) {
  if (T < 1) return MOE_EINVAL;
  return T > MOE_DENSE_MAX_TOKENS ? MOE_EUNSUPPORTED : MOE_OK;
}

// Collects the checks of a call's matrices: element-aligned, rows that do not overlap, strides in range.
struct Mats {
  int rc = MOE_OK;
  void fail(int code) {
    if (rc == MOE_OK) rc = code;
  }
  void need(const void* p, int64_t ld, int64_t len, int elem = 2) {
    if (!p) fail(MOE_EINVAL);
    else opt(p, ld, len, elem);
  }
  void opt(const void* p, int64_t ld, int64_t len, int elem = 2) {
    if (!p) return;
    if ((uintptr_t)p % elem || ld < len) fail(MOE_EINVAL);
    else if (ld > MOE_DENSE_MAX_LD) fail(MOE_EUNSUPPORTED);
  }
  void vec(const void* p) { opt(p, 1, 1); }
};

static int check_dense_ws(const moe_dense_dims* d, int32_t T, bool backward, const void* ws, size_t ws_bytes) {
  if (!ws || ((uintptr_t)ws & 255)) return MOE_EWORKSPACE;
  return ws_bytes < dense_ws(d, T, backward).total ? MOE_EWORKSPACE : MOE_OK;
}

static int dense_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

static TileArgs tile_args(const moe_dense_dims* d, int64_t T, bool backward, void* ws) {
  const DenseWs L = dense_ws(d, T, backward);
  auto at = [&](size_t off) { return off ? (uint16_t*)((uint8_t*)ws + off) : nullptr; };
  TileArgs a{};
  a.part = (float*)at(L.part);
  a.part_bytes = part_bytes(d, T, backward);
  a.pack_a = at(L.x);  // the forward's A is x, its B the weights
  a.pack_b[0] = at(L.w[0]);
  a.pack_b[1] = at(L.w[1]);
  return a;
}

static uint8_t* ws_at(void* ws, size_t off) { return (uint8_t*)ws + off; }

// dx = sum over mats of dz[m] W[m], dW[m] = dz[m]^T x, and the bias gradients (db.runs 0: none).
static int run_products(const moe_dense_dims* d, int mats, const void* x, int64_t ldx, int32_t T, const void* const* w,
                        const int64_t* ldw, const void* const* dz, int64_t ldz, int32_t len_dz, void* dx, int64_t ld_dx,
                        void* const* dw, const int64_t* ld_dw, const BiasSumArgs& db, void* ws, hipStream_t st) {
  TileArgs ax = tile_args(d, T, true, ws), aw = tile_args(d, T, true, ws);
  if (dx) {
    for (int m = 0; m < mats; ++m) {
      ax.a[m] = dz[m];
      ax.lda[m] = ldz;
      ax.b[m] = w[m];
      ax.ldb[m] = ldw[m];
    }
    ax.M = T;
    ax.N = d->n_in;
    ax.R = d->n_out;
    ax.len_a = len_dz;
    ax.pack_a = nullptr;
    ax.nseg = mats;
    ax.nbatch = 1;
    ax.epi.y[0] = dx;
    ax.epi.ldy[0] = ld_dx;
  }
  aw.M = d->n_out;
  aw.N = d->n_in;
  aw.R = T;
  aw.nseg = 1;
  aw.pack_b[0] = aw.pack_a;  // here B is x, once for both batches
  aw.pack_a = nullptr;
  aw.b[0] = aw.b[1] = x;
  aw.ldb[0] = aw.ldb[1] = ldx;
  for (int m = 0; m < mats; ++m) {
    if (!dw[m]) continue;
    aw.a[aw.nbatch] = dz[m];
    aw.lda[aw.nbatch] = ldz;
    aw.epi.y[aw.nbatch] = dw[m];
    aw.epi.ldy[aw.nbatch] = ld_dw[m];
    ++aw.nbatch;
  }
  return dense_status(d->dtype == MOE_BF16 ? launch_backward_bf16(ax, aw, db, st) : launch_backward_f16(ax, aw, db, st));
}

static int run_forward(const moe_dense_dims* d, const TileArgs& a, int kind, hipStream_t st) {
  if (a.M <= MOE_DENSE_ROW_TOKENS) return dense_status(launch_rows(d->dtype, a, kind, st));
  return dense_status(d->dtype == MOE_BF16 ? launch_forward_bf16(a, kind, st) : launch_forward_f16(a, kind, st));
}

}  // namespace moe

using namespace moe;

extern "C" {

MOE_API size_t moe_dense_workspace_bytes(const moe_dense_dims* dims, int32_t max_tokens, int32_t backward) {
  if (check_dense(dims) != MOE_OK || check_tokens(max_tokens) != MOE_OK) return 0;
  return dense_ws(dims, max_tokens, backward != 0).total;
}

MOE_API int moe_debug_force_dense_plan(int32_t kernel, int32_t splits) {
  if (kernel < MOE_DENSE_AUTO || kernel > MOE_DENSE_ANY128 || splits < 0 || splits > kMaxSplits) return MOE_EINVAL;
  g_dense_plan = {kernel, splits, 0};
  return MOE_OK;
}

MOE_API int moe_linear_forward(const moe_dense_dims* dims, const void* x, int64_t ldx, int32_t n_tokens, const void* w,
                               int64_t ldw, const void* bias_or_null, const void* residual_or_null, int64_t ld_residual,
                               void* y, int64_t ldy, int32_t y_dtype, void* pre_or_null, int64_t ld_pre, void* ws,
                               size_t ws_bytes, void* stream) {
  int rc = check_dense(dims);
  if (rc || (rc = check_tokens(n_tokens))) return rc;
  if (y_dtype != dims->dtype && y_dtype != MOE_F32) return MOE_EUNSUPPORTED;
  const int ye = y_dtype == MOE_F32 ? 4 : 2;
  Mats m;
  m.need(x, ldx, dims->n_in);
  m.need(w, ldw, dims->n_in);
  m.need(y, ldy, dims->n_out, ye);
  m.opt(residual_or_null, ld_residual, dims->n_out, ye);
  m.opt(pre_or_null, ld_pre, dims->n_out);
  m.vec(bias_or_null);
  if (m.rc) return m.rc;
  if ((rc = check_dense_ws(dims, n_tokens, false, ws, ws_bytes))) return rc;
  TileArgs a = tile_args(dims, n_tokens, false, ws);
  a.a[0] = x;
  a.lda[0] = ldx;
  a.b[0] = w;
  a.ldb[0] = ldw;
  a.M = n_tokens;
  a.N = dims->n_out;
  a.R = a.len_a = a.len_b = dims->n_in;
  a.nseg = a.nbatch = 1;
  a.epi.y[0] = y;
  a.epi.ldy[0] = ldy;
  a.epi.y_f32 = y_dtype == MOE_F32;
  a.epi.bias[0] = bias_or_null;
  a.epi.res = residual_or_null;
  a.epi.ldr = ld_residual;
  a.epi.pre[0] = pre_or_null;
  a.epi.ldp[0] = ld_pre;
  a.epi.act = dims->act;
  return run_forward(dims, a, kEpiLinear, (hipStream_t)stream);
}

MOE_API int moe_gated_forward(const moe_dense_dims* dims, const void* x, int64_t ldx, int32_t n_tokens,
                              const void* w_gate, int64_t ld_wg, const void* w_up, int64_t ld_wu,
                              const void* bias_gate_or_null, const void* bias_up_or_null, void* h, int64_t ldh,
                              void* gate_or_null, int64_t ld_gate, void* up_or_null, int64_t ld_up, void* ws,
                              size_t ws_bytes, void* stream) {
  int rc = check_dense(dims);
  if (rc || (rc = check_tokens(n_tokens))) return rc;
  if (!gate_or_null != !up_or_null) return MOE_EINVAL;
  Mats m;
  m.need(x, ldx, dims->n_in);
  m.need(w_gate, ld_wg, dims->n_in);
  m.need(w_up, ld_wu, dims->n_in);
  m.need(h, ldh, dims->n_out);
  m.opt(gate_or_null, ld_gate, dims->n_out);
  m.opt(up_or_null, ld_up, dims->n_out);
  m.vec(bias_gate_or_null);
  m.vec(bias_up_or_null);
  if (m.rc) return m.rc;
  if ((rc = check_dense_ws(dims, n_tokens, false, ws, ws_bytes))) return rc;
  TileArgs a = tile_args(dims, n_tokens, false, ws);
  a.a[0] = x;
  a.lda[0] = ldx;
  a.b[0] = w_gate;
  a.b[1] = w_up;
  a.ldb[0] = ld_wg;
  a.ldb[1] = ld_wu;
  a.M = n_tokens;
  a.N = dims->n_out;
  a.R = a.len_a = a.len_b = dims->n_in;
  a.nseg = a.nbatch = 1;
  a.epi.y[0] = h;
  a.epi.ldy[0] = ldh;
  a.epi.bias[0] = bias_gate_or_null;
  a.epi.bias[1] = bias_up_or_null;
  a.epi.pre[0] = gate_or_null;
  a.epi.pre[1] = up_or_null;
  a.epi.ldp[0] = ld_gate;
  a.epi.ldp[1] = ld_up;
  a.epi.act = dims->act;
  return run_forward(dims, a, kEpiGated, (hipStream_t)stream);
}

MOE_API int moe_linear_backward(const moe_dense_dims* dims, const void* x, int64_t ldx, int32_t n_tokens, const void* w,
                                int64_t ldw, const void* pre_or_null, int64_t ld_pre, const void* dy, int64_t ld_dy,
                                void* dx_or_null, int64_t ld_dx, void* dw_or_null, int64_t ld_dw, void* dbias_or_null,
                                void* ws, size_t ws_bytes, void* stream) {
  int rc = check_dense(dims);
  if (rc || (rc = check_tokens(n_tokens))) return rc;
  if (!dx_or_null && !dw_or_null && !dbias_or_null) return MOE_EINVAL;
  const bool act = dims->act != MOE_ACT_NONE;
  Mats m;
  m.need(x, ldx, dims->n_in);
  m.need(w, ldw, dims->n_in);
  if (act) m.need(pre_or_null, ld_pre, dims->n_out);
  m.need(dy, ld_dy, dims->n_out);
  m.opt(dx_or_null, ld_dx, dims->n_in);
  m.opt(dw_or_null, ld_dw, dims->n_in);
  m.vec(dbias_or_null);
  if (m.rc) return m.rc;
  if ((rc = check_dense_ws(dims, n_tokens, true, ws, ws_bytes))) return rc;
  hipStream_t st = (hipStream_t)stream;
  const DenseWs L = dense_ws(dims, n_tokens, true);
  // without an activation dz is dy itself, and is copied only to give its rows whole 16-byte chunks
  const bool products = dx_or_null || dw_or_null;
  const bool whole = (uintptr_t)dy % 16 == 0 && ld_dy % 8 == 0 && dims->n_out % 8 == 0;
  const bool make = products && (act || !whole);
  BiasSumArgs db{};
  if (make || dbias_or_null) {
    GradArgs g{};
    g.dy = dy;
    g.pre0 = act ? pre_or_null : nullptr;
    g.ld_dy = ld_dy;
    g.ldp0 = ld_pre;
    g.ldz = L.ldz;
    g.dz0 = make ? ws_at(ws, L.dz0) : nullptr;
    g.part = dbias_or_null ? (float*)ws_at(ws, L.bias_part) : nullptr;
    g.T = n_tokens;
    g.N = dims->n_out;
    g.act = dims->act;
    g.rows = grad_rows(n_tokens, dims->n_out);
    if ((rc = dense_status(launch_grad_in(dims->dtype, g, false, st)))) return rc;
    if (dbias_or_null) db = {g.part, {dbias_or_null, nullptr}, (n_tokens + g.rows - 1) / g.rows, 1, dims->n_out};
  }
  const void* dz = make ? ws_at(ws, L.dz0) : dy;
  return run_products(dims, 1, x, ldx, n_tokens, &w, &ldw, &dz, make ? L.ldz : ld_dy,
                      make ? (int32_t)L.ldz : dims->n_out, dx_or_null, ld_dx, &dw_or_null, &ld_dw, db, ws, st);
}

MOE_API int moe_gated_backward(const moe_dense_dims* dims, const void* x, int64_t ldx, int32_t n_tokens,
                               const void* w_gate, int64_t ld_wg, const void* w_up, int64_t ld_wu, const void* gate,
                               int64_t ld_gate, const void* up, int64_t ld_up, const void* dh, int64_t ld_dh,
                               void* dx_or_null, int64_t ld_dx, void* dw_gate_or_null, int64_t ld_dwg,
                               void* dw_up_or_null, int64_t ld_dwu, void* dbias_gate_or_null, void* dbias_up_or_null,
                               void* ws, size_t ws_bytes, void* stream) {
  int rc = check_dense(dims);
  if (rc || (rc = check_tokens(n_tokens))) return rc;
  const bool sums = dbias_gate_or_null || dbias_up_or_null;
  const bool products = dx_or_null || dw_gate_or_null || dw_up_or_null;
  if (!products && !sums) return MOE_EINVAL;
  Mats m;
  m.need(x, ldx, dims->n_in);
  m.need(w_gate, ld_wg, dims->n_in);
  m.need(w_up, ld_wu, dims->n_in);
  m.need(gate, ld_gate, dims->n_out);
  m.need(up, ld_up, dims->n_out);
  m.need(dh, ld_dh, dims->n_out);
  m.opt(dx_or_null, ld_dx, dims->n_in);
  m.opt(dw_gate_or_null, ld_dwg, dims->n_in);
  m.opt(dw_up_or_null, ld_dwu, dims->n_in);
  m.vec(dbias_gate_or_null);
  m.vec(dbias_up_or_null);
  if (m.rc) return m.rc;
  if ((rc = check_dense_ws(dims, n_tokens, true, ws, ws_bytes))) return rc;
  hipStream_t st = (hipStream_t)stream;
  const DenseWs L = dense_ws(dims, n_tokens, true);
  GradArgs g{};
  g.dy = dh;
  g.pre0 = gate;
  g.pre1 = up;
  g.ld_dy = ld_dh;
  g.ldp0 = ld_gate;
  g.ldp1 = ld_up;
  g.ldz = L.ldz;
  g.dz0 = products ? ws_at(ws, L.dz0) : nullptr;
  g.dz1 = products ? ws_at(ws, L.dz1) : nullptr;
  g.part = sums ? (float*)ws_at(ws, L.bias_part) : nullptr;
  g.T = n_tokens;
  g.N = dims->n_out;
  g.act = dims->act;
  g.rows = grad_rows(n_tokens, dims->n_out);
  if ((rc = dense_status(launch_grad_in(dims->dtype, g, true, st)))) return rc;
  BiasSumArgs db{};
  if (sums) db = {g.part, {dbias_gate_or_null, dbias_up_or_null}, (n_tokens + g.rows - 1) / g.rows, 2, dims->n_out};
  const void* w[2] = {w_gate, w_up};
  const int64_t ldw[2] = {ld_wg, ld_wu};
  const void* dz[2] = {g.dz0, g.dz1};
  void* dw[2] = {dw_gate_or_null, dw_up_or_null};
  const int64_t ld_dw[2] = {ld_dwg, ld_dwu};
  return run_products(dims, 2, x, ldx, n_tokens, w, ldw, dz, L.ldz, (int32_t)L.ldz, dx_or_null, ld_dx, dw, ld_dw, db, ws, st);
}

}  // extern "C"
