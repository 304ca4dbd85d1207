// The experts' products' C interface (moe_experts_*): host-side validation, workspace carving and launches.
#include "experts.hpp"

namespace moe {

// Workspace: control words, then for a backward pass dz (gated: dg, du) with rows padded to whole 16-byte chunks.  dims do not say
// which call: the linear one uses one matrix of dz where dys has no whole chunks, else none.  dg and du are rounded to 16 bits for the
// matrix cores, which costs dx and dW the whole of their distance to sums of unrounded ones: 512 experts, 40960 rows, bf16 2.3e-3 off the
// definition, from unrounded dz 1.7e-3 (the results' own rounding).
struct ExpertsWs {
  size_t dz0, dz1, total;
  int64_t ldz;
};
static ExpertsWs experts_ws(const moe_experts_dims* d, int64_t P, bool backward) {
  ExpertsWs L{};
  L.total = kCtrlBytes;
  if (backward) {
    L.ldz = ((int64_t)d->n_out + 7) / 8 * 8;
    L.dz0 = L.total;
    L.dz1 = dense_align(L.dz0 + 2 * (size_t)(P * L.ldz));
    L.total = dense_align(L.dz1 + 2 * (size_t)(P * L.ldz));
  }
  return L;
}

static int check_experts(const moe_experts_dims* d) {
  if (!d || d->n_experts < 1 || d->n_in < 1 || d->n_out < 1) return MOE_EINVAL;
  if (d->n_experts > kMaxExperts || d->n_in > MOE_DENSE_MAX_WIDTH || d->n_out > MOE_DENSE_MAX_WIDTH) return MOE_EUNSUPPORTED;
  if (d->dtype != MOE_BF16 && d->dtype != MOE_F16) return MOE_EUNSUPPORTED;
  return d->act < MOE_ACT_NONE || d->act > MOE_ACT_SIGMOID ? MOE_EUNSUPPORTED : MOE_OK;
}

static int check_experts_rows(const moe_experts_dims* d, int32_t P, bool gated) {
  const int rc = check_experts(d);
  if (rc) return rc;
  if (!gated && d->act != MOE_ACT_NONE) return MOE_EUNSUPPORTED;
  if (P < 1) return MOE_EINVAL;
  return P > MOE_ROWS_MAX ? MOE_EUNSUPPORTED : MOE_OK;
}

// An [E][n_out][n_in] tensor.
static void check_weights(Mats& m, const moe_experts_dims* d, const void* p, int64_t ld, int64_t stride, bool optional) {
  if (optional && !p) return;
  m.need(p, ld, d->n_in);
  if (m.rc) return;
  if (stride < (d->n_out - 1) * ld + d->n_in) m.fail(MOE_EINVAL);
  else if (stride > ((int64_t)1 << 44)) m.fail(MOE_EUNSUPPORTED);
}

static int check_experts_ws(const moe_experts_dims* d, int32_t P, bool backward, const void* ws, size_t ws_bytes) {
  if (!ws || ((uintptr_t)ws & 255)) return MOE_EWORKSPACE;
  return ws_bytes < experts_ws(d, P, backward).total ? MOE_EWORKSPACE : MOE_OK;
}

static GroupArgs group_args(const moe_experts_dims* d, const int32_t* offsets, int32_t P, void* ws) {
  GroupArgs g{};
  g.offsets = offsets;
  g.ctrl = (int32_t*)ws;
  g.E = d->n_experts;
  g.P = P;
  g.mats = 1;
  g.tile.nseg = g.tile.nbatch = 1;
  return g;
}

static int run_experts_forward(const moe_experts_dims* d, GroupArgs& g, int kind, const void* x, int64_t ldx,
                               const void* const* w, int64_t ldw, int64_t stride, hipStream_t st) {
  g.tile.a[0] = x;
  g.tile.lda[0] = ldx;
  for (int m = 0; m < (kind == kEpiGated ? 2 : 1); ++m) {
    g.tile.b[m] = w[m];
    g.tile.ldb[m] = ldw;
  }
  g.stride = stride;
  g.tile.N = d->n_out;
  g.tile.R = g.tile.len_a = g.tile.len_b = d->n_in;
  return dense_status(d->dtype == MOE_BF16 ? launch_experts_forward_bf16(g, kind, st) : launch_experts_forward_f16(g, kind, st));
}

// dx = sum over mats of dz[m] W[m], dW[m] = dz[m]^T x, expert by expert.
static int run_experts_products(const moe_experts_dims* d, int mats, const GroupArgs& base, const void* x, int64_t ldx,
                                const void* const* w, int64_t ldw, int64_t stride, const void* const* dz, int64_t ldz,
                                int32_t len_dz, void* dx, int64_t ld_dx, void* const* dw, int64_t ld_dw, int64_t dw_stride,
                                hipStream_t st) {
  GroupArgs gx = base, gw = base;
  gx.tile.nseg = gw.mats = 0;
  if (dx) {
    for (int m = 0; m < mats; ++m) {
      gx.tile.a[m] = dz[m];
      gx.tile.lda[m] = ldz;
      gx.tile.b[m] = w[m];
      gx.tile.ldb[m] = ldw;
    }
    gx.stride = stride;
    gx.tile.N = d->n_in;
    gx.tile.R = d->n_out;
    gx.tile.len_a = len_dz;
    gx.tile.nseg = mats;
    gx.tile.epi.y[0] = dx;
    gx.tile.epi.ldy[0] = ld_dx;
  }
  for (int m = 0; m < mats; ++m)
    if (dw[m]) {
      gw.tile.a[gw.mats] = dz[m];
      gw.tile.epi.y[gw.mats++] = dw[m];
    }
  gw.tile.lda[0] = ldz;
  gw.tile.b[0] = x;
  gw.tile.ldb[0] = ldx;
  gw.stride = dw_stride;
  gw.tile.M = d->n_out;
  gw.tile.N = d->n_in;
  gw.tile.epi.ldy[0] = ld_dw;
  return dense_status(d->dtype == MOE_BF16 ? launch_experts_backward_bf16(gx, gw, st) : launch_experts_backward_f16(gx, gw, st));
}

}  // namespace moe

using namespace moe;

extern "C" {

MOE_API size_t moe_experts_workspace_bytes(const moe_experts_dims* dims, int32_t max_rows, int32_t backward) {
  if (check_experts(dims) != MOE_OK || max_rows < 1 || max_rows > MOE_ROWS_MAX) return 0;
  return experts_ws(dims, max_rows, backward != 0).total;
}

MOE_API int moe_experts_linear_forward(const moe_experts_dims* dims, const void* xs, int64_t ld_xs, int32_t n_rows,
                                       const int32_t* offsets, const void* w, int64_t ldw, int64_t w_stride, void* ys,
                                       int64_t ld_ys, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_experts_rows(dims, n_rows, false);
  if (rc) return rc;
  Mats m;
  m.need(xs, ld_xs, dims->n_in);
  m.need(offsets, 1, 1, 4);
  check_weights(m, dims, w, ldw, w_stride, false);
  m.need(ys, ld_ys, dims->n_out);
  if (m.rc) return m.rc;
  if ((rc = check_experts_ws(dims, n_rows, false, ws, ws_bytes))) return rc;
  GroupArgs g = group_args(dims, offsets, n_rows, ws);
  g.tile.epi.y[0] = ys;
  g.tile.epi.ldy[0] = ld_ys;
  return run_experts_forward(dims, g, kEpiStore, xs, ld_xs, &w, ldw, w_stride, (hipStream_t)stream);
}

MOE_API int moe_experts_gated_forward(const moe_experts_dims* dims, const void* xs, int64_t ld_xs, int32_t n_rows,
                                      const int32_t* offsets, const void* w_gate, const void* w_up, int64_t ldw,
                                      int64_t w_stride, void* h, int64_t ldh, void* gate_or_null, void* up_or_null,
                                      int64_t ld_saved, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_experts_rows(dims, n_rows, true);
  if (rc) return rc;
  if (!gate_or_null != !up_or_null) return MOE_EINVAL;
  Mats m;
  m.need(xs, ld_xs, dims->n_in);
  m.need(offsets, 1, 1, 4);
  check_weights(m, dims, w_gate, ldw, w_stride, false);
  check_weights(m, dims, w_up, ldw, w_stride, false);
  m.need(h, ldh, dims->n_out);
  m.opt(gate_or_null, ld_saved, dims->n_out);
  m.opt(up_or_null, ld_saved, dims->n_out);
  if (m.rc) return m.rc;
  if ((rc = check_experts_ws(dims, n_rows, false, ws, ws_bytes))) return rc;
  GroupArgs g = group_args(dims, offsets, n_rows, ws);
  g.tile.epi.y[0] = h;
  g.tile.epi.ldy[0] = ldh;
  g.tile.epi.pre[0] = gate_or_null;
  g.tile.epi.pre[1] = up_or_null;
  g.tile.epi.ldp[0] = g.tile.epi.ldp[1] = ld_saved;
  g.tile.epi.act = dims->act;
  const void* w[2] = {w_gate, w_up};
  return run_experts_forward(dims, g, kEpiGated, xs, ld_xs, w, ldw, w_stride, (hipStream_t)stream);
}

MOE_API int moe_experts_linear_backward(const moe_experts_dims* dims, const void* xs, int64_t ld_xs, int32_t n_rows,
                                        const int32_t* offsets, const void* w, int64_t ldw, int64_t w_stride,
                                        const void* dys, int64_t ld_dys, void* dxs_or_null, int64_t ld_dxs,
                                        void* dw_or_null, int64_t ld_dw, int64_t dw_stride, void* ws, size_t ws_bytes,
                                        void* stream) {
  int rc = check_experts_rows(dims, n_rows, false);
  if (rc) return rc;
  if (!dxs_or_null && !dw_or_null) return MOE_EINVAL;
  Mats m;
  m.need(xs, ld_xs, dims->n_in);
  m.need(offsets, 1, 1, 4);
  check_weights(m, dims, w, ldw, w_stride, false);
  m.need(dys, ld_dys, dims->n_out);
  m.opt(dxs_or_null, ld_dxs, dims->n_in);
  check_weights(m, dims, dw_or_null, ld_dw, dw_stride, true);
  if (m.rc) return m.rc;
  if ((rc = check_experts_ws(dims, n_rows, true, ws, ws_bytes))) return rc;
  hipStream_t st = (hipStream_t)stream;
  const ExpertsWs L = experts_ws(dims, n_rows, true);
  const void* dz = dys;
  int64_t ldz = ld_dys;
  int32_t len = dims->n_out;
  if ((uintptr_t)dys % 16 || ld_dys % 8 || dims->n_out % 8) {  // a copy whose rows are whole 16-byte chunks
    GradArgs a{};
    a.dy = dys;
    a.ld_dy = ld_dys;
    a.ldz = ldz = len = L.ldz;
    dz = a.dz0 = (uint8_t*)ws + L.dz0;
    a.T = n_rows;
    a.N = dims->n_out;
    a.rows = grad_rows(n_rows, dims->n_out);
    if ((rc = dense_status(launch_grad_in(dims->dtype, a, false, st)))) return rc;
  }
  return run_experts_products(dims, 1, group_args(dims, offsets, n_rows, ws), xs, ld_xs, &w, ldw, w_stride, &dz, ldz, len,
                              dxs_or_null, ld_dxs, &dw_or_null, ld_dw, dw_stride, st);
}

MOE_API int moe_experts_gated_backward(const moe_experts_dims* dims, const void* xs, int64_t ld_xs, int32_t n_rows,
                                       const int32_t* offsets, const void* w_gate, const void* w_up, int64_t ldw,
                                       int64_t w_stride, const void* gate, const void* up, int64_t ld_saved,
                                       const void* dh, int64_t ld_dh, void* dxs_or_null, int64_t ld_dxs,
                                       void* dw_gate_or_null, void* dw_up_or_null, int64_t ld_dw, int64_t dw_stride,
                                       void* ws, size_t ws_bytes, void* stream) {
  int rc = check_experts_rows(dims, n_rows, true);
  if (rc) return rc;
  if (!dxs_or_null && !dw_gate_or_null && !dw_up_or_null) return MOE_EINVAL;
  Mats m;
  m.need(xs, ld_xs, dims->n_in);
  m.need(offsets, 1, 1, 4);
  check_weights(m, dims, w_gate, ldw, w_stride, false);
  check_weights(m, dims, w_up, ldw, w_stride, false);
  m.need(gate, ld_saved, dims->n_out);
  m.need(up, ld_saved, dims->n_out);
  m.need(dh, ld_dh, dims->n_out);
  m.opt(dxs_or_null, ld_dxs, dims->n_in);
  check_weights(m, dims, dw_gate_or_null, ld_dw, dw_stride, true);
  check_weights(m, dims, dw_up_or_null, ld_dw, dw_stride, true);
  if (m.rc) return m.rc;
  if ((rc = check_experts_ws(dims, n_rows, true, ws, ws_bytes))) return rc;
  hipStream_t st = (hipStream_t)stream;
  const ExpertsWs L = experts_ws(dims, n_rows, true);
  GradArgs a{};
  a.dy = dh;
  a.pre0 = gate;
  a.pre1 = up;
  a.ld_dy = ld_dh;
  a.ldp0 = a.ldp1 = ld_saved;
  a.ldz = L.ldz;
  a.dz0 = (uint8_t*)ws + L.dz0;
  a.dz1 = (uint8_t*)ws + L.dz1;
  a.T = n_rows;
  a.N = dims->n_out;
  a.act = dims->act;
  a.rows = grad_rows(n_rows, dims->n_out);
  if ((rc = dense_status(launch_grad_in(dims->dtype, a, true, st)))) return rc;
  const void* w[2] = {w_gate, w_up};
  const void* dz[2] = {a.dz0, a.dz1};
  void* dw[2] = {dw_gate_or_null, dw_up_or_null};
  return run_experts_products(dims, 2, group_args(dims, offsets, n_rows, ws), xs, ld_xs, w, ldw, w_stride, dz, L.ldz,
                              (int32_t)L.ldz, dxs_or_null, ld_dxs, dw, ld_dw, dw_stride, st);
}

}  // extern "C"
