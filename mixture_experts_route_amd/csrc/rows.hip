// Rows by expert (moe_dispatch_*, moe_combine_*): token rows gathered into the order of perm, and each token's rows
// added up again with its router weights; their gradients are the same two movements the other way round.
//
// All of it is bound by memory.  A group of `span` threads (a power of two) takes a row or a token, 8 elements (16
// bytes) per thread and pass; spans below a wave keep narrow rows from idling lanes.  A token's row numbers and weights
// are read once per wave and broadcast from a lane, so that the loads of the rows themselves need no address
// arithmetic per lane beyond the column.
#include "checks.hpp"
#include "dense.hpp"

namespace moe {

struct RowsArgs {
  const void* src;      // x; dxs, ys; dy
  const void* ys;       // combine's backward
  const void* res;
  void* dst;            // xs; dx, y; dys
  const int32_t* perm;
  int32_t* inv;
  const float* w;
  float* dw;
  int32_t* ctrl;
  int64_t ld_src, ld_ys, ld_res, ld_dst;
  int32_t T, k, P, H;
  int32_t shift;        // log2 of the span
  int32_t blocks;       // combine's backward: workgroups that take tokens; the others look after padding rows
};

constexpr int kInvPairs = 2048;  // pairs and rows whose inverse map one workgroup makes in LDS

// inv of up to kInvPairs pairs by one workgroup: no second launch for the initial -1.
MOE_DEV void invert_small(const RowsArgs& a, int32_t* map) {
  const int pairs = a.T * a.k;
  int bad = 0;
  for (int p = threadIdx.x; p < pairs; p += 256) map[p] = -1;
  __syncthreads();
#pragma unroll 4
  for (int r = threadIdx.x; r < a.P; r += 256) {
    const int p = a.perm[r];
    if (p >= 0 && p < pairs && atomicMax(&map[p], r) != -1) bad = MOE_DERR_ROWS;
  }
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += 256) a.inv[p] = map[p];
  if (bad) set_error(a.ctrl, bad);
}

__global__ __launch_bounds__(256) void k_inv_clear(int32_t* inv, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) inv[i] = -1;
}

// xs[r] = x[perm[r] / k], four rows of a thread in flight.  SMALL: the last workgroup makes inv; otherwise it is -1
// already, and each row enters itself (the highest row where a pair has several, whatever the order).
template <typename T, bool SMALL>
__global__ __launch_bounds__(256) void k_dispatch(RowsArgs a) {
  __shared__ int32_t map[SMALL ? kInvPairs : 1];
  if constexpr (SMALL) {
    if (blockIdx.x == gridDim.x - 1) {
      invert_small(a, map);
      return;
    }
  }
  typedef typename Operand<T>::v8 v8;
  typedef v8 v8_any __attribute__((aligned(2)));
  constexpr int U = 4;
  const int span = 1 << a.shift, per = 256 >> a.shift;
  const int lane = threadIdx.x & (span - 1), slot = threadIdx.x >> a.shift;
  const int64_t movers = gridDim.x - (SMALL ? 1 : 0);
  const int64_t pairs = (int64_t)a.T * a.k;
  for (int64_t base = (int64_t)blockIdx.x * per * U; base < a.P; base += movers * per * U) {
    int32_t pair[U];
    const T* src[U];
    T* dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = base + u * per + slot;
      pair[u] = r < a.P ? a.perm[r] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = base + u * per + slot;
      if (pair[u] >= pairs) {
        if (lane == 0) set_error(a.ctrl, MOE_DERR_ROWS);
        pair[u] = -1;
      }
      if (!SMALL && lane == 0 && pair[u] >= 0 && atomicMax(&a.inv[pair[u]], (int32_t)r) != -1) set_error(a.ctrl, MOE_DERR_ROWS);
      src[u] = (const T*)a.src + (int64_t)(pair[u] < 0 ? 0 : pair[u] / a.k) * a.ld_src;
      dst[u] = (T*)a.dst + r * a.ld_dst;
    }
    for (int c = lane * 8; c < a.H; c += span * 8) {
      const int n = a.H - c;
      if (n >= 8) {
        v8 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = *(const v8_any*)(src[u] + c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (pair[u] < 0) v[u] = v8{};
          if (base + u * per + slot < a.P) *(v8_any*)(dst[u] + c) = v[u];
        }
      } else {
        for (int u = 0; u < U; ++u)
          if (base + u * per + slot < a.P)
            for (int i = 0; i < n; ++i) dst[u][c + i] = pair[u] < 0 ? (T)0.0f : src[u][c + i];
      }
    }
  }
}

// acc += the chunks of N rows of a token, all loads before the sums.  An absent row reads row 0, which exists, and
// is left out by a select, so that nothing of it (a NaN) arrives.
template <typename T, int N, bool WEIGHTS, typename Row, typename Weight>
MOE_DEV void add_rows(const RowsArgs& a, int j0, int c, int n, Row row, Weight weight, float (&acc)[8]) {
  float v[N][8];
  int32_t r[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    r[j] = row(j0 + j);
    load8<T>(a.src, (int64_t)(r[j] < 0 ? 0 : r[j]) * a.ld_src + c, n, v[j]);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float w = WEIGHTS ? weight(j0 + j) : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = r[j] < 0 ? acc[i] : (WEIGHTS ? fmaf(w, v[j][i], acc[i]) : acc[i] + v[j][i]);
  }
}

// The row numbers and weights of one token.  WIDE: the whole wave has the same token; lane j holds choice j's.
template <bool WIDE>
struct Choices {
  const int32_t* inv;
  const float* w;
  int32_t row_l;
  float w_l;
  int32_t P;
  MOE_DEV void init(const RowsArgs& a, int64_t t, bool weights) {
    inv = a.inv + t * a.k;
    w = weights ? a.w + t * a.k : nullptr;
    P = a.P;
    if constexpr (WIDE) {
      const int l = threadIdx.x & 63;
      row_l = l < a.k ? inv[l] : -1;
      w_l = weights && l < a.k ? w[l] : 0.0f;
      if (row_l >= P) {
        set_error(a.ctrl, MOE_DERR_ROWS);
        row_l = -1;
      }
    }
  }
  MOE_DEV int32_t row(int j) const {
    if constexpr (WIDE) return __builtin_amdgcn_readlane(row_l, j);
    const int32_t r = inv[j];
    return r < P ? r : -1;
  }
  MOE_DEV float weight(int j) const {
    if constexpr (WIDE) return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w_l), j));
    return w[j];
  }
};

// y[t] = sum_j w[t][j] rows[inv[t][j]] + r[t] (WEIGHTS), or without the weights; Y the type of y and r.
template <typename T, typename Y, bool WEIGHTS, bool WIDE>
__global__ __launch_bounds__(256) void k_combine(RowsArgs a) {
  const int span = 1 << a.shift, per = 256 >> a.shift;
  const int lane = threadIdx.x & (span - 1);
  int slot = threadIdx.x >> a.shift;
  if (WIDE) slot = __builtin_amdgcn_readfirstlane(slot);
  for (int64_t t = (int64_t)blockIdx.x * per + slot; t < a.T; t += (int64_t)gridDim.x * per) {
    Choices<WIDE> ch;
    ch.init(a, t, WEIGHTS);
    if (!WIDE && lane == 0)
      for (int j = 0; j < a.k; ++j)
        if (ch.inv[j] >= a.P) set_error(a.ctrl, MOE_DERR_ROWS);
    auto row = [&](int j) { return ch.row(j); };
    auto weight = [&](int j) { return ch.weight(j); };
    for (int c = lane * 8; c < a.H; c += span * 8) {
      const int n = a.H - c < 8 ? a.H - c : 8;
      float acc[8] = {};
      int j = 0;
      for (; j + 8 <= a.k; j += 8) add_rows<T, 8, WEIGHTS>(a, j, c, n, row, weight, acc);
      if (a.k & 4) {
        add_rows<T, 4, WEIGHTS>(a, j, c, n, row, weight, acc);
        j += 4;
      }
      if (a.k & 2) {
        add_rows<T, 2, WEIGHTS>(a, j, c, n, row, weight, acc);
        j += 2;
      }
      if (a.k & 1) add_rows<T, 1, WEIGHTS>(a, j, c, n, row, weight, acc);
      if (a.res) {
        float v[8];
        load8<Y>(a.res, t * a.ld_res + c, n, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[i];
      }
      store8<Y>(a.dst, t * a.ld_dst + c, n, acc);
    }
  }
}

// dys and dw of N of a token's choices for one chunk: dot[j] += dy . ys[row], dys[row] = w dy.
template <typename T, int N>
MOE_DEV void grad_rows_of(const RowsArgs& a, int c, int n, const float (&dy)[8], const int32_t* row, const float* w, float* dot) {
  if (a.dw) {
    float v[N][8];
#pragma unroll
    for (int j = 0; j < N; ++j) load8<T>(a.ys, (int64_t)(row[j] < 0 ? 0 : row[j]) * a.ld_ys + c, n, v[j]);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float s = dot[j];
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(dy[i], v[j][i], s);  // both zero past the row's end
      dot[j] = row[j] < 0 ? 0.0f : s;
    }
  }
  if (a.dst) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (row[j] >= 0) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[j] * dy[i];
        store8<T>(a.dst, (int64_t)row[j] * a.ld_dst + c, n, v);
      }
  }
}

// A token's dy is read once per four choices and serves their rows: dys[row] = w dy, dw = dy . ys[row].  A pair takes row
// inv[p] only where perm says the same, so every row of dys is written once: by its pair, or as a padding row by the
// workgroups behind the tokens'.
template <typename T, typename Y>
__global__ __launch_bounds__(256) void k_combine_grad(RowsArgs a) {
  __shared__ float sums[4][kMaxK];
  const int64_t pairs = (int64_t)a.T * a.k;
  if ((int)blockIdx.x >= a.blocks) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t movers = (int64_t)(gridDim.x - a.blocks) * 4;
    for (int64_t r0 = ((int64_t)(blockIdx.x - a.blocks) * 4 + wave) * 64; r0 < a.P; r0 += movers * 64) {
      const int64_t r = r0 + lane;
      bool zero = false;
      if (r < a.P) {
        const int32_t p = a.perm[r];
        if (p >= 0) {
          zero = p >= pairs || a.inv[p] != r;
          if (zero) set_error(a.ctrl, MOE_DERR_ROWS);
        } else {
          zero = true;
        }
      }
      uint64_t todo = __ballot(zero);
      if (!a.dst) continue;
      while (todo) {
        const int64_t row = r0 + __ffsll((unsigned long long)todo) - 1;
        todo &= todo - 1;
        float v[8] = {};
        for (int c = lane * 8; c < a.H; c += 512) store8<T>(a.dst, row * a.ld_dst + c, a.H - c < 8 ? a.H - c : 8, v);
      }
    }
    return;
  }
  const int span = 1 << a.shift, per = 256 >> a.shift;
  const int lane = threadIdx.x & (span - 1), slot = threadIdx.x >> a.shift;
  for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.T; t0 += (int64_t)a.blocks * per) {
    const int64_t t = t0 + slot;
    const bool live = t < a.T;
    for (int j0 = 0; j0 < a.k; j0 += 4) {
      int32_t row[4];
      float w[4], dot[4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool on = live && j0 + j < a.k;
        row[j] = on ? a.inv[t * a.k + j0 + j] : -1;
        w[j] = on && a.dst ? a.w[t * a.k + j0 + j] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (row[j] >= 0 && (row[j] >= a.P || a.perm[row[j]] != t * a.k + j0 + j)) {
          if (lane == 0) set_error(a.ctrl, MOE_DERR_ROWS);
          row[j] = -1;
        }
      if (live)
        for (int c = lane * 8; c < a.H; c += span * 8) {
          const int n = a.H - c < 8 ? a.H - c : 8;
          float dy[8];
          load8<Y>(a.src, t * a.ld_src + c, n, dy);
          grad_rows_of<T, 4>(a, c, n, dy, row, w, dot);
        }
      if (!a.dw) continue;
      const int inner = span < 64 ? span : 64;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        for (int o = inner >> 1; o; o >>= 1) dot[j] += __shfl_xor(dot[j], o, 64);
      if (span > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
#pragma unroll
          for (int j = 0; j < 4; ++j) sums[threadIdx.x >> 6][j] = dot[j];
        __syncthreads();
        if (lane == 0) {
          const int first = threadIdx.x >> 6;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            for (int i = 1; i < span >> 6; ++i) dot[j] += sums[first + i][j];
        }
      }
      if (live && lane == 0)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j0 + j < a.k) a.dw[t * a.k + j0 + j] = dot[j];
    }
  }
}

// Threads per row: the power of two from 8 to `most` that idles the fewest in a row of `chunks` 16-byte chunks.
static int span_shift(int chunks, int most) {
  int best = 3;
  int64_t waste = INT64_MAX;
  for (int s = 3; (1 << s) <= most; ++s) {
    const int64_t n = ((int64_t)chunks + (1 << s) - 1) / (1 << s) << s;
    if (n <= waste) {
      waste = n;
      best = s;
    }
  }
  return best;
}
static uint32_t grid_of(int64_t blocks) { return (uint32_t)(blocks < (1 << 20) ? blocks : 1 << 20); }

template <typename T>
static hipError_t start_dispatch(RowsArgs a, hipStream_t st) {
  const int64_t pairs = (int64_t)a.T * a.k;
  a.shift = span_shift((a.H + 7) / 8, 256);
  const int64_t per = (256 >> a.shift) * 4;
  const uint32_t grid = grid_of((a.P + per - 1) / per);
  if (pairs <= kInvPairs && a.P <= kInvPairs) {
    k_dispatch<T, true><<<grid + 1, 256, 0, st>>>(a);
    return hipGetLastError();
  }
  const int64_t clear = (pairs + 1023) / 1024;
  k_inv_clear<<<(uint32_t)(clear < 4096 ? clear : 4096), 256, 0, st>>>(a.inv, pairs);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_dispatch<T, false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, typename Y, bool WEIGHTS>
static hipError_t start_combine(RowsArgs a, hipStream_t st) {
  a.shift = span_shift((a.H + 7) / 8, a.T < 2048 ? 256 : 64);
  const int64_t per = 256 >> a.shift;
  const uint32_t grid = grid_of((a.T + per - 1) / per);
  if (a.shift >= 6) k_combine<T, Y, WEIGHTS, true><<<grid, 256, 0, st>>>(a);
  else k_combine<T, Y, WEIGHTS, false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, typename Y>
static hipError_t start_combine_grad(RowsArgs a, hipStream_t st) {
  a.shift = span_shift((a.H + 7) / 8, a.T < 2048 ? 256 : 64);
  const int64_t per = 256 >> a.shift, rows = ((int64_t)a.P + 255) / 256;
  a.blocks = (int32_t)grid_of((a.T + per - 1) / per);
  k_combine_grad<T, Y><<<a.blocks + (uint32_t)(rows < 1024 ? rows : 1024), 256, 0, st>>>(a);
  return hipGetLastError();
}

static int check_rows(const moe_rows_dims* d) {
  if (!d || d->width < 1 || d->top_k < 1) return MOE_EINVAL;
  if (d->width > MOE_DENSE_MAX_WIDTH || d->top_k > kMaxK) return MOE_EUNSUPPORTED;
  return d->dtype == MOE_BF16 || d->dtype == MOE_F16 ? MOE_OK : MOE_EUNSUPPORTED;
}

static int check_counts(const moe_rows_dims* d, int32_t T, int32_t P) {
  int rc = check_rows(d);
  if (rc || (rc = check_tokens(T))) return rc;
  if (P < 1) return MOE_EINVAL;
  return P > MOE_ROWS_MAX ? MOE_EUNSUPPORTED : MOE_OK;
}

static int check_rows_ws(const void* ws, size_t ws_bytes) {
  return !ws || ((uintptr_t)ws & 255) || ws_bytes < kCtrlBytes ? MOE_EWORKSPACE : MOE_OK;
}

// dispatch's backward (w NULL) and combine's forward.
static int run_combine(const moe_rows_dims* d, bool weights, const void* rows, int64_t ld_rows, int32_t P,
                       const int32_t* inv, const float* w, int32_t T, const void* res, int64_t ld_res, void* y,
                       int64_t ldy, int32_t y_dtype, void* ws, size_t ws_bytes, hipStream_t st) {
  int rc = check_counts(d, T, P);
  if (rc) return rc;
  if (y_dtype != d->dtype && y_dtype != MOE_F32) return MOE_EUNSUPPORTED;
  const int ye = y_dtype == MOE_F32 ? 4 : 2;
  Mats m;
  m.need(rows, ld_rows, d->width);
  m.need(inv, 1, 1, 4);
  if (weights) m.need(w, 1, 1, 4);
  m.opt(res, ld_res, d->width, ye);
  m.need(y, ldy, d->width, ye);
  if (m.rc) return m.rc;
  if ((rc = check_rows_ws(ws, ws_bytes))) return rc;
  RowsArgs a{};
  a.src = rows;
  a.ld_src = ld_rows;
  a.inv = (int32_t*)inv;
  a.w = w;
  a.res = res;
  a.ld_res = ld_res;
  a.dst = y;
  a.ld_dst = ldy;
  a.ctrl = (int32_t*)ws;
  a.T = T;
  a.k = d->top_k;
  a.P = P;
  a.H = d->width;
  const bool f32 = y_dtype == MOE_F32;
  if (d->dtype == MOE_BF16) {
    if (weights) return dense_status(f32 ? start_combine<__bf16, float, true>(a, st) : start_combine<__bf16, __bf16, true>(a, st));
    return dense_status(f32 ? start_combine<__bf16, float, false>(a, st) : start_combine<__bf16, __bf16, false>(a, st));
  }
  if (weights) return dense_status(f32 ? start_combine<_Float16, float, true>(a, st) : start_combine<_Float16, _Float16, true>(a, st));
  return dense_status(f32 ? start_combine<_Float16, float, false>(a, st) : start_combine<_Float16, _Float16, false>(a, st));
}

}  // namespace moe

using namespace moe;

extern "C" {

MOE_API size_t moe_rows_workspace_bytes(const moe_rows_dims* dims, int32_t max_tokens) {
  return check_rows(dims) != MOE_OK || check_tokens(max_tokens) != MOE_OK ? 0 : kCtrlBytes;
}

MOE_API int moe_dispatch_forward(const moe_rows_dims* dims, const void* x, int64_t ldx, int32_t n_tokens,
                                 const int32_t* perm, int32_t n_rows, void* xs, int64_t ld_xs, int32_t* inv, void* ws,
                                 size_t ws_bytes, void* stream) {
  int rc = check_counts(dims, n_tokens, n_rows);
  if (rc) return rc;
  Mats m;
  m.need(x, ldx, dims->width);
  m.need(perm, 1, 1, 4);
  m.need(xs, ld_xs, dims->width);
  m.need(inv, 1, 1, 4);
  if (m.rc) return m.rc;
  if ((rc = check_rows_ws(ws, ws_bytes))) return rc;
  RowsArgs a{};
  a.src = x;
  a.ld_src = ldx;
  a.perm = perm;
  a.dst = xs;
  a.ld_dst = ld_xs;
  a.inv = inv;
  a.ctrl = (int32_t*)ws;
  a.T = n_tokens;
  a.k = dims->top_k;
  a.P = n_rows;
  a.H = dims->width;
  hipStream_t st = (hipStream_t)stream;
  return dense_status(dims->dtype == MOE_BF16 ? start_dispatch<__bf16>(a, st) : start_dispatch<_Float16>(a, st));
}

MOE_API int moe_dispatch_backward(const moe_rows_dims* dims, const void* dxs, int64_t ld_dxs, int32_t n_rows,
                                  const int32_t* inv, int32_t n_tokens, const void* residual_or_null,
                                  int64_t ld_residual, void* dx, int64_t ld_dx, int32_t dx_dtype, void* ws,
                                  size_t ws_bytes, void* stream) {
  return run_combine(dims, false, dxs, ld_dxs, n_rows, inv, nullptr, n_tokens, residual_or_null, ld_residual, dx, ld_dx,
                     dx_dtype, ws, ws_bytes, (hipStream_t)stream);
}

MOE_API int moe_combine_forward(const moe_rows_dims* dims, const void* ys, int64_t ld_ys, int32_t n_rows,
                                const int32_t* inv, const float* topk_w, int32_t n_tokens, const void* residual_or_null,
                                int64_t ld_residual, void* y, int64_t ldy, int32_t y_dtype, void* ws, size_t ws_bytes,
                                void* stream) {
  return run_combine(dims, true, ys, ld_ys, n_rows, inv, topk_w, n_tokens, residual_or_null, ld_residual, y, ldy, y_dtype,
                     ws, ws_bytes, (hipStream_t)stream);
}

MOE_API int moe_combine_backward(const moe_rows_dims* dims, const void* dy, int64_t ld_dy, int32_t dy_dtype,
                                 int32_t n_tokens, const int32_t* perm, const int32_t* inv, int32_t n_rows,
                                 const float* topk_w, const void* ys_or_null, int64_t ld_ys, void* dys_or_null,
                                 int64_t ld_dys, float* dtopk_w_or_null, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_counts(dims, n_tokens, n_rows);
  if (rc) return rc;
  if (dy_dtype != dims->dtype && dy_dtype != MOE_F32) return MOE_EUNSUPPORTED;
  if (!dys_or_null && !dtopk_w_or_null) return MOE_EINVAL;
  Mats m;
  m.need(dy, ld_dy, dims->width, dy_dtype == MOE_F32 ? 4 : 2);
  m.need(perm, 1, 1, 4);
  m.need(inv, 1, 1, 4);
  m.need(topk_w, 1, 1, 4);
  if (dtopk_w_or_null) m.need(ys_or_null, ld_ys, dims->width);
  m.opt(dys_or_null, ld_dys, dims->width);
  m.opt(dtopk_w_or_null, 1, 1, 4);
  if (m.rc) return m.rc;
  if ((rc = check_rows_ws(ws, ws_bytes))) return rc;
  RowsArgs a{};
  a.src = dy;
  a.ld_src = ld_dy;
  a.ys = ys_or_null;
  a.ld_ys = ld_ys;
  a.perm = perm;
  a.inv = (int32_t*)inv;
  a.w = topk_w;
  a.dst = dys_or_null;
  a.ld_dst = ld_dys;
  a.dw = dtopk_w_or_null;
  a.ctrl = (int32_t*)ws;
  a.T = n_tokens;
  a.k = dims->top_k;
  a.P = n_rows;
  a.H = dims->width;
  hipStream_t st = (hipStream_t)stream;
  const bool f32 = dy_dtype == MOE_F32;
  if (dims->dtype == MOE_BF16)
    return dense_status(f32 ? start_combine_grad<__bf16, float>(a, st) : start_combine_grad<__bf16, __bf16>(a, st));
  return dense_status(f32 ? start_combine_grad<_Float16, float>(a, st) : start_combine_grad<_Float16, _Float16>(a, st));
}

}  // extern "C"
