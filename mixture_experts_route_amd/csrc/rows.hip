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
  int32_t blocks;       // workgroups that take tokens; those behind them look after padding rows
};

// A thread's chunk at column c of a row of H: the 8 elements from the returned column on.  The last chunk of an odd width begins
// earlier, inside the one before it, so that every access is a whole 16 bytes; the elements that both have are written
// twice with the same value.  Rows under 8 elements are one short chunk.
MOE_DEV int chunk_at(int c, int H) { return c + 8 <= H || H < 8 ? c : H - 8; }
MOE_DEV int chunk_len(int H) { return H < 8 ? H : 8; }

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

// Each row enters itself: the highest one where a pair has several, whatever the order.
__global__ __launch_bounds__(256) void k_inv_fill(RowsArgs a) {
  const int64_t pairs = (int64_t)a.T * a.k;
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < a.P; r += (int64_t)gridDim.x * 256) {
    const int p = a.perm[r];
    if (p >= 0 && p < pairs) atomicMax(&a.inv[p], (int32_t)r);
  }
}

// Zeros in the rows that are no pair's, by the workgroups from a.blocks on: padding rows, and the rows of a bad layout
// (a pair out of range, a pair that another row has), which are reported.
template <typename T>
MOE_DEV void zero_rows(const RowsArgs& a) {
  const int64_t pairs = (int64_t)a.T * a.k;
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
      for (int c = lane * 8; c < a.H; c += 512) store8<T>(a.dst, row * a.ld_dst + chunk_at(c, a.H), chunk_len(a.H), v);
    }
  }
}

// The dispatch of a few pairs in one launch, row by row: xs[r] = x[perm[r] / k], four rows of a thread in flight; the last
// workgroup makes inv.  Bound by latency: 8 tokens' ten rows of 2048 in 4.1 us.
template <typename T>
__global__ __launch_bounds__(256) void k_dispatch_few(RowsArgs a) {
  __shared__ int32_t map[kInvPairs];
  if (blockIdx.x == gridDim.x - 1) {
    invert_small(a, map);
    return;
  }
  typedef typename Operand<T>::v8 v8;
  typedef v8 v8_any __attribute__((aligned(2)));
  constexpr int U = 4;
  const int span = 1 << a.shift, per = 256 >> a.shift;
  const int lane = threadIdx.x & (span - 1), slot = threadIdx.x >> a.shift;
  const int base = blockIdx.x * per * U, pairs = a.T * a.k;
  int32_t pair[U];
  const T* src[U];
  T* dst[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = base + u * per + slot;
    pair[u] = r < a.P ? a.perm[r] : -1;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (pair[u] >= pairs) {
      if (lane == 0) set_error(a.ctrl, MOE_DERR_ROWS);
      pair[u] = -1;
    }
    src[u] = (const T*)a.src + (int64_t)(pair[u] < 0 ? 0 : pair[u] / a.k) * a.ld_src;
    dst[u] = (T*)a.dst + (int64_t)(base + u * per + slot) * a.ld_dst;
  }
  for (int col = lane * 8; col < a.H; col += span * 8) {
    const int c = chunk_at(col, a.H);
    if (a.H >= 8) {
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
          for (int i = 0; i < a.H; ++i) dst[u][i] = pair[u] < 0 ? (T)0.0f : src[u][i];
    }
  }
}

// The 8 elements of a chunk as they are stored (the first n, zeros after them).
template <typename T>
MOE_DEV typename Operand<T>::v8 load_raw(const void* base, int64_t off, int n) {
  typedef typename Operand<T>::v8 v8;
  typedef v8 v8_any __attribute__((aligned(2)));
  const T* p = (const T*)base + off;
  if (n == 8) return *(const v8_any*)p;
  v8 v = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) v[i] = p[i];
  return v;
}

// acc += the chunks of N rows of a token, all loads before the sums.  An absent row reads row 0, which exists, and
// is left out by a select, so that nothing of it (a NaN) arrives.
template <typename T, int N, bool WEIGHTS, typename Row, typename Weight>
MOE_DEV void add_rows(const RowsArgs& a, int j0, int c, int n, Row row, Weight weight, float (&acc)[8]) {
  typename Operand<T>::v8 v[N];
  int32_t r[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    r[j] = row(j0 + j);
    v[j] = load_raw<T>(a.src, (int64_t)(r[j] < 0 ? 0 : r[j]) * a.ld_src + c, n);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float w = WEIGHTS ? weight(j0 + j) : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = r[j] < 0 ? acc[i] : (WEIGHTS ? fmaf(w, (float)v[j][i], acc[i]) : acc[i] + (float)v[j][i]);
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

// y[t] = sum_j w[t][j] rows[inv[t][j]] + r[t] (WEIGHTS), or without the weights; Y the type of y and r.  K: the number of
// choices, all of whose rows are then on their way at once, held as they are stored (4 registers a row: ten rows in 70
// registers), or 0: any number, in groups (narrow rows).  32768 tokens' ten rows of 2048 onto 16 bits 312 us, 5.2 TB/s; 4096
// tokens' onto fp32 47 us, 5.0 (in two groups, converted as they come: 328 and 59).
template <typename T, typename Y, bool WEIGHTS, int K>
__global__ __launch_bounds__(256) void k_combine(RowsArgs a) {
  constexpr bool WIDE = K > 0;
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
    for (int col = lane * 8; col < a.H; col += span * 8) {
      const int c = chunk_at(col, a.H), n = chunk_len(a.H);
      float acc[8] = {}, r[8] = {};
      if (a.res) load8<Y>(a.res, t * a.ld_res + c, n, r);
      if constexpr (K > 0) {
        add_rows<T, K, WEIGHTS>(a, 0, c, n, row, weight, acc);
      } else {
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
      }
      if (a.res) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += r[i];
      }
      if (c < col && a.res == a.dst) {  // in place: what the chunk before has belongs to it alone, which may have it no longer
#pragma unroll
        for (int i = 1; i < 8; ++i)
          if (i >= col - c) ((Y*)a.dst)[t * a.ld_dst + c + i] = (Y)acc[i];
      } else {
        store8<Y>(a.dst, t * a.ld_dst + c, n, acc);
      }
    }
  }
}

// The dispatch, token by token once inv is there: x is read once and written to its token's rows: 32768 tokens' ten rows of
// 2048 in 301 us with inv's two launches, 4.9 TB/s (row by row 437 us: every row read again from memory).
template <typename T, bool WIDE>
__global__ __launch_bounds__(256) void k_dispatch(RowsArgs a) {
  if ((int)blockIdx.x >= a.blocks) return zero_rows<T>(a);
  typedef typename Operand<T>::v8 v8;
  typedef v8 v8_any __attribute__((aligned(2)));
  const int span = 1 << a.shift, per = 256 >> a.shift;
  const int lane = threadIdx.x & (span - 1);
  int slot = threadIdx.x >> a.shift;
  if (WIDE) slot = __builtin_amdgcn_readfirstlane(slot);
  for (int64_t t = (int64_t)blockIdx.x * per + slot; t < a.T; t += (int64_t)a.blocks * per) {
    Choices<WIDE> ch;
    ch.init(a, t, false);
    const T* src = (const T*)a.src + t * a.ld_src;
    for (int col = lane * 8; col < a.H; col += span * 8) {
      const int c = chunk_at(col, a.H);
      if (a.H >= 8) {
        const v8 v = *(const v8_any*)(src + c);
        for (int j = 0; j < a.k; ++j) {
          const int32_t r = ch.row(j);
          if (r >= 0) *(v8_any*)((T*)a.dst + r * a.ld_dst + c) = v;
        }
      } else {
        for (int j = 0; j < a.k; ++j) {
          const int32_t r = ch.row(j);
          if (r >= 0)
            for (int i = 0; i < a.H; ++i) ((T*)a.dst)[r * a.ld_dst + i] = src[i];
        }
      }
    }
  }
}

// A token's dy is read once per four choices and serves their rows: dys[row] = w dy, dw = dy . ys[row].  32768 tokens' ten rows
// of 2048 577 us, 4.9 TB/s; 8191 tokens' four of 1357 57 us, 3.5.  A pair takes row
// inv[p] only where perm says the same, so every row of dys is written once: by its pair, or as a padding row by the
// workgroups behind the tokens'.
template <typename T, typename Y>
__global__ __launch_bounds__(256) void k_combine_grad(RowsArgs a) {
  __shared__ float sums[4][kMaxK];
  if ((int)blockIdx.x >= a.blocks) return zero_rows<T>(a);
  const int span = 1 << a.shift, per = 256 >> a.shift;
  const int lane = threadIdx.x & (span - 1), slot = threadIdx.x >> a.shift;
  for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.T; t0 += (int64_t)a.blocks * per) {
    const int64_t t = t0 + slot;
    const bool live = t < a.T;
    for (int j0 = 0; j0 < a.k; j0 += 4) {
      int32_t row[4], pair[4];
      float w[4], dot[4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool on = live && j0 + j < a.k;
        row[j] = on ? a.inv[t * a.k + j0 + j] : -1;
        w[j] = on && a.dst ? a.w[t * a.k + j0 + j] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (row[j] >= a.P) {
          if (lane == 0) set_error(a.ctrl, MOE_DERR_ROWS);
          row[j] = -1;
        }
        pair[j] = a.perm[row[j] < 0 ? 0 : row[j]];  // compared after the rows' loads have left
      }
      for (int col = lane * 8; live && col < a.H; col += span * 8) {
        const int c = chunk_at(col, a.H), n = chunk_len(a.H);
        float dy[8];
        typename Operand<T>::v8 v[4];
        load8<Y>(a.src, t * a.ld_src + c, n, dy);
        if (a.dw)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = load_raw<T>(a.ys, (int64_t)(row[j] < 0 ? 0 : row[j]) * a.ld_ys + c, n);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (row[j] >= 0 && pair[j] != t * a.k + j0 + j) {
            if (lane == 0) set_error(a.ctrl, MOE_DERR_ROWS);
            row[j] = -1;
          }
        if (a.dst)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row[j] >= 0) {
              float o[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = w[j] * dy[i];
              store8<T>(a.dst, (int64_t)row[j] * a.ld_dst + c, n, o);
            }
        if (a.dw)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float s = dot[j];
#pragma unroll
            for (int i = 0; i < 8; ++i) s = i < col - c ? s : fmaf(dy[i], (float)v[j][i], s);  // (zeros past a short row's end)
            dot[j] = row[j] < 0 ? 0.0f : s;
          }
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

// Threads per row: of the powers of two up to `most` that take a row of `chunks` 16-byte chunks in at most four passes, or the
// largest, the one that idles the fewest; the larger of two that idle as many.  (8 threads for 168 chunks, which idle none,
// took 72 us where 64 take 51: 8191 tokens' four rows.)
static int span_shift(int chunks, int most) {
  int best = 3;
  int64_t waste = INT64_MAX;
  for (int s = 3; (1 << s) <= most; ++s) {
    if (chunks > 4 << s && (2 << s) <= most) continue;
    const int64_t n = ((int64_t)chunks + (1 << s) - 1) / (1 << s) << s;
    if (n <= waste) {
      waste = n;
      best = s;
    }
  }
  return best;
}
static uint32_t grid_of(int64_t blocks) { return (uint32_t)(blocks < (1 << 20) ? blocks : 1 << 20); }

// Threads of a token: up to 256 while fewer than `wave` tokens leave room for them, else a wave at most.
static int token_span(int64_t T, int H, int64_t wave) { return span_shift((H + 7) / 8, T < wave ? 256 : 64); }
static uint32_t row_blocks(int64_t P) { return (uint32_t)((P + 255) / 256 < 1024 ? (P + 255) / 256 : 1024); }

template <typename T>
static hipError_t start_dispatch(RowsArgs a, hipStream_t st) {
  const int64_t pairs = (int64_t)a.T * a.k;
  if (pairs <= kInvPairs && a.P <= kInvPairs) {
    a.shift = span_shift((a.H + 7) / 8, 256);
    const int per = (256 >> a.shift) * 4;
    k_dispatch_few<T><<<(a.P + per - 1) / per + 1, 256, 0, st>>>(a);
    return hipGetLastError();
  }
  const int64_t clear = (pairs + 1023) / 1024, fill = ((int64_t)a.P + 255) / 256;
  k_inv_clear<<<(uint32_t)(clear < 4096 ? clear : 4096), 256, 0, st>>>(a.inv, pairs);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_inv_fill<<<grid_of(fill), 256, 0, st>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  a.shift = token_span(a.T, a.H, 16384);
  const int64_t per = 256 >> a.shift;
  a.blocks = (int32_t)grid_of((a.T + per - 1) / per);
  if (a.shift >= 6) k_dispatch<T, true><<<a.blocks + row_blocks(a.P), 256, 0, st>>>(a);
  else k_dispatch<T, false><<<a.blocks + row_blocks(a.P), 256, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, typename Y, bool WEIGHTS>
static hipError_t start_combine(RowsArgs a, hipStream_t st) {
  a.shift = token_span(a.T, a.H, 16384);
  const int64_t per = 256 >> a.shift;
  const uint32_t grid = grid_of((a.T + per - 1) / per);
#define MOE_COMBINE_CASE(K)                                          \
  case K:                                                            \
    k_combine<T, Y, WEIGHTS, K><<<grid, 256, 0, st>>>(a);            \
    break;
  switch (a.shift >= 6 ? a.k : 0) {
    MOE_COMBINE_CASE(1) MOE_COMBINE_CASE(2) MOE_COMBINE_CASE(3) MOE_COMBINE_CASE(4)
    MOE_COMBINE_CASE(5) MOE_COMBINE_CASE(6) MOE_COMBINE_CASE(7) MOE_COMBINE_CASE(8)
    MOE_COMBINE_CASE(9) MOE_COMBINE_CASE(10) MOE_COMBINE_CASE(11) MOE_COMBINE_CASE(12)
    MOE_COMBINE_CASE(13) MOE_COMBINE_CASE(14) MOE_COMBINE_CASE(15) MOE_COMBINE_CASE(16)
    default: k_combine<T, Y, WEIGHTS, 0><<<grid, 256, 0, st>>>(a);
  }
#undef MOE_COMBINE_CASE
  return hipGetLastError();
}

template <typename T, typename Y>
static hipError_t start_combine_grad(RowsArgs a, hipStream_t st) {
  a.shift = token_span(a.T, a.H, 2048);
  const int64_t per = 256 >> a.shift;
  a.blocks = (int32_t)grid_of((a.T + per - 1) / per);
  k_combine_grad<T, Y><<<a.blocks + row_blocks(a.P), 256, 0, st>>>(a);
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
