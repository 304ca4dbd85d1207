// Softmax cross entropy over an output head (moe_loss_*): C interface, workspace and the kernels beside the products.
//
// Forward: one pass of tiles over the whole vocabulary; a tile's logits live in registers only and leave a maximum and a
// sum per row (8 bytes per row and tile of 64 to 256 columns), which a second launch joins.
// Backward, for one piece of the vocabulary after another: dz = dloss (exp(z - lse) - [target]) of the piece from its
// logits, computed again and rounded to the operands' type; then dW of the piece, whole, and the piece's share of dx, summed
// in fp32 over the pieces.  8192 tokens, 100003 x 2048, bf16: 8.3 to 8.5 ms, 1,190 to 1,210 TFLOP/s; a piece of 16384 columns
// takes 472 us for dz, 413 for dW and 430 for its share of dx.
#include "loss.hpp"

namespace moe {

constexpr int kLossTokens = 8192;          // tokens of a forward launch: bounds the parts
// dz of a piece, about.  8192 tokens, 100003 x 2048: 128 MiB 8.43 ms, 256 8.36, 512 8.38, 1024 8.46.  A limit on the piece's
// weights too, for few tokens, so that dx finds them in the last-level cache, costs more than it brings: 5 tokens, the same
// head, 325 us in one piece, 372 in pieces of 128 MiB of weights.
constexpr size_t kLossDzBytes = 256u << 20;
constexpr int kLossTile = 64;              // the smallest tile's columns
constexpr int kMostBlocks = 256;           // workgroups that look for fp16's largest |x|
constexpr int64_t kLiftFew = 1 << 15;      // elements of x up to which each does so for itself, and
constexpr int32_t kLiftFewTokens = 256;    // tokens: each of their workgroups goes through all of them

struct LossWs {
  size_t part, scale, scaled, undo, most, x, lifted, w, dz, acc, sums, sums_bytes, total;
  int64_t ld_in, piece, ldz;
};

// Columns of a piece: a multiple of 256, at least one, its dz within the limit where that allows it.
static int64_t piece_columns(int64_t T, int64_t V) {
  int64_t c = (int64_t)(kLossDzBytes / 2) / T / 1024 * 1024;
  if (c < 1024) c = (int64_t)(kLossDzBytes / 2) / T / 256 * 256;
  if (c < 256) c = 256;
  const int64_t all = (V + 7) / 8 * 8;
  return c < all ? c : all;
}

// Every part's room never falls as tokens are added, so that the workspace of one count serves those below it: dz has at most
// max(kLossDzBytes / 2, 256 T) elements however its piece is rounded, and a smaller count's larger piece (all of the vocabulary at
// most) bounds the split sums of dW.
static LossWs loss_ws(const moe_loss_dims* d, int64_t T, bool backward) {
  LossWs L{};
  const int64_t V = d->vocab, whole = (V + 7) / 8 * 8, chunk = T < kLossTokens ? T : kLossTokens;
  L.ld_in = ((int64_t)d->n_in + 7) / 8 * 8;
  size_t off = kCtrlBytes;
  L.scale = off;
  off = dense_align(off + 4 * sizeof(float));
  L.part = off;
  off = dense_align(off + sizeof(float2) * (size_t)(chunk * ((V + kLossTile - 1) / kLossTile)));
  // copies of operands without whole 16-byte rows: x always (its stride is the caller's; the forward pass takes a launch's tokens
  // at a time), the weights when n_in says so
  L.x = off;
  off = dense_align(off + 2 * (size_t)((backward ? T : chunk) * L.ld_in));
  if (d->n_in % 8) {
    L.w = off;
    off = dense_align(off + 2 * (size_t)(V * L.ld_in));
  }
  if (backward) {
    if (d->dtype == MOE_F16) {
      L.scaled = off;
      off = dense_align(off + sizeof(float) * (size_t)T);
      L.undo = off;
      off = dense_align(off + sizeof(float) * (size_t)T);
      L.most = off;
      off = dense_align(off + sizeof(float) * kMostBlocks);
      L.lifted = off;
      off = dense_align(off + 2 * (size_t)(T * L.ld_in));
    }
    L.piece = piece_columns(T, V);
    L.ldz = L.piece;
    const int64_t limit = (int64_t)(kLossDzBytes / 2) > 256 * T ? (int64_t)(kLossDzBytes / 2) : 256 * T;
    L.dz = off;
    off = dense_align(off + 2 * (size_t)(T * whole < limit ? T * whole : limit));
    L.acc = off;
    if (L.piece < V) off = dense_align(off + sizeof(float) * (size_t)(T * L.ld_in));
    L.sums = off;
    auto sums = [&](int64_t piece) {
      const size_t dx = split_bytes(kMaxSplits, 1, T, d->n_in), dw = split_bytes(kMaxSplits, 1, piece, d->n_in), most = dx > dw ? dx : dw;
      return most < kDensePartBytes ? most : kDensePartBytes;
    };
    L.sums_bytes = sums(L.piece);
    off = dense_align(off + sums(whole));
  }
  L.total = off;
  return L;
}

struct LossJoinArgs {
  const float2* part;
  const void *x, *w;
  const int32_t* targets;
  float *loss, *lse;
  int32_t* ctrl;
  int64_t ldx, ldw;
  int32_t T, tiles, vocab, ignore, K;
};

// A token's tiles joined: with m, s the maximum and sum of the other columns and zt the target's logit,
//   loss = log(1 + s exp(m - zt)) or, with zt below m, (m - zt) + log(s + exp(zt - m));  lse = zt + loss likewise.
// zt is summed here, in 64 bits (16-bit products are exact in 32): a sure token's loss is nothing but its distance from the
// others, and the target's logit, the largest in magnitude, would bring the most error into it.
// BLOCK tokens per workgroup share its 256 threads: neighbouring threads have neighbouring tokens while they read the
// tiles, and parts of the same token, in one wave (BLOCK 1: the workgroup), for the rest.  Every order is fixed.  Bound by the latency of a few dependent
// loads at small sizes, then by memory.
template <typename T, int BLOCK>
__global__ __launch_bounds__(256) void k_loss_join(LossJoinArgs a) {
  constexpr int kShares = 256 / BLOCK, kWaveShares = kShares < 64 ? kShares : 64;
  static_assert(BLOCK == 1 || kShares <= 64, "a token's threads are the workgroup or in one wave");
  __shared__ float ms[kShares][BLOCK + 1], ss[kShares][BLOCK + 1];
  __shared__ double zs[4];
  const int t = blockIdx.x * BLOCK + threadIdx.x / kShares, part = threadIdx.x % kShares;
  double zt = 0.0;
  const int target = t < a.T ? a.targets[t] : -1;
  const bool live = t < a.T && (uint32_t)target < (uint32_t)a.vocab && target != a.ignore;
  if (live) {
#pragma unroll 4
    for (int c = part * 8; c < a.K; c += kShares * 8) {
      const int n = a.K - c < 8 ? a.K - c : 8;
      float u[8], v[8];
      load8<T>(a.x, t * a.ldx + c, n, u);
      load8<T>(a.w, target * a.ldw + c, n, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) zt += (double)(u[i] * v[i]);
    }
  }
  {
    const int to = blockIdx.x * BLOCK + threadIdx.x % BLOCK, share = threadIdx.x / BLOCK;
    float m = -INFINITY, s = 0.0f;
    if (to < a.T) {
      for (int i = share; i < a.tiles; i += kShares * 8) {
        float2 p[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int at = i + u * kShares;
          p[u] = a.part[(int64_t)(at < a.tiles ? at : i) * a.T + to];
          if (at >= a.tiles) p[u] = make_float2(-INFINITY, 0.0f);
        }
        float most = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) most = fmaxf(most, p[u].x);
        const float base = not_infinite(most);
        s = m == most ? s : s * exp_below(m, base);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += p[u].x == most ? p[u].y : p[u].y * exp_below(p[u].x, base);
        m = most;
      }
    }
    ms[share][threadIdx.x % BLOCK] = m;
    ss[share][threadIdx.x % BLOCK] = s;
  }
  __syncthreads();
  float m = ms[part][threadIdx.x / kShares], s = ss[part][threadIdx.x / kShares];
#pragma unroll
  for (int o = 1; o < kWaveShares; o <<= 1) {
    const float mo = __shfl_xor(m, o, 64), so = __shfl_xor(s, o, 64), most = fmaxf(m, mo), base = not_infinite(most);
    const float mine = m == most ? s : s * exp_below(m, base), other = mo == most ? so : so * exp_below(mo, base);
    s = mine + other;
    m = most;
    zt += __shfl_xor(zt, o, 64);
  }
  if constexpr (BLOCK == 1) {  // the four waves'
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      ms[threadIdx.x >> 6][0] = m;
      ss[threadIdx.x >> 6][0] = s;
      zs[threadIdx.x >> 6] = zt;
    }
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < 4; ++w) {
      const float mo = ms[w][0], so = ss[w][0], most = fmaxf(m, mo), base = not_infinite(most);
      const float mine = m == most ? s : s * exp_below(m, base), other = mo == most ? so : so * exp_below(mo, base);
      s = mine + other;
      m = most;
      zt += zs[w];
    }
  }
  if (part || t >= a.T) return;
  float loss = 0.0f, lse = 0.0f;
  if (live) {
    const float z = (float)zt;
    if (z >= m) {
      loss = log1pf(s * expf((float)(m - zt)));
      lse = z + loss;
    } else {
      const float rest = logf(s + expf((float)(zt - m)));
      loss = (float)((m - zt) + rest);
      lse = m + rest;
    }
  } else if (target != a.ignore) {
    set_error(a.ctrl, MOE_DERR_TARGET);
    loss = lse = __builtin_nanf("");
  }
  a.loss[t] = loss;
  a.lse[t] = lse;
}

template <typename T>
static hipError_t start_join(const LossJoinArgs& j, hipStream_t st) {
  if (j.T >= 4096) k_loss_join<T, 16><<<(j.T + 15) / 16, 256, 0, st>>>(j);
  else if (j.T <= 256) k_loss_join<T, 1><<<j.T, 256, 0, st>>>(j);
  else k_loss_join<T, 4><<<(j.T + 3) / 4, 256, 0, st>>>(j);
  return hipGetLastError();
}

// dz is formed with dloss over the largest |dloss|, and the products are multiplied by that again, in fp32: with the same dloss
// for every token, a mean's 1 / count, an unsure token's dz at its target is then near -1, which no rounding moves, and not
// near -dloss, which one and the same rounding moves for all of them (bf16: dx and dW of a few tokens up to 2.6e-3 off their
// definition that way, 1.7e-3 to 2.0e-3 so; the plain form 1.7e-3).
// fp16 has not the range for one factor: a token whose dloss is 2^-20 of the largest would have no probabilities below 2^-16 left, most
// of its softmax (its dx had the wrong sign).  So each token has a power of two of its own besides, 2^lift, that brings its dz to
// 2^13 .. 2^15 at a probability of 1: normal down to probabilities of 2^-27, zero below 2^-38.  dx undoes it row by row; for
// dW, whose sum runs over the tokens, x carries 2^-lift in a copy, the call's largest |x| brought to 2^14 (exact down to 2^-28 of
// that).  Up to kLiftFew elements of x and kLiftFewTokens every workgroup finds the maxima by itself, in one launch, else two.
// Against one factor for all, fp16: 5 tokens, 100003 x 2048, 331 -> 333 us; 333 tokens, 32771 x 1000, 138 -> 145; 8192 tokens,
// 100003 x 2048, 8.69 -> 8.73 ms; 16 tokens, 300 x 2048 (in one launch) 25.9 -> 30.6, 64 tokens (in two) 26.0 -> 32.2.
struct LossScaleArgs {
  const float* dloss;
  const int32_t* targets;
  const void* x;
  float* scale;             // {factor of dloss, of the products, of fp16's dW, the largest |dloss|}
  float *scaled, *undo;     // fp16: each token's dloss with its factor; what dx undoes
  float* most;              // the largest |x| of each workgroup behind the first
  void* lifted;
  int64_t ldx, ld_lifted;
  float most_dz;
  int32_t T, K, vocab, ignore, blocks;  // blocks: that `most` has
  MOE_DEV bool live(int t) const { return (uint32_t)targets[t] < (uint32_t)vocab && targets[t] != ignore; }
};

// The largest m and x of 1024 threads, for all of them.
MOE_DEV void most_of_all(float& m, float& x) {
  __shared__ float2 most[16];
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    m = fmaxf(m, __shfl_xor(m, o, 64));
    x = fmaxf(x, __shfl_xor(x, o, 64));
  }
  if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = make_float2(m, x);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    m = fmaxf(m, most[i].x);
    x = fmaxf(x, most[i].y);
  }
}

// A thread's share of the largest |dloss|.
MOE_DEV float most_dloss(const LossScaleArgs& a) {
  float m = 0.0f;
#pragma unroll 4
  for (int t = threadIdx.x; t < a.T; t += 1024) {
    const float g = fabsf(a.dloss[t]);
    if (a.live(t) && g < INFINITY) m = fmaxf(m, g);
  }
  return m;
}
MOE_DEV float scale_base(float m) { return fminf(fmaxf(m, 0x1p-100f), 0x1p100f); }

// A thread's share of the largest finite |x|: chunks of 8 elements, from `first` on by `step`.
MOE_DEV float most_x(const LossScaleArgs& a, int64_t first, int64_t step) {
  const int64_t chunks = (a.K + 7) / 8, total = a.T * chunks;
  float m = 0.0f;
#pragma unroll 4
  for (int64_t id = first; id < total; id += step) {
    const int t = (int)(id / chunks), c = (int)(id - t * chunks) * 8;
    float v[8];
    load8<_Float16>(a.x, t * a.ldx + c, a.K - c < 8 ? a.K - c : 8, v);
    const bool live = a.live(t);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = live && fabsf(v[i]) < INFINITY ? fmaxf(m, fabsf(v[i])) : m;
  }
  return m;
}

MOE_DEV int lift_of(float m, float dloss) {
  const float g = fabsf(dloss);
  const int below = ilogbf(m) - (g > 0.0f && g < INFINITY ? ilogbf(g) : 1000);
  return below < 0 || below > 150 ? 0 : below;
}

// By the workgroup that writes them: the factors, and fp16's of every token.
MOE_DEV void store_scale(const LossScaleArgs& a, float m) {
  const float scale = a.most_dz / m, back = m / a.most_dz;
  if (threadIdx.x == 0) {
    a.scale[0] = scale;
    a.scale[1] = back;
    a.scale[3] = m;
  }
  if (!a.scaled) return;
#pragma unroll 4
  for (int t = threadIdx.x; t < a.T; t += 1024) {
    const float g = a.dloss[t];
    const int lift = lift_of(m, g);
    a.scaled[t] = __builtin_ldexpf(g * scale, lift);
    a.undo[t] = __builtin_ldexpf(back, -lift);
  }
}

__global__ __launch_bounds__(1024) void k_loss_scale(LossScaleArgs a) {
  float m = 0.0f, x = 0.0f;
  if (blockIdx.x == 0) m = most_dloss(a);
  else x = most_x(a, (int64_t)(blockIdx.x - 1) * 1024 + threadIdx.x, a.blocks * 1024);
  most_of_all(m, x);
  if (blockIdx.x == 0) store_scale(a, scale_base(m));
  else if (threadIdx.x == 0) a.most[blockIdx.x - 1] = x;
}

// lifted = x 2^(k - lift) in rows of whole chunks, zero for a token without a gradient; dW's factor is the products' times 2^-k.
template <bool FEW>
__global__ __launch_bounds__(1024) void k_loss_lift(LossScaleArgs a) {
  float m = 0.0f, x = 0.0f;
  if constexpr (FEW) {
    m = most_dloss(a);
    x = most_x(a, threadIdx.x, 1024);
    most_of_all(m, x);
    m = scale_base(m);
    if (blockIdx.x == 0) store_scale(a, m);
  } else {
    m = a.scale[3];
    for (int i = threadIdx.x & 63; i < a.blocks; i += 64) x = fmaxf(x, a.most[i]);
#pragma unroll
    for (int o = 32; o; o >>= 1) x = fmaxf(x, __shfl_xor(x, o, 64));
  }
  const int k = x > 0.0f ? 14 - ilogbf(x) : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.scale[2] = __builtin_ldexpf(m / a.most_dz, -k);
  const int64_t chunks = (a.K + 7) / 8, total = a.T * chunks;
  for (int64_t id = (int64_t)blockIdx.x * 1024 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 1024) {
    const int t = (int)(id / chunks), c = (int)(id - t * chunks) * 8;
    const bool live = a.live(t);
    const int by = k - lift_of(m, a.dloss[t]);
    float v[8];
    load8<_Float16>(a.x, t * a.ldx + c, a.K - c < 8 ? a.K - c : 8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = live ? __builtin_ldexpf(v[i], by) : 0.0f;
    store8<_Float16>(a.lifted, t * a.ld_lifted + c, 8, v);
  }
}

static int check_loss(const moe_loss_dims* d) {
  if (!d || d->n_in < 1 || d->vocab < 1) return MOE_EINVAL;
  if (d->n_in > MOE_DENSE_MAX_WIDTH || d->vocab > MOE_DENSE_MAX_WIDTH) return MOE_EUNSUPPORTED;
  return d->dtype == MOE_BF16 || d->dtype == MOE_F16 ? MOE_OK : MOE_EUNSUPPORTED;
}

static int check_loss_tokens(const moe_loss_dims* d, int32_t T) {
  const int rc = check_loss(d);
  if (rc) return rc;
  if (T < 1) return MOE_EINVAL;
  return T > MOE_LOSS_MAX_TOKENS ? MOE_EUNSUPPORTED : MOE_OK;
}

static int check_loss_ws(const moe_loss_dims* d, int32_t T, bool backward, const void* ws, size_t ws_bytes) {
  if (!ws || ((uintptr_t)ws & 255)) return MOE_EWORKSPACE;
  return ws_bytes < loss_ws(d, T, backward).total ? MOE_EWORKSPACE : MOE_OK;
}

static TileArgs logits_args(const moe_loss_dims* d, const int32_t* targets, void* ws) {
  TileArgs a{};
  a.nseg = a.nbatch = 1;
  a.R = a.len_a = a.len_b = d->n_in;
  a.epi.loss.targets = targets;
  a.epi.loss.ctrl = (int32_t*)ws;
  a.epi.loss.vocab = d->vocab;
  a.epi.loss.ignore = d->ignore;
  return a;
}

}  // namespace moe

using namespace moe;

extern "C" {

MOE_API size_t moe_loss_workspace_bytes(const moe_loss_dims* dims, int32_t max_tokens, int32_t backward) {
  return check_loss_tokens(dims, max_tokens) != MOE_OK ? 0 : loss_ws(dims, max_tokens, backward != 0).total;
}

MOE_API int moe_loss_forward(const moe_loss_dims* dims, const void* x, int64_t ldx, int32_t n_tokens, const void* w,
                             int64_t ldw, const int32_t* targets, float* loss, float* lse, void* ws, size_t ws_bytes,
                             void* stream) {
  int rc = check_loss_tokens(dims, n_tokens);
  if (rc) return rc;
  Mats m;
  m.need(x, ldx, dims->n_in);
  m.need(w, ldw, dims->n_in);
  m.need(targets, 1, 1, 4);
  m.need(loss, 1, 1, 4);
  m.need(lse, 1, 1, 4);
  if (m.rc) return m.rc;
  if ((rc = check_loss_ws(dims, n_tokens, false, ws, ws_bytes))) return rc;
  hipStream_t st = (hipStream_t)stream;
  const LossWs L = loss_ws(dims, n_tokens, false);
  auto at = [&](size_t off) { return (uint8_t*)ws + off; };
  for (int32_t t0 = 0; t0 < n_tokens; t0 += kLossTokens) {
    TileArgs a = logits_args(dims, targets + t0, ws);
    a.a[0] = (const uint16_t*)x + t0 * ldx;
    a.lda[0] = ldx;
    a.b[0] = w;
    a.ldb[0] = ldw;
    a.M = n_tokens - t0 < kLossTokens ? n_tokens - t0 : kLossTokens;
    a.N = dims->vocab;
    a.pack_a = (uint16_t*)at(L.x);
    a.pack_b[0] = L.w ? (uint16_t*)at(L.w) : nullptr;
    a.epi.loss.part = (float2*)at(L.part);
    LossJoinArgs j{};
    if ((rc = dense_status(dims->dtype == MOE_BF16 ? launch_loss_bf16(a, &j.tiles, st) : launch_loss_f16(a, &j.tiles, st)))) return rc;
    j.part = a.epi.loss.part;
    j.x = a.a[0];
    j.w = w;
    j.ldx = ldx;
    j.ldw = ldw;
    j.targets = targets + t0;
    j.loss = loss + t0;
    j.lse = lse + t0;
    j.ctrl = (int32_t*)ws;
    j.T = a.M;
    j.K = dims->n_in;
    j.vocab = dims->vocab;
    j.ignore = dims->ignore;
    if ((rc = dense_status(dims->dtype == MOE_BF16 ? start_join<__bf16>(j, st) : start_join<_Float16>(j, st)))) return rc;
  }
  return MOE_OK;
}

MOE_API int moe_loss_backward(const moe_loss_dims* dims, const void* x, int64_t ldx, int32_t n_tokens, const void* w,
                              int64_t ldw, const int32_t* targets, const float* loss, const float* lse,
                              const float* dloss, void* dx_or_null, int64_t ld_dx, void* dw_or_null, int64_t ld_dw,
                              void* ws, size_t ws_bytes, void* stream) {
  int rc = check_loss_tokens(dims, n_tokens);
  if (rc) return rc;
  if (!dx_or_null && !dw_or_null) return MOE_EINVAL;
  Mats m;
  m.need(x, ldx, dims->n_in);
  m.need(w, ldw, dims->n_in);
  m.need(targets, 1, 1, 4);
  m.need(loss, 1, 1, 4);
  m.need(lse, 1, 1, 4);
  m.need(dloss, 1, 1, 4);
  m.opt(dx_or_null, ld_dx, dims->n_in);
  m.opt(dw_or_null, ld_dw, dims->n_in);
  if (m.rc) return m.rc;
  if ((rc = check_loss_ws(dims, n_tokens, true, ws, ws_bytes))) return rc;
  hipStream_t st = (hipStream_t)stream;
  const bool bf16 = dims->dtype == MOE_BF16;
  const LossWs L = loss_ws(dims, n_tokens, true);
  auto at = [&](size_t off) { return (uint8_t*)ws + off; };
  float* scale = (float*)at(L.scale);
  const void *xs = x, *wt = w;
  int64_t ld_x = ldx, ld_w = ldw;
  int32_t len = dims->n_in;
  PackArgs p{};
  // Rows of whole 16-byte chunks for all three products, by one copy.  With an odd n_in that copies the weights too, which few
  // tokens do not pay for unless they are few as well: 2047 x 100003, 16 tokens 614 us, without 480; 128 tokens 704 and 641; 256
  // tokens 757 and 889; 1001 x 5000, 16 tokens 39 and 44.
  const bool pack = dims->n_in % 8 == 0 || n_tokens >= 192 || 2 * dims->vocab * L.ld_in <= 32 << 20;
  if (pack && ((uintptr_t)x % 16 || ldx % 8 || dims->n_in % 8)) {
    p.m[p.count++] = {(const uint16_t*)x, (uint16_t*)at(L.x), ldx, L.ld_in, n_tokens, dims->n_in};
    xs = at(L.x);
    ld_x = L.ld_in;
  }
  if (pack && L.w) {
    p.m[p.count++] = {(const uint16_t*)w, (uint16_t*)at(L.w), ldw, L.ld_in, dims->vocab, dims->n_in};
    wt = at(L.w);
    ld_w = len = L.ld_in;
  }
  if (p.count && (rc = dense_status(launch_pack(p, st)))) return rc;
  LossScaleArgs f{};
  f.dloss = dloss;
  f.targets = targets;
  f.x = xs;
  f.ldx = ld_x;
  f.scale = scale;
  if (!bf16) {
    f.scaled = (float*)at(L.scaled);
    f.undo = (float*)at(L.undo);
  }
  f.most_dz = bf16 ? 1.0f : 0x1p14f;
  f.T = n_tokens;
  f.K = dims->n_in;
  f.vocab = dims->vocab;
  f.ignore = dims->ignore;
  const void* x_dw = xs;  // dW's x and its stride
  int64_t ld_xdw = ld_x;
  const int64_t chunks = n_tokens * (L.ld_in / 8), copies = (chunks + 1023) / 1024;
  if (!bf16 && dw_or_null) {
    f.most = (float*)at(L.most);
    x_dw = f.lifted = at(L.lifted);
    ld_xdw = f.ld_lifted = L.ld_in;
    f.blocks = copies / 2 + 1 < kMostBlocks ? (int32_t)(copies / 2 + 1) : kMostBlocks;  // two chunks a thread at least
  }
  if (f.lifted && n_tokens <= kLiftFewTokens && (int64_t)n_tokens * dims->n_in <= kLiftFew) {
    k_loss_lift<true><<<(uint32_t)copies, 1024, 0, st>>>(f);
  } else {
    k_loss_scale<<<1 + f.blocks, 1024, 0, st>>>(f);
    if (f.lifted) k_loss_lift<false><<<(uint32_t)(copies < 1024 ? copies : 1024), 1024, 0, st>>>(f);
  }
  if (hipGetLastError() != hipSuccess) return MOE_EHIP;
  for (int32_t c0 = 0; c0 < dims->vocab; c0 += L.piece) {
    const int32_t cols = dims->vocab - c0 < L.piece ? dims->vocab - c0 : (int32_t)L.piece, whole = (cols + 7) / 8 * 8;
    const bool first = c0 == 0, last = c0 + cols == dims->vocab;
    const uint16_t* wp = (const uint16_t*)wt + c0 * ld_w;
    TileArgs z = logits_args(dims, targets, ws);
    z.a[0] = xs;
    z.lda[0] = ld_x;
    z.b[0] = wp;
    z.ldb[0] = ld_w;
    z.M = n_tokens;
    z.N = cols;
    z.R = z.len_a = z.len_b = len;
    z.epi.y[0] = at(L.dz);
    z.epi.ldy[0] = L.ldz;
    z.epi.loss.loss = loss;
    z.epi.loss.lse = lse;
    z.epi.loss.dloss = bf16 ? dloss : f.scaled;
    z.epi.loss.scale = scale;
    z.epi.loss.col0 = c0;
    if ((rc = dense_status(bf16 ? launch_loss_dz_bf16(z, st) : launch_loss_dz_f16(z, st)))) return rc;
    TileArgs s{};
    s.nseg = s.nbatch = 1;
    s.part = (float*)at(L.sums);
    s.part_bytes = L.sums_bytes;
    s.a[0] = at(L.dz);
    s.lda[0] = L.ldz;
    if (dw_or_null) {
      TileArgs a = s;
      a.b[0] = x_dw;
      a.ldb[0] = ld_xdw;
      a.M = cols;
      a.N = dims->n_in;
      a.R = n_tokens;
      a.epi.loss.scale = bf16 ? scale + 1 : scale + 2;
      a.epi.y[0] = (uint16_t*)dw_or_null + c0 * ld_dw;
      a.epi.ldy[0] = ld_dw;
      if ((rc = dense_status(bf16 ? launch_loss_dw_bf16(a, st) : launch_loss_dw_f16(a, st)))) return rc;
    }
    if (dx_or_null) {
      TileArgs a = s;
      a.b[0] = wp;
      a.ldb[0] = ld_w;
      a.M = n_tokens;
      a.N = dims->n_in;
      a.R = cols;
      a.len_a = whole;
      a.epi.loss.acc = first ? nullptr : (const float*)at(L.acc);
      a.epi.ldr = L.ld_in;
      a.epi.y_f32 = !last;
      a.epi.y[0] = last ? dx_or_null : at(L.acc);
      a.epi.ldy[0] = last ? ld_dx : L.ld_in;
      a.epi.loss.scale = last ? scale + 1 : nullptr;
      a.epi.loss.row_scale = f.undo;
      if ((rc = dense_status(bf16 ? launch_loss_dx_bf16(a, st) : launch_loss_dx_f16(a, st)))) return rc;
    }
  }
  return MOE_OK;
}

}  // extern "C"
