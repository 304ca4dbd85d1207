// The dense operators' types, activations, epilogue and launch arguments (moe_linear_*, moe_gated_*).
#pragma once

#include <float.h>
#include <math.h>

#include "kernels.hpp"

namespace moe {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));

// Operand types: 8-value vectors, the matrix step and 4-value vectors for the epilogue.
template <typename T>
struct Operand;
template <>
struct Operand<__bf16> {
  typedef bf16x8 v8;
  typedef bf16x4 v4;
  static MOE_DEV float4v mma(v8 a, v8 b, float4v c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
template <>
struct Operand<_Float16> {
  typedef half8 v8;
  typedef half4 v4;
  static MOE_DEV float4v mma(v8 a, v8 b, float4v c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};

// ---- activations ----------------------------------------------------------------------------------
// sigmoid by the hardware's exp2 and reciprocal (each within 1 ulp), its argument rounded once: relative error about
// (2 + |z|) 2^-24 (measured: up to 1.15 times that). That is 2^-17.3 at z = -87 and 2^-19.7 at -17, where fp16's
// numbers end: at least 2^7 below a 16-bit output's half step; of an fp32 output it is 2 + |z| half steps. Below
// z = -87 the reciprocal of 1 + exp(-z) is no normal number and the result is 0 (sigmoid is under 2^-125 there);
// exp2's underflow gives 1, as it should.
MOE_DEV float fast_sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

constexpr float kGeluC = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;

// Phi(z) and e = exp(-z^2 / 2). For z < 0 Phi(z) = e erfcx(x) / 2, x = |z| / sqrt 2, without the cancellation of
// (1 + erf) / 2 (5 % off at z = -5, 0 below -5.5); for z > 0 1 - Phi(-z). erfcx(x) / 2 = t P(t) with t = 1 / (1 + 0.45 x) and P
// of degree 9, fitted over all x >= 0 to a relative 3.2e-8. In fp32 the whole is within (1.5 z^2 + 10) 2^-24 of its value
// (z^2 / 2 rounded, then exp2; the hardware's exp2 and reciprocal 1 ulp each). No branches: gelu, 4096 x 4096 gated outputs
// of 2048 terms 127.6 us with erff, 134.3 with erfcf, 121.0 with this.
MOE_DEV float normal_cdf(float z, float& e) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.318198052f * fabsf(z));
  e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
  float q = -0.0206957665f;
  q = q * t + 0.0953447786f;
  q = q * t - 0.15029258f;
  q = q * t + 0.0712016206f;
  q = q * t - 0.011179518f;
  q = q * t + 0.0599753662f;
  q = q * t + 0.0876260416f;
  q = q * t + 0.114135822f;
  q = q * t + 0.126941581f;
  q = q * t + 0.12694266f;
  const float tail = e * t * q;
  return z < 0.0f ? tail : 1.0f - tail;
}

MOE_DEV float act_value(int act, float z) {
  switch (act) {
    case MOE_ACT_SILU: return z * fast_sigmoid(z);
    case MOE_ACT_GELU: {
      float e;
      return z * normal_cdf(z, e);
    }
    case MOE_ACT_GELU_TANH: return z * fast_sigmoid(2.0f * kGeluC * z * (1.0f + kGeluK * z * z));  // (1 + tanh v) / 2 = sigmoid(2 v)
    case MOE_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case MOE_ACT_SIGMOID: return fast_sigmoid(z);
    default: return z;
  }
}

// act_value of 8 values, the activation chosen once for all of them.
MOE_DEV void act_values(int act, float (&v)[8]) {
#define MOE_ACT_CASE(A)                                   \
  case A:                                                 \
    _Pragma("unroll") for (int c = 0; c < 8; ++c) v[c] = act_value(A, v[c]); \
    break;
  switch (act) {
    MOE_ACT_CASE(MOE_ACT_SILU)
    MOE_ACT_CASE(MOE_ACT_GELU)
    MOE_ACT_CASE(MOE_ACT_GELU_TANH)
    MOE_ACT_CASE(MOE_ACT_RELU)
    MOE_ACT_CASE(MOE_ACT_SIGMOID)
    default: break;
  }
#undef MOE_ACT_CASE
}

// s = sigmoid(z) and c = 1 - s without cancellation: e s, with e = exp(-z); 1 where e is too large for its
// reciprocal to be a normal number (s is 0 there, so a product with s is exactly the derivative's limit, however
// large z is).  NaN passes.
MOE_DEV void fast_sigmoid_pair(float z, float& s, float& c) {
  const float e = __builtin_amdgcn_exp2f(z * -1.44269504088896341f);
  const bool large = e > 1e37f;
  s = large ? 0.0f : __builtin_amdgcn_rcpf(1.0f + e);
  c = large ? 1.0f : e * s;
}

// Value and derivative together (the gated block's backward pass needs both).
MOE_DEV void act_both(int act, float z, float& v, float& d) {
  switch (act) {
    case MOE_ACT_SILU: {
      float s, c;
      fast_sigmoid_pair(z, s, c);
      v = z * s;
      d = s + z * (s * c);
      break;
    }
    case MOE_ACT_GELU: {
      float e;
      const float cdf = normal_cdf(z, e);
      v = z * cdf;
      d = cdf + z * 0.39894228040143268f * e;
      break;
    }
    case MOE_ACT_GELU_TANH: {
      float s, c;
      fast_sigmoid_pair(2.0f * kGeluC * z * (1.0f + kGeluK * z * z), s, c);
      v = z * s;
      const float q = z * (s * c);  // before the powers of z: 0 times them where they overflow fp32
      d = s + 2.0f * kGeluC * (q + 3.0f * kGeluK * (z * (z * q)));
      break;
    }
    case MOE_ACT_RELU:
      v = z > 0.0f ? z : (z != z ? z : 0.0f);
      d = z > 0.0f ? 1.0f : 0.0f;
      break;
    case MOE_ACT_SIGMOID: {
      float s, c;
      fast_sigmoid_pair(z, s, c);
      v = s;
      d = s * c;
      break;
    }
    default:
      v = z;
      d = 1.0f;
  }
}

// The same where z may be infinite (saved in 16 bits, past their range) and a tail's zero would meet it as NaN: taken as
// fp32's largest number it gives the limits, and the value stays infinite where the activation has no bound. NaN passes.
MOE_DEV void act_both_far(int act, float z, float& v, float& d) {
  act_both(act, z < -FLT_MAX ? -FLT_MAX : (z > FLT_MAX ? FLT_MAX : z), v, d);
  if (fabsf(v) == FLT_MAX) v = z;
}
// p times a saved factor f (u, or act(g)) that may be infinite in the same way: a p of zero gives zero, as it does for
// every value that f may have had. NaN passes.
MOE_DEV float times_far(float p, float f) { return p == 0.0f && f == f ? p : p * f; }

// exp(z - m) below a maximum m.  One that is infinite is not subtracted: its exponentials are then infinite, zero or NaN as
// the sum's limit is.
MOE_DEV float not_infinite(float m) { return __builtin_isinf(m) ? 0.0f : m; }
MOE_DEV float exp_below(float z, float m) { return __builtin_amdgcn_exp2f((z - m) * 1.44269504088896341f); }

// ---- epilogues ------------------------------------------------------------------------------------
enum DenseEpiKind { kEpiStore = 0, kEpiLinear = 1, kEpiGated = 2,
                    kEpiLoss = 3,    // logits: a row's maximum and sum of exponentials over the tile's columns
                    kEpiLossDz = 4,  // logits: their gradient, from the row's saved loss and lse
                    kEpiSum = 5 };   // sums onto earlier ones, scaled

// The loss's epilogues (moe_loss_*); the arrays are indexed by the product's rows.
struct LossEpi {
  const int32_t* targets;
  const float *loss, *lse, *dloss;  // kEpiLossDz (fp16's dloss: scaled already)
  float2* part;                     // kEpiLoss: [tiles_j][M], the target's column left out
  const float* scale;               // kEpiLossDz, bf16: dloss's factor; kEpiSum: the results' (NULL: 1, for sums that go on)
  const float* acc;                 // kEpiSum: the earlier sums, row stride DenseEpi::ldr (NULL: none)
  const float* row_scale;           // kEpiSum: a factor for each row in scale's place (NULL: none)
  int32_t* ctrl;
  int32_t col0, vocab, ignore;      // the product's first column, and all of them
};

struct DenseEpi {
  void* y[2];          // the output (kEpiStore: one per batch)
  int64_t ldy[2];
  const void* bias[2];  // linear: [0]; gated: gate, up
  const void* res;
  int64_t ldr;
  void* pre[2];        // saved z; g and u
  int64_t ldp[2];
  int32_t y_f32;       // linear: y and res are fp32
  int32_t act;
  int32_t stream;      // outputs larger than the L2s: stored with the non-temporal hint (launch_tile), so that
                       // they leave the operands in the caches (4096 tokens and outputs: 512 inputs 28.6 ->
                       // 24.9 us, 4096 inputs 110.8 -> 106.3 us)
  LossEpi loss;
};

// 8 consecutive elements of a row as fp32, or the first n of them. Global accesses of 16 bytes need only the
// element's alignment here, so rows of any address and stride move 8 elements at a time.
template <typename T>
MOE_DEV void load8(const void* base, int64_t off, int n, float (&v)[8]) {
  const T* p = (const T*)base + off;
  if (n == 8) {
    typedef T v8 __attribute__((ext_vector_type(8)));
    typedef v8 v8_any __attribute__((aligned(sizeof(T))));
    const v8 t = *(const v8_any*)p;
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = (float)t[c];
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = c < n ? (float)p[c] : 0.0f;
  }
}
template <typename T>
MOE_DEV void store8(void* base, int64_t off, int n, const float (&v)[8], bool stream = false) {
  T* p = (T*)base + off;
  if (n == 8) {
    typedef T v8 __attribute__((ext_vector_type(8)));
    typedef v8 v8_any __attribute__((aligned(sizeof(T))));
    v8 t;
#pragma unroll
    for (int c = 0; c < 8; ++c) t[c] = (T)v[c];
    if (stream) __builtin_nontemporal_store(t, (v8_any*)p);
    else *(v8_any*)p = t;
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < n) p[c] = (T)v[c];
  }
}

// Outputs (i, j .. j + n - 1), n = 1..8, j a multiple of 8: s0 = the fp32 sums (gated: the gate's), s1 = the up's.
template <typename T, int KIND>
MOE_DEV void finish8(const DenseEpi& e, int batch, int64_t i, int j, int n, float (&s0)[8], float (&s1)[8]) {
  const bool stream = e.stream;
  if constexpr (KIND == kEpiStore) {
    store8<T>(batch ? e.y[1] : e.y[0], i * (batch ? e.ldy[1] : e.ldy[0]) + j, n, s0, stream);
    return;
  }
  float t[8];
  if constexpr (KIND == kEpiSum) {
    if (e.loss.acc) {
      load8<float>(e.loss.acc, i * e.ldr + j, n, t);
#pragma unroll
      for (int c = 0; c < 8; ++c) s0[c] += t[c];
    }
    if (e.loss.scale) {
      const float f = e.loss.row_scale ? e.loss.row_scale[i] : *e.loss.scale;
#pragma unroll
      for (int c = 0; c < 8; ++c) s0[c] *= f;
    }
    if (e.y_f32) store8<float>(e.y[0], i * e.ldy[0] + j, n, s0, false);
    else store8<T>(e.y[0], i * e.ldy[0] + j, n, s0, stream);
    return;
  }
  if (e.bias[0]) {
    load8<T>(e.bias[0], j, n, t);
#pragma unroll
    for (int c = 0; c < 8; ++c) s0[c] += t[c];
  }
  if constexpr (KIND == kEpiGated) {
    if (e.bias[1]) {
      load8<T>(e.bias[1], j, n, t);
#pragma unroll
      for (int c = 0; c < 8; ++c) s1[c] += t[c];
    }
  }
  if (e.pre[0]) {
    store8<T>(e.pre[0], i * e.ldp[0] + j, n, s0, stream);
    if constexpr (KIND == kEpiGated) store8<T>(e.pre[1], i * e.ldp[1] + j, n, s1, stream);
  }
  act_values(e.act, s0);
  if constexpr (KIND == kEpiGated) {
#pragma unroll
    for (int c = 0; c < 8; ++c) s0[c] *= s1[c];
    store8<T>(e.y[0], i * e.ldy[0] + j, n, s0, stream);
  } else {
    if (e.res) {
      if (e.y_f32)
        load8<float>(e.res, i * e.ldr + j, n, t);
      else
        load8<T>(e.res, i * e.ldr + j, n, t);
#pragma unroll
      for (int c = 0; c < 8; ++c) s0[c] += t[c];
    }
    if (e.y_f32)
      store8<float>(e.y[0], i * e.ldy[0] + j, n, s0, stream);
    else
      store8<T>(e.y[0], i * e.ldy[0] + j, n, s0, stream);
  }
}

// ---- tile products: out[i][j] = sum_r A(i, r) B(j, r) ------------------------------------------------
// An operand is stored with its reduction index contiguous (kRows: A[i][r]) or its output index
// contiguous (kCols: A[r][i]).
//   forward     A = x   kRows, B = W   kRows   (gated: B[0] = Wg, B[1] = Wu, both sums per output)
//   dx          A = dz  kRows, B = W   kCols   (gated: two segments, dg Wg then du Wu, in one sum)
//   dW          A = dz  kCols, B = x   kCols   (gated: two batches, dg and du)
enum OperandOrder { kRows = 0, kCols = 1 };
// Where workgroups share a tile's reduction they leave their fp32 sums in the workspace, and a second launch
// adds them in split order and applies the epilogue: [split][mat][i - head_rows][part_ld], mat = the batch
// (gated: gate, up).
constexpr size_t kDensePartBytes = 32u << 20;
constexpr int kMaxSplits = 8;

struct TileArgs {
  const void* a[2];
  const void* b[2];
  int64_t lda[2], ldb[2];
  int32_t M, N, R;         // outputs i, j; reduction per segment
  int32_t len_a, len_b;    // readable elements of A's and B's rows (kRows): R, or more where what follows is zeros
  int32_t nseg, nbatch;    // 1 or 2 each
  int32_t tiles_i, tiles_j;
  int32_t b_once;          // B's rows are read by one row of tiles only (the experts' products)
  int32_t splits;          // workgroups sharing a tile's reduction, in rows of tiles from `head` on
  int32_t head, head_rows; // rows of tiles before them, each tile by one workgroup; their outputs' rows
  float* part;
  size_t part_bytes;
  uint16_t *pack_a, *pack_b[2];  // workspace for copies of the operands with whole 16-byte rows (NULL: none)
  DenseEpi epi;
};
// The tile kernel, its splits and head (TileArgs).  g_dense_plan is moe_debug_force_dense_plan's: MOE_DENSE_AUTO and
// 0 splits: chosen by size.
struct DensePlan {
  int kernel, splits, head;
};
extern DensePlan g_dense_plan;

inline size_t split_bytes(int splits, int mats, int64_t M, int64_t N) {
  return sizeof(float) * splits * mats * (size_t)(M * ((N + 7) / 8 * 8));
}
MOE_DEV float* part_at(const TileArgs& a, int split, int mats, int mat, int64_t i, int j) {
  const int64_t ld = (a.N + 7) / 8 * 8;
  return a.part + (((int64_t)split * mats + mat) * (a.M - a.head_rows) + i - a.head_rows) * ld + j;
}

// finish8, or for a split reduction the sums parked for the second launch.
template <typename T, int KIND>
MOE_DEV void finish_or_park(const TileArgs& a, int split, int batch, int64_t i, int j, int n, float (&s0)[8], float (&s1)[8]) {
  if (a.splits == 1) {
    finish8<T, KIND>(a.epi, batch, i, j, n, s0, s1);
  } else if constexpr (KIND == kEpiGated) {
    store8<float>(part_at(a, split, 2, 0, i, j), 0, 8, s0);
    store8<float>(part_at(a, split, 2, 1, i, j), 0, 8, s1);
  } else {
    store8<float>(part_at(a, split, a.nbatch, batch, i, j), 0, 8, s0);
  }
}

// dz of a backward pass: dz0 = dy * act'(pre0) (dy itself without an activation), or gated dz0 = dh * u * act'(g),
// dz1 = dh * act(g) with pre0 = g, pre1 = u; rows of ldz elements, zero from N to ldz.  Column sums of the
// unrounded values over runs of `rows` rows go to `part` [run][mats][N] when wanted.
struct GradArgs {
  const void* dy;
  const void* pre0;
  const void* pre1;
  int64_t ld_dy, ldp0, ldp1, ldz;
  void* dz0;  // NULL: the sums only
  void* dz1;
  float* part;  // NULL: no sums
  int32_t T, N;
  int32_t act;
  int32_t rows;
};
// Runs of rows: about 1024 workgroups (with 512 columns each), at least 4 rows (one per wave).
inline int64_t grad_runs_most(int64_t N) { return (1024 + (N + 511) / 512 - 1) / ((N + 511) / 512); }
inline int grad_rows(int64_t T, int64_t N) {
  const int64_t rows = (T + grad_runs_most(N) - 1) / grad_runs_most(N);
  return (int)((rows + 3) / 4 * 4);
}

// The bias gradients from such sums: db[m][n] = sum over runs of part[run][m][n], in run order.
struct BiasSumArgs {
  const float* part;
  void* db[2];  // NULL: not wanted
  int32_t runs, mats, N;
};
// 32 columns per workgroup of 256, 8 threads per column take contiguous shares of the runs, added in LDS in
// order. (One thread per column took 31 us for 128 runs of 2048 columns: a chain of loads on 8 CUs; this 4 us.)
template <typename T>
MOE_DEV void bias_sum_block(const BiasSumArgs& a, uint32_t block, float* sums) {
  const int64_t width = (int64_t)a.mats * a.N;
  const int64_t c = (int64_t)block * 32 + (threadIdx.x & 31);
  const int g = threadIdx.x >> 5;
  float s = 0.0f;
  if (c < width) {
    const int end = (int)((int64_t)a.runs * (g + 1) / 8);
#pragma unroll 8
    for (int r = (int)((int64_t)a.runs * g / 8); r < end; ++r) s += a.part[r * width + c];
  }
  sums[g * 33 + (threadIdx.x & 31)] = s;
  __syncthreads();
  if (g || c >= width) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += sums[i * 33 + threadIdx.x];
  T* db = (T*)(c < a.N ? a.db[0] : a.db[1]);
  if (db) db[c < a.N ? c : c - a.N] = (T)s;
}

// dense_tile_bf16.hip, dense_tile_f16.hip
hipError_t launch_forward_bf16(const TileArgs& a, int epi_kind, hipStream_t st);
hipError_t launch_forward_f16(const TileArgs& a, int epi_kind, hipStream_t st);
hipError_t launch_backward_bf16(const TileArgs& dx, const TileArgs& dw, const BiasSumArgs& db, hipStream_t st);
hipError_t launch_backward_f16(const TileArgs& dx, const TileArgs& dw, const BiasSumArgs& db, hipStream_t st);
// dense_rows.hip: up to MOE_DENSE_ROW_TOKENS tokens
hipError_t launch_rows(int dtype, const TileArgs& a, int epi_kind, hipStream_t st);
// dense_grad.hip. PackArgs: copies of up to three matrices with rows of whole 16-byte chunks, zeros past a
// row's end.
struct PackArgs {
  struct {
    const uint16_t* src;
    uint16_t* dst;
    int64_t ld, dst_ld, lines;
    int32_t len;
  } m[3];
  int32_t count;
};
hipError_t launch_pack(const PackArgs& p, hipStream_t st);
hipError_t launch_finish(int dtype, const TileArgs& a, int epi_kind, hipStream_t st);
hipError_t launch_grad_in(int dtype, const GradArgs& a, bool gated, hipStream_t st);
hipError_t launch_bias_sum(int dtype, const BiasSumArgs& a, hipStream_t st);

}  // namespace moe
