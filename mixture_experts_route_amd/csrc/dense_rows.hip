// The dense operators' forward pass for up to MOE_DENSE_ROW_TOKENS tokens: the weights streamed once, every
// token at a time on the matrix cores.
#include "dense.hpp"

namespace moe {

// Bound by the weights' bytes. One v_mfma_f32_16x16x32 takes 16 weight rows (one row per lane index l % 16, 16
// bytes of it per lane) and all tokens as its 16 columns; a column depends on its own token only, so absent
// tokens repeat the last one and are dropped, and a token's result is the same in any batch. A workgroup owns
// FRAGS x 16 weight rows: as many outputs (linear), or half as many outputs' rows of Wg and of Wu (FRAGS = 1: 8
// rows of each in one fragment). Its 8 waves take the blocks of 64 elements of its share of the reduction in
// turn, each from global memory straight into registers (four blocks in flight per wave), and their sums meet
// in LDS in wave order. Nothing in that order, nor in the choice of FRAGS and splits, depends on the tokens.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

constexpr int kRowWaves = 8, kRowAhead = 4;

template <typename T, int KIND, int FRAGS, bool WHOLE>
__global__ __launch_bounds__(64 * kRowWaves, 4) void k_rows(TileArgs a) {
  typedef typename Operand<T>::v8 v8;
  constexpr bool kGated = KIND == kEpiGated;
  constexpr int OUTS = kGated ? 8 * FRAGS : 16 * FRAGS;
  __shared__ float red[kRowWaves][FRAGS][16][20];  // [wave][fragment][token][row], rows padded against bank conflicts
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int split = blockIdx.x % a.splits;
  const int64_t j0 = (int64_t)(blockIdx.x / a.splits) * OUTS;
  const int row = lane & 15, k_lane = (lane >> 4) * 8;

  const uint16_t* w[FRAGS];
#pragma unroll
  for (int f = 0; f < FRAGS; ++f) {
    // the output this lane's weight row belongs to, and whether it is the up's
    const bool up = kGated && (FRAGS == 1 ? row >= 8 : f == 1);
    int64_t j = j0 + (kGated ? (FRAGS == 1 ? row & 7 : row) : f * 16 + row);
    if (j >= a.N) j = a.N - 1;
    w[f] = (up ? (const uint16_t*)a.b[1] + j * a.ldb[1] : (const uint16_t*)a.b[0] + j * a.ldb[0]) + k_lane;
  }
  const uint16_t* x = (const uint16_t*)a.a[0] + (int64_t)(row < a.M ? row : a.M - 1) * a.lda[0] + k_lane;

  auto load_w = [&](int f, int k) -> u32x4 {
    if constexpr (WHOLE) return __builtin_nontemporal_load((const u32x4*)(w[f] + k));
    return *(const u32x4_any*)(w[f] + k);
  };
  auto load_x = [&](int k) -> u32x4 {
    if constexpr (WHOLE) return *(const u32x4*)(x + k);
    return *(const u32x4_any*)(x + k);
  };

  float4v acc[FRAGS] = {};
  auto blocks = [&](int b, auto U) {  // blocks b, b + 8, .. of this wave: all loads, then the products
    constexpr int u = decltype(U)::value;
    u32x4 fw[u][2][FRAGS], fx[u][2];
#pragma unroll
    for (int i = 0; i < u; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (b + i * kRowWaves) * 64 + h * 32;
#pragma unroll
        for (int f = 0; f < FRAGS; ++f) fw[i][h][f] = load_w(f, k);
        fx[i][h] = load_x(k);
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < u; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < FRAGS; ++f)
          acc[f] = Operand<T>::mma(__builtin_bit_cast(v8, fw[i][h][f]), __builtin_bit_cast(v8, fx[i][h]), acc[f]);
  };
  const int whole_blocks = a.R / 64;
  const int full = (int)((int64_t)whole_blocks * (split + 1) / a.splits);  // end of this split's whole blocks
  int b = (int)((int64_t)whole_blocks * split / a.splits) + wave;
  for (; b + (kRowAhead - 1) * kRowWaves < full; b += kRowAhead * kRowWaves)
    blocks(b, std::integral_constant<int, kRowAhead>{});
  for (; b < full; b += kRowWaves) blocks(b, std::integral_constant<int, 1>{});
  if (b == full && split == a.splits - 1 && full * 64 < a.R) {  // the last, partial block: elements past the rows' end are zeros on both sides
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = full * 64 + h * 32, left = a.R - (k + k_lane);
      u32x4 fw[FRAGS] = {}, fx = {};
      if (left >= 8) {
#pragma unroll
        for (int f = 0; f < FRAGS; ++f) fw[f] = load_w(f, k);
        fx = load_x(k);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < left) {
#pragma unroll
            for (int f = 0; f < FRAGS; ++f) fw[f][i >> 1] |= (uint32_t)w[f][k + i] << (16 * (i & 1));
            fx[i >> 1] |= (uint32_t)x[k + i] << (16 * (i & 1));
          }
      }
#pragma unroll
      for (int f = 0; f < FRAGS; ++f)
        acc[f] = Operand<T>::mma(__builtin_bit_cast(v8, fw[f]), __builtin_bit_cast(v8, fx), acc[f]);
    }
  }
  // lane l holds rows 4 (l / 16) ..+3 of token l % 16
#pragma unroll
  for (int f = 0; f < FRAGS; ++f)
    *(float4v*)&red[wave][f][lane & 15][4 * (lane >> 4)] = acc[f];
  __syncthreads();
  for (int e = threadIdx.x; e < FRAGS * 256; e += 64 * kRowWaves) {  // one sum per thread and pass, in wave order
    float* p = &red[0][0][0][0] + (e >> 4) * 20 + (e & 15);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kRowWaves; ++i) sum += p[i * FRAGS * 320];
    *p = sum;
  }
  __syncthreads();
  // 8 outputs of a token per thread
  const int t = threadIdx.x / (OUTS / 8), c = threadIdx.x % (OUTS / 8) * 8;
  const int64_t left = a.N - (j0 + c);
  if (t >= a.M || t >= 16 || left <= 0) return;
  float s0[8], s1[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (!kGated) {
      s0[i] = red[0][c >> 4][t][(c & 15) + i];
    } else {
      s0[i] = red[0][0][t][c + i];
      s1[i] = FRAGS == 1 ? red[0][0][t][8 + i] : red[0][FRAGS - 1][t][c + i];
    }
  }
  finish_or_park<T, KIND>(a, split, 0, t, (int)(j0 + c), left < 8 ? (int)left : 8, s0, s1);
}

template <typename T, int KIND, int FRAGS, bool WHOLE>
static hipError_t start_rows(const TileArgs& a, hipStream_t st) {
  constexpr int OUTS = KIND == kEpiGated ? 8 * FRAGS : 16 * FRAGS;
  k_rows<T, KIND, FRAGS, WHOLE>
      <<<dim3((uint32_t)((a.N + OUTS - 1) / OUTS * a.splits)), dim3(64 * kRowWaves), 0, st>>>(a);
  return hipGetLastError();
}

// How many weight rows a workgroup takes and how many workgroups share them, by the outputs and inputs alone.
// The time is the most loaded CU's: whole workgroups per CU times their rows (and the activations beside them,
// as 6 rows' worth); what its waves have in flight at once costs one latency, about 2 us, the rest comes at
// about 17 KB per microsecond. A shared reduction adds a launch, 2.5 us, and the traffic of its sums (16
// tokens'). Measured, 16 tokens: 8192 inputs and outputs 40.0 us with one fragment, 34.7 with two; 8192 inputs,
// 2048 outputs 19.8 us alone, 14.6 shared by four; 4096 inputs, 1024 outputs 11.1 us, 8.0 by four. One token:
// 2048 inputs, 768 gated outputs 5.6 us, 6.4 by two; 6912 inputs, 2304 gated outputs (288 workgroups for 256
// CUs) 24.8 us, 19.2 by eight.
struct RowPlan {
  int frags, splits;
};
// The workspace must hold the sums of MOE_DENSE_ROW_TOKENS tokens whatever a call's own are, so that a token is
// summed in the same order in every batch; fewer tokens' sums, and their room, are that much smaller.
static bool parts_fit(int splits, int mats, int64_t N) {
  return splits == 1 || split_bytes(splits, mats, MOE_DENSE_ROW_TOKENS, N) <= kDensePartBytes;
}
static RowPlan plan_rows(int64_t groups, int64_t R, int mats, int64_t N) {
  RowPlan best = {1, 1};
  double least = 1e300;
  const int64_t sums = mats * N;
  for (int f = 1; f <= 2; ++f)
    for (int s = 1; s <= kMaxSplits && (s == 1 || (R / s >= 512 && parts_fit(s, mats, N))); ++s) {
      const int64_t per_cu = ((groups + f - 1) / f * s + 255) / 256;
      const double late = (double)per_cu / s * (16 * f + 6) * R * 2 - 88e3;
      const double us = 2.0 + (late > 0 ? late / 17e3 : 0.0) + (s > 1 ? 2.5 + 16.0 * sums * s * 8 / 4e6 : 0.0);
      if (us < least) {
        least = us;
        best = {f, s};
      }
    }
  return best;
}

template <typename T, int KIND>
static hipError_t launch_rows_k(const TileArgs& args, hipStream_t st) {
  TileArgs a = args;
  auto whole_rows = [](const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; };
  bool whole = a.R % 8 == 0 && whole_rows(a.a[0], a.lda[0]) && whole_rows(a.b[0], a.ldb[0]);
  if (KIND == kEpiGated) whole = whole && whole_rows(a.b[1], a.ldb[1]);
  constexpr int outs = KIND == kEpiGated ? 8 : 16, mats = KIND == kEpiGated ? 2 : 1;
  const RowPlan plan = plan_rows((a.N + outs - 1) / outs, a.R, mats, a.N);
  a.splits = g_dense_plan.splits ? g_dense_plan.splits : plan.splits;
  while (!parts_fit(a.splits, mats, a.N)) --a.splits;
  hipError_t e;
  if (plan.frags == 1) e = whole ? start_rows<T, KIND, 1, true>(a, st) : start_rows<T, KIND, 1, false>(a, st);
  else e = whole ? start_rows<T, KIND, 2, true>(a, st) : start_rows<T, KIND, 2, false>(a, st);
  return e != hipSuccess || a.splits == 1 ? e : launch_finish(__is_same(T, __bf16) ? MOE_BF16 : MOE_F16, a, KIND, st);
}

hipError_t launch_rows(int dtype, const TileArgs& a, int kind, hipStream_t st) {
  if (dtype == MOE_BF16)
    return kind == kEpiGated ? launch_rows_k<__bf16, kEpiGated>(a, st) : launch_rows_k<__bf16, kEpiLinear>(a, st);
  return kind == kEpiGated ? launch_rows_k<_Float16, kEpiGated>(a, st) : launch_rows_k<_Float16, kEpiLinear>(a, st);
}

}  // namespace moe
