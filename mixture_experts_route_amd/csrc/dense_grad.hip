// The elementwise part of the dense operators' backward passes: dz from dy and the saved pre-activations,
// and the bias gradients' sums.
#include "dense.hpp"

namespace moe {

// 8 consecutive elements from `e` of a row of N (zeros past N), any alignment.
template <typename T>
MOE_DEV void load8f(const void* base, int64_t off, int e, int N, float v[8]) {
  const T* p = (const T*)base + off + e;
  if (e + 8 <= N) {
    typedef T v8 __attribute__((ext_vector_type(8)));
    typedef v8 __attribute__((aligned(2))) v8_u;
    const v8 t = *(const v8_u*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)t[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = e + i < N ? (float)p[i] : 0.0f;
  }
}

// Memory-bound: reads dy and the saved values once, writes dz once (gated, 8192 x 8192: 671 MB in 117 us, 5.7
// TB/s). A workgroup takes 512 columns (8 per lane, 16 bytes a load) of a run of rows; its 4 waves take every
// fourth row and keep the column sums of their rows in registers, added over the waves in LDS in wave order. Infinite saved
// values show as NaN in dz, and only a chunk with one is computed again with their limits (checks of every element
// took the pass from 117 to 130 us). dz is rounded to the operands' type, as the matrix cores need it: dx and dW are
// 2.34e-3 off their definition against 1.66e-3 with an fp32 dz (bf16; fp16 2.9e-4 and 2.1e-4), at half the products of a dz in
// two 16-bit parts; the column sums take it unrounded.
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void k_grad_in(GradArgs a) {
  __shared__ float red[3][2][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.y * 512 + lane * 8;
  const int t0 = blockIdx.x * a.rows;
  const int t1 = a.T - t0 < a.rows ? a.T : t0 + a.rows;
  float sum0[8] = {}, sum1[8] = {};
  if (e < a.ldz) {
    for (int t = t0 + wave; t < t1; t += 4) {
      float dy[8], z0[8], z1[8];
      load8f<T>(a.dy, (int64_t)t * a.ld_dy, e, a.N, dy);
      if (GATED) {
        float g[8], u[8];
        load8f<T>(a.pre0, (int64_t)t * a.ldp0, e, a.N, g);
        load8f<T>(a.pre1, (int64_t)t * a.ldp1, e, a.N, u);
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v, d;
          act_both(a.act, g[i], v, d);
          z0[i] = dy[i] * d * u[i];
          z1[i] = dy[i] * v;
          nan |= __builtin_isunordered(z0[i], z1[i]);
        }
        if (nan) {  // from memory again, so that no register is held for this
          load8f<T>(a.dy, (int64_t)t * a.ld_dy, e, a.N, dy);
          load8f<T>(a.pre0, (int64_t)t * a.ldp0, e, a.N, g);
          load8f<T>(a.pre1, (int64_t)t * a.ldp1, e, a.N, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v, d;
            act_both_far(a.act, g[i], v, d);
            z0[i] = times_far(dy[i] * d, u[i]);
            z1[i] = times_far(dy[i], v);
          }
        }
      } else if (a.act != MOE_ACT_NONE) {
        float g[8];
        load8f<T>(a.pre0, (int64_t)t * a.ldp0, e, a.N, g);
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v, d;
          act_both(a.act, g[i], v, d);
          z0[i] = dy[i] * d;
          nan |= z0[i] != z0[i];
        }
        if (nan)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v, d;
            act_both_far(a.act, g[i], v, d);
            z0[i] = dy[i] * d;
          }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) z0[i] = dy[i];
      }
      typename Operand<T>::v8 o;
      if (a.dz0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (T)z0[i];
        *(typename Operand<T>::v8*)((T*)a.dz0 + (int64_t)t * a.ldz + e) = o;
        if (GATED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = (T)z1[i];
          *(typename Operand<T>::v8*)((T*)a.dz1 + (int64_t)t * a.ldz + e) = o;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum0[i] += z0[i];
        if (GATED) sum1[i] += z1[i];
      }
    }
  }
  if (!a.part) return;
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      red[wave - 1][0][lane * 8 + i] = sum0[i];
      if (GATED) red[wave - 1][1][lane * 8 + i] = sum1[i];
    }
  }
  __syncthreads();
  if (wave > 0) return;
  constexpr int mats = GATED ? 2 : 1;
  float* out = a.part + (int64_t)blockIdx.x * mats * a.N;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e + i >= a.N) break;
#pragma unroll
    for (int w = 0; w < 3; ++w) {
      sum0[i] += red[w][0][lane * 8 + i];
      if (GATED) sum1[i] += red[w][1][lane * 8 + i];
    }
    out[e + i] = sum0[i];
    if (GATED) out[a.N + e + i] = sum1[i];
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_bias_sum(BiasSumArgs a) {
  __shared__ float sums[8 * 33];
  bias_sum_block<T>(a, blockIdx.x, sums);
}

// Copies with whole 16-byte rows, memory-bound: a chunk of 8 elements per thread and pass; blockIdx.y is the
// matrix.
__global__ __launch_bounds__(256) void k_pack(PackArgs p) {
  const auto& m = p.m[blockIdx.y];
  const int64_t chunks = m.dst_ld / 8, total = m.lines * chunks;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
    const int64_t line = id / chunks, e = id % chunks * 8;
    const uint16_t* src = m.src + line * m.ld + e;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (e + 8 <= m.len) {
      typedef u32x4 __attribute__((aligned(2))) u32x4_any;
      v = *(const u32x4_any*)src;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < m.len) v[i >> 1] |= (uint32_t)src[i] << (16 * (i & 1));
    }
    *(u32x4*)(m.dst + line * m.dst_ld + e) = v;
  }
}

hipError_t launch_pack(const PackArgs& p, hipStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < p.count; ++i) most = p.m[i].lines * (p.m[i].dst_ld / 8) > most ? p.m[i].lines * (p.m[i].dst_ld / 8) : most;
  const int64_t blocks = (most + 255) / 256;
  k_pack<<<dim3((uint32_t)(blocks < 4096 ? blocks : 4096), p.count), 256, 0, st>>>(p);
  return hipGetLastError();
}

// Adds the sums of a split reduction in split order and applies the epilogue: 8 outputs per thread. Bound by
// two loads' latency at the sizes that are split (16 x 2048 outputs, 4 parts: 4.0 us), then by
// bytes (452 x 4096, 2 parts, gelu, saved and final results: 23 MB in 5.8 us).
template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_finish(TileArgs a) {
  const int chunks = (a.N + 7) / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  constexpr int kMats = KIND == kEpiGated ? 2 : 1;
  const int mats = KIND == kEpiGated ? 2 : a.nbatch;
  const int rows = a.M - a.head_rows;
  if (id >= (int64_t)chunks * rows * (mats / kMats)) return;
  const int j = (int)(id % chunks) * 8;
  const int64_t row = id / chunks;
  const int batch = row >= rows;
  const int64_t i = a.head_rows + row - (int64_t)batch * rows;
  // every load goes out before the first sum
  float t[kMaxSplits][kMats][8], s[2][8] = {};
#pragma unroll
  for (int p = 0; p < kMaxSplits; ++p)
#pragma unroll
    for (int m = 0; m < kMats; ++m)
      if (p < a.splits) load8<float>(part_at(a, p, mats, KIND == kEpiGated ? m : batch, i, j), 0, 8, t[p][m]);
#pragma unroll
  for (int p = 0; p < kMaxSplits; ++p)
    if (p < a.splits)
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int c = 0; c < 8; ++c) s[m][c] += t[p][m][c];
  finish8<T, KIND>(a.epi, batch, i, j, a.N - j < 8 ? a.N - j : 8, s[0], s[1]);
}

template <typename T>
static void start_finish(const TileArgs& a, int kind, hipStream_t st) {
  const int64_t threads = (int64_t)((a.N + 7) / 8) * (a.M - a.head_rows) * (kind == kEpiGated ? 1 : a.nbatch);
  const dim3 grid((uint32_t)((threads + 255) / 256)), block(256);
  if (kind == kEpiGated) k_finish<T, kEpiGated><<<grid, block, 0, st>>>(a);
  else if (kind == kEpiLinear) k_finish<T, kEpiLinear><<<grid, block, 0, st>>>(a);
  else if (kind == kEpiSum) k_finish<T, kEpiSum><<<grid, block, 0, st>>>(a);
  else k_finish<T, kEpiStore><<<grid, block, 0, st>>>(a);
}

hipError_t launch_finish(int dtype, const TileArgs& a, int kind, hipStream_t st) {
  if (dtype == MOE_BF16) start_finish<__bf16>(a, kind, st);
  else start_finish<_Float16>(a, kind, st);
  return hipGetLastError();
}

hipError_t launch_grad_in(int dtype, const GradArgs& a, bool gated, hipStream_t st) {
  const dim3 grid((uint32_t)((a.T + a.rows - 1) / a.rows), (uint32_t)((a.ldz + 511) / 512));
  if (dtype == MOE_BF16) {
    if (gated) k_grad_in<__bf16, true><<<grid, 256, 0, st>>>(a);
    else k_grad_in<__bf16, false><<<grid, 256, 0, st>>>(a);
  } else {
    if (gated) k_grad_in<_Float16, true><<<grid, 256, 0, st>>>(a);
    else k_grad_in<_Float16, false><<<grid, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_bias_sum(int dtype, const BiasSumArgs& a, hipStream_t st) {
  const uint32_t grid = (uint32_t)((a.mats * (int64_t)a.N + 31) / 32);
  if (dtype == MOE_BF16) k_bias_sum<__bf16><<<grid, 256, 0, st>>>(a);
  else k_bias_sum<_Float16><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
