// Tile products of the dense operators on the matrix cores: out[i][j] = sum_r A(i, r) B(j, r).
//
// A workgroup's output tile is cut into two halves along i and two along j (gated: the j halves are
// the gate's and the up's rows of the same outputs, so a lane ends up with both sums of an output).
// Along the reduction it advances 64 elements at a time: four LDS half tiles (A0 A1 B0 B1) of 64
// reduction elements each.
//
// LDS order of a half tile of H outputs:
//   kRows  [H][64]: an output's 64 elements are eight 16-byte chunks, chunk c of row i at c ^ (i & 7).
//          A lane's fragment (row l % 16, elements 8 (l / 16) ..+7) is one 16-byte read.
//   kCols  [64][H]: pairs of 16-byte chunks (16 outputs), pair p of reduction row r at p ^ mix(r).
//          A fragment is two transposing reads: 16 lanes read four rows of 16 outputs and lane l
//          receives output l % 16 of the four rows.
// Both swizzles keep a wave's reads on distinct LDS banks.  An MFMA takes B's fragment first, so lane l
// holds outputs i = l % 16, j = 4 (l / 16) ..+3: four consecutive elements of a row.
#pragma once

#include "dense.hpp"

namespace moe {

constexpr int kStepR = 64;  // reduction elements per step

// pair swizzle of a kCols half tile: rows r .. r+3 (one 16-lane read) and rows 8 apart on distinct banks
template <int H>
MOE_DEV int col_mix(int r) {
  if constexpr (H >= 128) return (r & 3) | (((r >> 3) & 1) << 2);
  if constexpr (H == 64) return ((r >> 1) & 1) | (((r >> 3) & 1) << 1);
  return (r >> 3) & 1;
}

// Element offset in a half tile of the 16-byte chunk `c` of line `m` (kRows: line = output, kCols: line = reduction row).
template <int ORDER, int H>
MOE_DEV int chunk_pos(int m, int c) {
  if constexpr (ORDER == kRows) return m * kStepR + ((c ^ (m & 7)) << 3);
  return m * H + (((c >> 1) ^ col_mix<H>(m)) << 4) + ((c & 1) << 3);
}

// Fragment of outputs o .. o+15 (o a multiple of 16), reduction elements 32 kk ..+31.
template <typename T, int ORDER, int H>
MOE_DEV typename Operand<T>::v8 read_frag(const uint16_t* half, int o, int kk, int lane) {
  typedef typename Operand<T>::v8 v8;
  if constexpr (ORDER == kRows) {
    return *(const v8*)(half + chunk_pos<kRows, H>(o + (lane & 15), kk * 4 + (lane >> 4)));
  } else {
    typedef short s4 __attribute__((ext_vector_type(4)));
    const int r = kk * 32 + 8 * (lane >> 4) + ((lane & 15) >> 2);
    const uint16_t* p = half + r * H + (((o >> 4) ^ col_mix<H>(r)) << 4) + ((lane & 3) << 2);
    typedef __attribute__((address_space(3))) s4 lds4;
    const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
    const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * H));  // col_mix(r + 4) = col_mix(r)
    struct {
      s4 a, b;
    } v = {lo, hi};
    return __builtin_bit_cast(v8, v);
  }
}

// Tile of this workgroup.  Consecutive workgroups go to the 8 XCDs in turn; each XCD takes a contiguous run of
// tiles, walked in groups of 8 tiles along i per column of tiles, so that its L2 keeps a group's A rows.
struct TileIndex {
  int batch, ti, tj, split;
};
MOE_DEV TileIndex tile_index(const TileArgs& a, int64_t id, int64_t count) {
  const int64_t q = count / 8, rem = count % 8;
  const int64_t xcd = id % 8, k = id / 8;
  int64_t t = xcd * q + (xcd < rem ? xcd : rem) + k;
  TileIndex x;
  x.split = (int)(t % a.splits);
  t /= a.splits;
  const int64_t per_batch = (int64_t)a.tiles_i * a.tiles_j;
  x.batch = (int)(t / per_batch);
  t -= x.batch * per_batch;
  const int64_t group = t / (8 * (int64_t)a.tiles_j);
  const int64_t in_group = t - group * 8 * a.tiles_j;
  const int rows = a.tiles_i - (int)group * 8 < 8 ? a.tiles_i - (int)group * 8 : 8;
  x.ti = (int)group * 8 + (int)(in_group % rows);
  x.tj = (int)(in_group / rows);
  return x;
}

// ---- any alignment --------------------------------------------------------------------------------
// 8 elements at (line, e .. e+7) of a row-major matrix of `lines` x `len`, zeros outside.
typedef u32x4 __attribute__((aligned(2))) u32x4_u;
MOE_DEV u32x4 load8_any(const uint16_t* base, int64_t ld, int64_t line, int64_t lines, int64_t e, int64_t len) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (line < lines) {
    const uint16_t* p = base + line * ld + e;
    if (e + 8 <= len) {
      v = *(const u32x4_u*)p;
    } else if (e < len) {
      const int n = (int)(len - e);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  return v;
}

// 128 x 128 tile, 4 waves of 64 x 64; operands pass through registers (a step ahead) on their way to LDS,
// so any address, stride and length works.
template <typename T, int OA, int OB, int KIND>
__global__ __launch_bounds__(256, 2) void k_tile_any(TileArgs a) {
  constexpr int H = 64;
  __shared__ __attribute__((aligned(1024))) uint16_t lds[4 * H * kStepR];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wi = wave >> 1, wj = wave & 1;
  const TileIndex x = tile_index(a, blockIdx.x, (int64_t)a.tiles_i * a.tiles_j * a.nbatch * a.splits);
  constexpr int JT = KIND == kEpiGated ? H : 2 * H;  // output columns per tile
  const int64_t i0 = (int64_t)x.ti * 2 * H, j0 = (int64_t)x.tj * JT;

  const int steps = (a.R + kStepR - 1) / kStepR;
  const int total = steps * a.nseg;

  u32x4 reg[8];
  auto fetch = [&](int s) {
    const int seg = s >= steps ? 1 : 0;
    const int64_t r0 = (int64_t)(s - seg * steps) * kStepR;
    const uint16_t* pa = (const uint16_t*)a.a[a.nbatch > 1 ? x.batch : seg];
    const int64_t lda = a.lda[a.nbatch > 1 ? x.batch : seg];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int q = tid + 256 * n, m = q >> 3, c = q & 7;
        if constexpr (OA == kRows)
          reg[2 * h + n] = load8_any(pa, lda, i0 + h * H + m, a.M, r0 + c * 8, a.R);
        else
          reg[2 * h + n] = load8_any(pa, lda, r0 + m, a.R, i0 + h * H + c * 8, a.M);
        const int sb = KIND == kEpiGated ? h : seg;
        const int64_t j = j0 + (KIND == kEpiGated ? 0 : h * H);
        const uint16_t* pb = (const uint16_t*)a.b[sb];
        if constexpr (OB == kRows)
          reg[4 + 2 * h + n] = load8_any(pb, a.ldb[sb], j + m, a.N, r0 + c * 8, a.R);
        else
          reg[4 + 2 * h + n] = load8_any(pb, a.ldb[sb], r0 + m, a.R, j + c * 8, a.N);
      }
  };

  float4v acc[2][2][2][2] = {};  // [i half][i fragment][j half][j fragment]
  fetch(0);
  for (int s = 0; s < total; ++s) {
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int q = tid + 256 * n, m = q >> 3, c = q & 7;
        *(u32x4*)(lds + h * H * kStepR + chunk_pos<OA, H>(m, c)) = reg[2 * h + n];
        *(u32x4*)(lds + (2 + h) * H * kStepR + chunk_pos<OB, H>(m, c)) = reg[4 + 2 * h + n];
      }
    __syncthreads();
    if (s + 1 < total) fetch(s + 1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      typename Operand<T>::v8 fb[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int g = 0; g < 2; ++g)
          fb[h][g] = read_frag<T, OB, H>(lds + (2 + h) * H * kStepR, wj * 32 + g * 16, kk, lane);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const auto fa = read_frag<T, OA, H>(lds + h * H * kStepR, wi * 32 + f * 16, kk, lane);
#pragma unroll
          for (int hj = 0; hj < 2; ++hj)
#pragma unroll
            for (int g = 0; g < 2; ++g) acc[h][f][hj][g] = Operand<T>::mma(fb[hj][g], fa, acc[h][f][hj][g]);
        }
    }
  }

#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int64_t i = i0 + h * H + wi * 32 + f * 16 + (lane & 15);
      if (i >= a.M) continue;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if constexpr (KIND == kEpiGated) {
          const int64_t j = j0 + wj * 32 + g * 16 + 4 * (lane >> 4);
          if (j < a.N) {
            float s0[4], s1[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) s0[c] = acc[h][f][0][g][c], s1[c] = acc[h][f][1][g][c];
            finish4<T, KIND>(a.epi, 0, i, (int)j, a.N - j < 4 ? (int)(a.N - j) : 4, s0, s1);
          }
        } else {
#pragma unroll
          for (int hj = 0; hj < 2; ++hj) {
            const int64_t j = j0 + hj * H + wj * 32 + g * 16 + 4 * (lane >> 4);
            if (j < a.N) {
              float s0[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) s0[c] = acc[h][f][hj][g][c];
              finish4<T, KIND>(a.epi, x.batch, i, (int)j, a.N - j < 4 ? (int)(a.N - j) : 4, s0, s0);
            }
          }
        }
      }
    }
}

template <typename T>
hipError_t launch_tile_t(const TileArgs& args, int oa, int ob, int kind, hipStream_t st) {
  TileArgs a = args;
  const int jt = kind == kEpiGated ? 64 : 128;
  a.tiles_i = (a.M + 127) / 128;
  a.tiles_j = (a.N + jt - 1) / jt;
  a.splits = 1;
  const int64_t count = (int64_t)a.tiles_i * a.tiles_j * a.nbatch;
  if (count > (int64_t)0xFFFFFFFF / 256) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)count), block(256);
  if (oa == kRows && ob == kRows && kind == kEpiLinear) k_tile_any<T, kRows, kRows, kEpiLinear><<<grid, block, 0, st>>>(a);
  else if (oa == kRows && ob == kRows && kind == kEpiGated) k_tile_any<T, kRows, kRows, kEpiGated><<<grid, block, 0, st>>>(a);
  else if (oa == kRows && ob == kCols && kind == kEpiStore) k_tile_any<T, kRows, kCols, kEpiStore><<<grid, block, 0, st>>>(a);
  else if (oa == kCols && ob == kCols && kind == kEpiStore) k_tile_any<T, kCols, kCols, kEpiStore><<<grid, block, 0, st>>>(a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_tile_bf16(const TileArgs& a, int oa, int ob, int kind, hipStream_t st);
hipError_t launch_tile_f16(const TileArgs& a, int oa, int ob, int kind, hipStream_t st);

}  // namespace moe
