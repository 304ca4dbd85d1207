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

// Element offset in a half tile of the 16-byte chunk `c` of line `m` (kRows: line = output, kCols: line =
// reduction row).
template <int ORDER, int H>
MOE_DEV int chunk_pos(int m, int c) {
  if constexpr (ORDER == kRows) return m * kStepR + ((c ^ (m & 7)) << 3);
  return m * H + (((c >> 1) ^ col_mix<H>(m)) << 4) + ((c & 1) << 3);
}

// A lane's LDS byte address for the fragment of outputs o .. o+15 (o a multiple of 16), reduction elements
// 0..31, of the half tile at byte address `half`. Fragments of a wave start at o = FR * 16 * (wave's index), FR
// a power of two, so fragment n's pair index is o / 16 ^ n and every further address differs by a constant or
// one exclusive or.
template <int ORDER, int H>
MOE_DEV uint32_t frag_addr(uint32_t half, int o, int lane) {
  if constexpr (ORDER == kRows) return half + 2 * chunk_pos<kRows, H>(o + (lane & 15), lane >> 4);
  const int r = 8 * (lane >> 4) + ((lane & 15) >> 2);
  return half + 2 * (r * H + (((o >> 4) ^ col_mix<H>(r)) << 4) + ((lane & 3) << 2));
}
// Fragment n (16 n outputs on), reduction elements 32 kk ..+31, from such an address; `offset` bytes further on.
template <typename T, int ORDER, int H>
MOE_DEV typename Operand<T>::v8 read_frag(uint32_t addr, int n, int kk, int offset) {
  typedef typename Operand<T>::v8 v8;
  if constexpr (ORDER == kRows) {
    typedef __attribute__((address_space(3))) const v8 lds8;
    return *(lds8*)(uintptr_t)((addr ^ (kk * 64)) + (offset + n * 16 * kStepR * 2));
  } else {
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4 lds4;
    const uint32_t p = (addr ^ (n * 32)) + (offset + kk * 32 * H * 2);
    const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)p);
    const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)(p + 4 * H * 2));  // col_mix(r + 4) = col_mix(r)
    struct {
      s4 a, b;
    } v = {lo, hi};
    return __builtin_bit_cast(v8, v);
  }
}

// Tile of this workgroup.  Consecutive workgroups go to the 8 XCDs in turn; each XCD takes a contiguous run of
// tiles, walked in groups of 8 tiles along i per column of tiles, so that its L2 keeps a group's A rows.
struct TileIndex {
  int batch, ti, tj, split, splits;
};
// HEAD: the rows of tiles before a.head and those from there on are numbered each by themselves (else a.head = 0).
template <bool HEAD>
MOE_DEV TileIndex tile_index(const TileArgs& a, uint32_t id, uint32_t count) {
  const uint32_t n_head = HEAD ? (uint32_t)a.head * a.tiles_j : 0;
  const bool tail = !HEAD || id >= n_head;
  if (HEAD) {
    if (tail) id -= n_head;
    count = tail ? count - n_head : n_head;
  }
  const uint32_t q = count / 8, rem = count % 8, xcd = id % 8;
  uint32_t t = xcd * q + (xcd < rem ? xcd : rem) + id / 8;
  TileIndex x = {0, 0, 0, 0, tail ? a.splits : 1};
  if (x.splits > 1) {
    x.split = (int)(t % x.splits);
    t /= x.splits;
  }
  const uint32_t per_batch = (uint32_t)a.tiles_i * a.tiles_j;
  if (a.nbatch > 1 && t >= per_batch) {
    x.batch = 1;
    t -= per_batch;
  }
  const uint32_t in_full = 8u * a.tiles_j;
  const uint32_t group = t / in_full, in_group = t - group * in_full;
  const uint32_t left = (!HEAD ? a.tiles_i : tail ? a.tiles_i - a.head : a.head) - group * 8;
  const uint32_t rows = left < 8 ? left : 8;
  x.tj = (int)(rows == 8 ? in_group >> 3 : in_group / rows);
  x.ti = (int)(group * 8 + in_group - x.tj * rows) + (HEAD && tail ? a.head : 0);
  return x;
}

// ---- epilogue -------------------------------------------------------------------------------------
// A wave's FI x FJ fragments of outputs (i0.., j0..): lane l holds rows f 16 + l % 16, columns g 16 + 4 (l /
// 16) ..+3. They pass through the wave's own LDS (16-byte chunks swizzled by row) so that a lane stores 8
// consecutive elements. Plain results are rounded to 16 bits first, half the LDS bytes (4096 x 4096 outputs of
// 512 terms 27.2 -> 23.5 us, 8192 x 8192 of 2048 251 -> 244 us); with a bias, activation or residual the fp32
// sums pass, in a loop, so that the code of an activation exists once per kernel and no registers spill.
template <typename T, int KIND, int FI, int FJ>
MOE_DEV void finish_fragments(const TileArgs& a, const TileIndex& x, int64_t i0, int64_t j0, const float4v (&s0)[FI][FJ],
                              const float4v (&s1)[FI][FJ], float* lds, int lane) {
  constexpr int R = FI * 16, C = FJ * 16, kChunks = C / 4, kMask = (kChunks < 8 ? kChunks : 8) - 1;
  constexpr int kLanes = C / 8, kRowsPer = 64 / kLanes;  // lanes per row, rows per pass
  auto pos = [&](int r, int c) { return r * C + ((c ^ (r & kMask)) << 2); };
#pragma unroll
  for (int f = 0; f < FI; ++f)
#pragma unroll
    for (int g = 0; g < FJ; ++g) {
      const int r = f * 16 + (lane & 15), c = g * 4 + (lane >> 4);
      *(float4v*)(lds + pos(r, c)) = s0[f][g];
      if constexpr (KIND == kEpiGated) *(float4v*)(lds + R * C + pos(r, c)) = s1[f][g];
    }
  __builtin_amdgcn_wave_barrier();  // one wave: its LDS operations take effect in issue order
  const int j = (lane % kLanes) * 8;
  const int n = a.N - (j0 + j) < 8 ? (int)(a.N - (j0 + j)) : 8;
#pragma clang loop unroll(disable)
  for (int r = lane / kLanes; r < R; r += kRowsPer) {
    float v0[8], v1[8];
    *(float4v*)v0 = *(const float4v*)(lds + pos(r, j / 4));
    *(float4v*)(v0 + 4) = *(const float4v*)(lds + pos(r, j / 4 + 1));
    if constexpr (KIND == kEpiGated) {
      *(float4v*)v1 = *(const float4v*)(lds + R * C + pos(r, j / 4));
      *(float4v*)(v1 + 4) = *(const float4v*)(lds + R * C + pos(r, j / 4 + 1));
    }
    if (i0 + r < a.M && n > 0) finish8<T, KIND>(a.epi, x.batch, i0 + r, (int)(j0 + j), n, v0, v1);
  }
  __builtin_amdgcn_wave_barrier();
}

template <typename T, int FI, int FJ>
MOE_DEV void store_block(void* y, int64_t ldy, int64_t i0, int64_t j0, int M, int N, bool stream,
                         const float4v (&s)[FI][FJ], uint16_t* lds, int lane) {
  typedef typename Operand<T>::v8 v8;
  typedef T v4 __attribute__((ext_vector_type(4)));
  constexpr int R = FI * 16, C = FJ * 16, kLanes = C / 8, kRowsPer = 64 / kLanes;  // lanes per row, rows per pass
  auto pos = [](int r, int chunk) { return r * C + ((chunk ^ ((r >> (FJ == 1 ? 3 : 2)) & (kLanes - 1))) << 3); };
#pragma unroll
  for (int f = 0; f < FI; ++f)
#pragma unroll
    for (int g = 0; g < FJ; ++g) {
      v4 t;
#pragma unroll
      for (int c = 0; c < 4; ++c) t[c] = (T)s[f][g][c];
      const int chunk = g * 2 + (lane >> 5);
      *(v4*)(lds + pos(f * 16 + (lane & 15), chunk) + ((lane >> 4) & 1) * 4) = t;
    }
  __builtin_amdgcn_wave_barrier();  // one wave: its LDS operations take effect in issue order
  const int r0 = lane / kLanes, j = (lane % kLanes) * 8;
  const int64_t cols = N - (j0 + j);
  T* p = (T*)y + (i0 + r0) * ldy + j0 + j;
  const int64_t rows = M - i0;
  typedef v8 v8_any __attribute__((aligned(2)));
  if (N - j0 >= C) {
#pragma unroll
    for (int r = 0; r < R; r += kRowsPer) {
      const v8 t = *(const v8*)(lds + pos(r0 + r, lane % kLanes));
      if (r0 + r < rows && r0 + r < R) {
        if (stream) __builtin_nontemporal_store(t, (v8_any*)(p + r * ldy));
        else *(v8_any*)(p + r * ldy) = t;
      }
    }
  } else {
#pragma clang loop unroll(disable)
    for (int r = r0; r < R; r += kRowsPer) {
      const v8 t = *(const v8*)(lds + pos(r, lane % kLanes));
      if (r >= rows) continue;
      if (cols >= 8) {
        *(v8_any*)(p + (r - r0) * ldy) = t;
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < cols) p[(r - r0) * ldy + c] = t[c];
      }
    }
  }
  __builtin_amdgcn_wave_barrier();
}

// Parked sums leave from the registers, 16 bytes per lane and 64 per row and fragment; N a multiple of 4.
template <int FI, int FJ>
MOE_DEV void store_block_f32(float* y, int64_t ldy, int64_t i0, int64_t j0, int64_t M, int64_t N, const float4v (&s)[FI][FJ],
                             int lane) {
#pragma unroll
  for (int f = 0; f < FI; ++f) {
    const int64_t i = i0 + f * 16 + (lane & 15);
#pragma unroll
    for (int g = 0; g < FJ; ++g) {
      const int64_t j = j0 + g * 16 + 4 * (lane >> 4);
      if (i < M && j < N) *(float4v*)(y + i * ldy + j) = s[f][g];
    }
  }
}

// act(g) * u of one block, in registers.
template <int ACT, int FI, int FJ>
MOE_DEV void gate_block(const float4v (&g)[FI][FJ], const float4v (&u)[FI][FJ], float4v (&h)[FI][FJ]) {
#pragma unroll
  for (int f = 0; f < FI; ++f)
#pragma unroll
    for (int n = 0; n < FJ; ++n) {
#pragma unroll
      for (int c = 0; c < 4; ++c) h[f][n][c] = act_value(ACT, g[f][n][c]) * u[f][n][c];
      __builtin_amdgcn_sched_barrier(0);  // a fragment at a time: the registers are full of sums
    }
}

// All of a wave's sums: NI x 2 blocks, block (h, hj) at rows i0 + h di, columns j0 + hj dj (gated: hj = 0 the
// gate's, 1 the up's sums of the same outputs).
template <typename T, int KIND, int OA, int NI, int FI, int FJ>
MOE_DEV void finish_blocks(const TileArgs& a, const TileIndex& x, int64_t i0, int64_t di, int64_t j0, int64_t dj,
                           const float4v (&s)[NI][2][FI][FJ], float* lds, int lane) {
  const DenseEpi& e = a.epi;
  constexpr bool kGated = KIND == kEpiGated;
  constexpr bool kRowScale = __is_same(T, _Float16) && OA == kRows;  // kEpiSum: dx, whose rows are tokens
  if constexpr (kGated) {
    if (x.splits == 1 && !e.bias[0] && !e.bias[1] && !e.pre[0]) {
#pragma unroll
      for (int h = 0; h < NI; ++h) {
        float4v v[FI][FJ];
        switch (e.act) {
          case MOE_ACT_SILU: gate_block<MOE_ACT_SILU>(s[h][0], s[h][1], v); break;
          case MOE_ACT_GELU: gate_block<MOE_ACT_GELU>(s[h][0], s[h][1], v); break;
          case MOE_ACT_GELU_TANH: gate_block<MOE_ACT_GELU_TANH>(s[h][0], s[h][1], v); break;
          case MOE_ACT_RELU: gate_block<MOE_ACT_RELU>(s[h][0], s[h][1], v); break;
          case MOE_ACT_SIGMOID: gate_block<MOE_ACT_SIGMOID>(s[h][0], s[h][1], v); break;
          default: gate_block<MOE_ACT_NONE>(s[h][0], s[h][1], v);
        }
        store_block<T, FI, FJ>(e.y[0], e.ldy[0], i0 + h * di, j0, a.M, a.N, e.stream, v, (uint16_t*)lds, lane);
      }
      return;
    }
  }
  if constexpr (KIND == kEpiLossDz) {
    const LossEpi& l = e.loss;
    constexpr bool kScaled = __is_same(T, _Float16);
    const float scale = kScaled ? 1.0f : *l.scale;
    const bool inside = j0 + dj + FJ * 16 <= a.N;
#pragma unroll
    for (int h = 0; h < NI; ++h) {
      float4v v[2][FI][FJ];
#pragma unroll
      for (int f = 0; f < FI; ++f) {
        const int64_t i = i0 + h * di + f * 16 + (lane & 15);
        const int64_t row = i < a.M ? i : a.M - 1;
        const int target = l.targets[row];
        const bool live = (uint32_t)target < (uint32_t)l.vocab && target != l.ignore;
        if (!live && target != l.ignore && j0 == 0 && l.col0 == 0) set_error(l.ctrl, MOE_DERR_TARGET);
        const float lse = l.lse[row], g = kScaled ? l.dloss[row] : l.dloss[row] * scale;
        const int at = target - l.col0 - (int)j0;  // its column in this block
#pragma unroll
        for (int hj = 0; hj < 2; ++hj)
#pragma unroll
          for (int n = 0; n < FJ; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float p = g * exp_below(s[h][hj][f][n][c], lse);
              v[hj][f][n][c] = live ? p : 0.0f;
            }
        if (!inside || __any(live && at >= 0 && at < (int)dj + FJ * 16)) {  // the targets' columns, and those past N
          const float own = g * expm1f(-l.loss[row]);
#pragma unroll
          for (int hj = 0; hj < 2; ++hj)
#pragma unroll
            for (int n = 0; n < FJ; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int j = hj * (int)dj + n * 16 + 4 * (lane >> 4) + c;
                if (live && j == at) v[hj][f][n][c] = own;
                if (j0 + j >= a.N) v[hj][f][n][c] = 0.0f;
              }
        }
      }
#pragma unroll
      for (int hj = 0; hj < 2; ++hj)  // rows zero past N up to whole 16-byte chunks; they are read again soon: no hint
        store_block<T, FI, FJ>(e.y[0], e.ldy[0], i0 + h * di, j0 + hj * dj, a.M, (a.N + 7) / 8 * 8, false, v[hj], (uint16_t*)lds, lane);
    }
    return;
  }
  if constexpr (KIND == kEpiSum) {
    if (x.splits == 1 && !e.loss.acc && !e.y_f32) {  // scaled in the registers
      const float scale = kRowScale ? 1.0f : *e.loss.scale;
#pragma unroll
      for (int h = 0; h < NI; ++h)
#pragma unroll
        for (int hj = 0; hj < 2; ++hj) {
          float4v v[FI][FJ];
#pragma unroll
          for (int f = 0; f < FI; ++f) {
            float of_row = scale;
            if constexpr (kRowScale) {
              const int64_t i = i0 + h * di + f * 16 + (lane & 15);
              of_row = e.loss.row_scale[i < a.M ? i : a.M - 1];
            }
#pragma unroll
            for (int n = 0; n < FJ; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) v[f][n][c] = s[h][hj][f][n][c] * of_row;
          }
          store_block<T, FI, FJ>(e.y[0], e.ldy[0], i0 + h * di, j0 + hj * dj, a.M, a.N, e.stream, v, (uint16_t*)lds, lane);
        }
      return;
    }
  }
  const bool plain = KIND == kEpiStore || (KIND == kEpiLinear && !e.bias[0] && !e.pre[0] && !e.res && !e.y_f32 && e.act == MOE_ACT_NONE);
#pragma unroll
  for (int h = 0; h < NI; ++h)
#pragma unroll
    for (int hj = 0; hj < 2; ++hj) {
      const int64_t i = i0 + h * di, j = j0 + (kGated ? 0 : hj * dj);
      if (x.splits > 1) {  // parked for the second launch; rows padded to 8 floats, with room for spare columns
        const int mat = kGated ? hj : x.batch, mats = kGated ? 2 : a.nbatch, ld = (a.N + 7) / 8 * 8;
        store_block_f32<FI, FJ>(part_at(a, x.split, mats, mat, 0, 0), ld, i, j, a.M, ld, s[h][hj], lane);
      } else if (!kGated && plain) {
        store_block<T, FI, FJ>(x.batch ? e.y[1] : e.y[0], x.batch ? e.ldy[1] : e.ldy[0], i, j, a.M, a.N, e.stream, s[h][hj],
                               (uint16_t*)lds, lane);
      } else if (KIND != kEpiStore && !(kGated && hj)) {
        finish_fragments<T, KIND, FI, FJ>(a, x, i, j, s[h][hj], s[h][1], lds, lane);
      }
    }
}

// A tile of logits: for each row the maximum over the tile's columns and the sum of exp(z - maximum), the row's target left
// out, so that a small loss is log1p of what the others add and keeps its digits.  A lane has 4
// columns of every fragment of a row, four lanes a row's fragment, and the WJ waves beside each other meet in LDS.  8192 tokens,
// 100003 x 2048: 2.70 ms with the join, 1,240 TFLOP/s (the exponentials add about 6 us to a round of 256-square tiles' 57).
template <int TI, int WJ, int NI, int FI, int FJ>
MOE_DEV void finish_loss(const TileArgs& a, const TileIndex& x, int64_t i0, int64_t di, int64_t j0, int64_t dj, int wj,
                         const float4v (&s)[NI][2][FI][FJ], float* lds, int lane) {
  const LossEpi& l = a.epi.loss;
  const int64_t first = (int64_t)x.ti * TI;
  const bool inside = j0 + dj + FJ * 16 <= a.N;
#pragma unroll
  for (int h = 0; h < NI; ++h)
#pragma unroll
    for (int f = 0; f < FI; ++f) {
      const int64_t i = i0 + h * di + f * 16 + (lane & 15);
      const int at = (i < a.M ? l.targets[i] : -1) - (int)j0;
      float z[2][FJ][4], m = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int hj = 0; hj < 2; ++hj)
#pragma unroll
        for (int n = 0; n < FJ; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) z[hj][n][c] = s[h][hj][f][n][c];
      if (!inside || __any(at >= 0 && at < (int)dj + FJ * 16)) {  // left out: exp gives 0
#pragma unroll
        for (int hj = 0; hj < 2; ++hj)
#pragma unroll
          for (int n = 0; n < FJ; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int j = hj * (int)dj + n * 16 + 4 * (lane >> 4) + c;
              if (j == at || j0 + j >= a.N) z[hj][n][c] = -INFINITY;
            }
      }
#pragma unroll
      for (int hj = 0; hj < 2; ++hj)
#pragma unroll
        for (int n = 0; n < FJ; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) m = fmaxf(m, z[hj][n][c]);
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      const float base = not_infinite(m);
#pragma unroll
      for (int hj = 0; hj < 2; ++hj)
#pragma unroll
        for (int n = 0; n < FJ; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) sum += exp_below(z[hj][n][c], base);
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      if (lane < 16) {
        float* p = lds + ((i - first) * WJ + wj) * 2;
        p[0] = m;
        p[1] = sum;
      }
    }
  __syncthreads();
  for (int r = threadIdx.x; r < TI; r += blockDim.x) {
    if (first + r >= a.M) break;
    const float* p = lds + r * WJ * 2;
    float m = p[0];
#pragma unroll
    for (int w = 1; w < WJ; ++w) m = fmaxf(m, p[2 * w]);
    const float base = not_infinite(m);
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WJ; ++w) sum += p[2 * w] == m ? p[2 * w + 1] : p[2 * w + 1] * exp_below(p[2 * w], base);
    l.part[(int64_t)x.tj * a.M + first + r] = make_float2(m, sum);
  }
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

// One operand's 16-byte chunks of a step, COUNT per thread, loaded at any alignment. A step that is not the
// matrix's last is loaded without checks: lines past the outputs repeat the last one, chunks past them (kCols)
// the first, and a chunk that straddles the end of a kCols line runs into the next line, which exists; all of
// that reaches only sums that are not stored.
template <int ORDER, int H, int COUNT>
struct AnyLoad {
  const uint16_t* p[COUNT];
  int64_t advance;
  const uint16_t* base;
  int64_t ld, o0;
  int O, R;
  bool careful;

  MOE_DEV void init(const void* m, int64_t ld_, int64_t o0_, int O_, int R_, int step, int tid) {
    base = (const uint16_t*)m;
    ld = ld_;
    o0 = o0_;
    O = O_;
    R = R_;
    careful = ORDER == kCols && ld < 8;
    advance = ORDER == kRows ? kStepR : kStepR * ld;
#pragma unroll
    for (int n = 0; n < COUNT; ++n) {
      const int q = tid + 256 * n;
      if constexpr (ORDER == kRows) {
        const int64_t i = o0 + (q >> 3);
        p[n] = base + (i < O ? i : O - 1) * ld + (q & 7) * 8 + step * advance;
      } else {
        const int64_t c = o0 + q % (H / 8) * 8;
        p[n] = base + (c < O ? c : 0) + (q / (H / 8)) * ld + step * advance;
      }
    }
  }
  // step: of this matrix; last: its last one
  MOE_DEV void load(u32x4 (&reg)[COUNT], int step, bool last, int tid) {
    if (last || careful) {
#pragma unroll
      for (int n = 0; n < COUNT; ++n) {
        const int q = tid + 256 * n;
        if constexpr (ORDER == kRows)
          reg[n] = load8_any(base, ld, o0 + (q >> 3), O, (int64_t)step * kStepR + (q & 7) * 8, R);
        else
          reg[n] = load8_any(base, ld, (int64_t)step * kStepR + q / (H / 8), R, o0 + q % (H / 8) * 8, O);
      }
    } else {
#pragma unroll
      for (int n = 0; n < COUNT; ++n) reg[n] = *(const u32x4_u*)p[n];
    }
#pragma unroll
    for (int n = 0; n < COUNT; ++n) p[n] += advance;
  }
  MOE_DEV static void park(const u32x4 (&reg)[COUNT], uint16_t* half, int tid) {
#pragma unroll
    for (int n = 0; n < COUNT; ++n) {
      const int q = tid + 256 * n;
      if constexpr (ORDER == kRows) *(u32x4*)(half + chunk_pos<kRows, H>(q >> 3, q & 7)) = reg[n];
      else *(u32x4*)(half + chunk_pos<kCols, H>(q / (H / 8), q % (H / 8))) = reg[n];
    }
  }
};

// (64 F) x (64 F) tile, 4 waves of (32 F) x (32 F); operands pass through registers, two steps ahead, into two
// LDS buffers, so that any address, stride and length works. Bound by the latency and rate of unaligned loads:
// 0.9 us a step with 64-square tiles, 1.5 with 128 (4096 x 4095 outputs of 4095 terms 216 us; through copies
// with whole rows 142 us).
constexpr int any_lds(int f) { return 2 * 4 * 32 * f * kStepR; }  // elements
template <typename T, int OA, int OB, int KIND, int F>
MOE_DEV void any_tile(const TileArgs& a, const TileIndex& x, uint16_t* lds) {
  constexpr int H = 32 * F, kBuf = 4 * H * kStepR;  // elements: A0 A1 B0 B1
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wi = wave >> 1, wj = wave & 1;
  constexpr int JT = KIND == kEpiGated ? H : 2 * H;  // output columns per tile
  const int64_t i0 = (int64_t)x.ti * 2 * H, j0 = (int64_t)x.tj * JT;
  const int steps = (a.R + kStepR - 1) / kStepR;
  const int s_begin = (int)((int64_t)steps * a.nseg * x.split / x.splits);
  const int s_end = (int)((int64_t)steps * a.nseg * (x.split + 1) / x.splits);
  constexpr bool kSegs = OA == kRows && OB == kCols, kBatches = OA == kCols;

  AnyLoad<OA, H, F> la[2];
  AnyLoad<OB, H, F> lb[2];
  auto point = [&](int s) __attribute__((always_inline)) {  // at step s
    const bool seg = kSegs && s >= steps, second_a = kBatches ? x.batch : seg;
    const int step = seg ? s - steps : s;
    const void *a0 = a.a[0], *a1 = a.a[1], *b0 = a.b[0], *b1 = a.b[1];
    const int64_t ldb0 = a.ldb[0], ldb1 = a.ldb[1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool second_b = KIND == kEpiGated ? h == 1 : seg;
      la[h].init(second_a ? a1 : a0, a.lda[0], i0 + h * H, a.M, a.R, step, tid);
      lb[h].init(second_b ? b1 : b0, second_b ? ldb1 : ldb0, j0 + (KIND == kEpiGated ? 0 : h * H), a.N, a.R, step, tid);
    }
  };
  u32x4 ra[2][2][F], rb[2][2][F];  // [set][half][chunk]
  auto fetch = [&](auto S, int s) __attribute__((always_inline)) {
    constexpr int set = decltype(S)::value;
    if (s >= s_end) return;
    if (kSegs && s == steps && s != s_begin) point(s);
    const int step = kSegs && s >= steps ? s - steps : s;
    const bool last = step == steps - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      la[h].load(ra[set][h], step, last, tid);
      lb[h].load(rb[set][h], step, last, tid);
    }
  };
  auto park = [&](auto S, int buf) __attribute__((always_inline)) {
    constexpr int set = decltype(S)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      la[h].park(ra[set][h], lds + buf * kBuf + h * H * kStepR, tid);
      lb[h].park(rb[set][h], lds + buf * kBuf + (2 + h) * H * kStepR, tid);
    }
  };

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t*)lds;
  const uint32_t addr_a = frag_addr<OA, H>(lds0, wi * 16 * F, lane), addr_b = frag_addr<OB, H>(lds0, wj * 16 * F, lane);
  constexpr int kHalf = H * kStepR * 2;  // bytes
  float4v acc[2][2][F][F] = {};          // [i half][j half]
  auto multiply = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      typename Operand<T>::v8 fb[2][F];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int g = 0; g < F; ++g) fb[h][g] = read_frag<T, OB, H>(addr_b + buf * kBuf * 2, g, kk, (2 + h) * kHalf);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const auto fa = read_frag<T, OA, H>(addr_a + buf * kBuf * 2, f, kk, h * kHalf);
#pragma unroll
          for (int hj = 0; hj < 2; ++hj)
#pragma unroll
            for (int g = 0; g < F; ++g) acc[h][hj][f][g] = Operand<T>::mma(fb[hj][g], fa, acc[h][hj][f][g]);
        }
    }
  };
  auto step = [&](int s, auto S) __attribute__((always_inline)) {  // step s, parked in buffer S; the next one is in register set 1 - S
    constexpr int set = decltype(S)::value;
    __syncthreads();
    fetch(S, s + 2);
    multiply(set);
    if (s + 1 < s_end) park(std::integral_constant<int, 1 - set>{}, 1 - set);
  };
  constexpr std::integral_constant<int, 0> zero{};
  constexpr std::integral_constant<int, 1> one{};
  point(s_begin);
  fetch(zero, s_begin);
  fetch(one, s_begin + 1);
  park(zero, 0);
  int s = s_begin;
  for (; s + 1 < s_end; s += 2) {
    step(s, zero);
    step(s + 1, one);
  }
  if (s < s_end) step(s, zero);

  __syncthreads();
  if constexpr (KIND == kEpiLoss)
    finish_loss<2 * H, 2>(a, x, i0 + wi * 16 * F, H, j0 + wj * 16 * F, H, wj, acc, (float*)lds, lane);
  else
    finish_blocks<T, KIND, OA>(a, x, i0 + wi * 16 * F, H, j0 + wj * 16 * F, H, acc,
                           (float*)lds + wave * (KIND == kEpiGated ? 2 : 1) * F * F * 256, lane);
}

template <typename T, int OA, int OB, int KIND, int F>
__global__ __launch_bounds__(256, 2) void k_tile_any(TileArgs a) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[any_lds(F)];
  any_tile<T, OA, OB, KIND, F>(a, tile_index<false>(a, blockIdx.x, gridDim.x), lds);
}

// ---- 16-byte aligned operands ------------------------------------------------------------------------
// Asynchronous copy global -> LDS, 16 bytes per lane: lane l's bytes at buffer offset voff land at lds_addr + 16 l
// (lds_addr wave-uniform); a lane past the resource's bytes writes zeros.  Issued from an assembly block without
// outputs: the compiler otherwise assumes that any LDS read may depend on any such copy in flight and waits for
// all of them; here the waits are counted by hand (copies complete in issue order).
MOE_DEV void copy_to_lds(u32x4 rsrc, uint32_t lds_addr, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

// The same with the non-temporal hint, for operands that are read once.
MOE_DEV void copy_to_lds_once(u32x4 rsrc, uint32_t lds_addr, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
               :
               : "s"(lds_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

// Waits until at most N of this wave's copies are outstanding and its LDS reads have returned, then for the
// workgroup's other waves to have done the same.
template <int N>
MOE_DEV void copies_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// Copies of one operand: WAVES waves, half tiles of H outputs; each wave issues kCopies copies per half tile
// and step.
template <int ORDER, int H, int WAVES>
struct OperandCopy {
  static constexpr int kCopies = H / 8 / WAVES;  // H * 128 bytes in 1-KiB copies
  static constexpr int kLines = ORDER == kRows ? 8 : 512 / H;  // lines per copy
  static constexpr int kLineChunks = ORDER == kRows ? 8 : H / 8;
  static_assert(kCopies * 8 * WAVES == H, "a half tile is a whole number of copies per wave");
  // the swizzles of line and line + WAVES * kLines are the same: only the line's bits 0..3 enter them
  static_assert(kCopies == 1 || (WAVES * kLines) % 16 == 0, "");
  uint32_t voff[kCopies];  // byte offset of this lane's chunk from the half tile's first element
  int chunk;               // this lane's chunk of its line

  MOE_DEV void init(int64_t ld, int wave, int lane) {
    const int line = wave * kLines + lane / kLineChunks, pos = lane % kLineChunks;
    chunk = ORDER == kRows ? pos ^ (line & 7) : (((pos >> 1) ^ col_mix<H>(line)) << 1) | (pos & 1);
#pragma unroll
    for (int d = 0; d < kCopies; ++d)
      voff[d] = (uint32_t)((line + d * WAVES * kLines) * (uint32_t)ld * 2u + (uint32_t)chunk * 16u);
  }
};

// The steps of one half tile, in order: a running address and the steps left, so that issuing a step costs few
// scalar instructions (a wave issues one instruction per four to five cycles: at ~40 per copy the 64 x 64 tile
// took 0.35 us a step, whatever was in flight). SEGS: a second matrix follows the first; kCols operands have a stride
// for each (dx: Wg and Wu), kRows ones the same (dg and du). HINT: the copies are hinted as `once` says.
template <int ORDER, int H, int WAVES, bool SEGS, bool HINT = false>
struct HalfStream {
  typedef OperandCopy<ORDER, H, WAVES> Copy;
  uint64_t p, p1;       // first element of the next step; of the second matrix
  uint64_t stride;      // bytes from a step to the next
  int32_t bytes;        // of the resource in a whole step, 0 if the half tile has no outputs
  int32_t cut;          // reduction elements that the last, partial step of a matrix lacks
  int32_t left, left1;  // steps left in this matrix, the one to be issued included; in the second one
  int32_t ld1;          // kCols: the second matrix's stride in elements
  bool once;            // HINT: the operand is read by this workgroup only
  int32_t end, end1;    // left's value after a matrix's last step if that is partial and this workgroup's, else one it never takes

  // first: the half tile's first element; outs: its outputs that exist; R: reduction length (kRows: readable
  // elements of a line); the workgroup takes steps begin .. begin + count - 1 of the one or two matrices of
  // `steps` steps each.
  MOE_DEV void init(Copy& c, const void* m0, const void* m1, int64_t ld, int64_t ld_second, int64_t o0, int O, int R, int steps,
                    int begin, int count) {
    const int64_t first = 2 * (ORDER == kRows ? o0 * ld : o0);
    stride = ORDER == kRows ? 2 * kStepR : 2 * kStepR * (uint64_t)ld;
    const int n = O - o0 < H ? (int)(O - o0) : H;
    // (an odd row's last element shares its 4-byte word with what follows; a word is read whole or not at all)
    bytes = n <= 0 ? 0 : ORDER == kRows ? 2 * ((n - 1) * (int32_t)ld + kStepR) : 2 * ((kStepR - 1) * (int32_t)ld + n + (n & 1));
    const int tail = R - (steps - 1) * kStepR;
    cut = n <= 0 ? 0 : kStepR - tail;
    const int in0 = begin >= steps ? 0 : (begin + count < steps ? count : steps - begin);
    const int b1 = begin > steps ? begin - steps : 0;
    p = (uint64_t)m0 + first + begin * stride;
    left = in0;
    end = cut && begin + count >= steps ? 0 : -(1 << 30);
    if constexpr (SEGS) {
      ld1 = (int32_t)ld_second;
      p1 = (uint64_t)m1 + (ORDER == kRows ? first + b1 * stride : 2 * (o0 + b1 * kStepR * ld_second));
      left1 = count - in0;
      end1 = cut && begin + count >= 2 * steps ? 0 : -(1 << 30);
      if (left == 0) second(c);
    }
  }
  MOE_DEV void second(Copy& c) {
    p = p1;
    left = left1;
    end = end1;
    left1 = 0;
    if constexpr (ORDER == kCols) {
      if (bytes) bytes += 2 * (kStepR - 1) * (ld1 - (int32_t)(stride / (2 * kStepR)));
      stride = 2 * kStepR * (uint64_t)ld1;
      c.init(ld1, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), threadIdx.x & 63);
    }
  }
  // Issues this wave's copies of the next step. With no steps left the same number of copies is issued, all
  // past the resource's end: nothing is read, zeros are written.
  MOE_DEV void issue(Copy& c, uint32_t lds_addr) {
    u32x4 rsrc;
    rsrc[0] = (uint32_t)p;
    rsrc[1] = (uint32_t)(p >> 32);  // the address's bits 48.. are zero: no stride, no swizzle
    rsrc[2] = left > 0 ? bytes : 0;
    rsrc[3] = 0x00020000u;
    p += stride;
    --left;
    const bool tail = left == end;
    if (__builtin_expect(tail, 0)) {
      rsrc[2] = bytes - 2 * cut * (ORDER == kRows ? 1 : (int32_t)(stride / (2 * kStepR)));
      // a kRows line continues past the reduction's end (its next line, or what lies between): those chunks are
      // not read
      if (ORDER == kRows && c.chunk * 8 >= kStepR - cut)
#pragma unroll
        for (int d = 0; d < Copy::kCopies; ++d) c.voff[d] |= 0x80000000u;
    }
    if (HINT && once) {
#pragma unroll
      for (int d = 0; d < Copy::kCopies; ++d) copy_to_lds_once(rsrc, lds_addr + d * WAVES * 1024, c.voff[d]);
    } else {
#pragma unroll
      for (int d = 0; d < Copy::kCopies; ++d) copy_to_lds(rsrc, lds_addr + d * WAVES * 1024, c.voff[d]);
    }
    if (ORDER == kRows && __builtin_expect(tail, 0))
#pragma unroll
      for (int d = 0; d < Copy::kCopies; ++d) c.voff[d] &= 0x7FFFFFFFu;
    if constexpr (SEGS) {
      if (left == 0 && left1 > 0) second(c);
    }
  }
};

// 64 x 64 tile (gated: 64 x 32 outputs), 4 waves of 32 x 2 x 16, for products with too few large tiles to fill
// the chip: there a step's arithmetic is short and the time is the copies' latency, so five LDS buffers of one
// step (64 reduction elements, 16 KB) keep four steps in flight (two workgroups of them fill a CU's LDS; eight
// buffers were no faster): 0.36 us a step alone on a CU, 0.52 for two; 300 x 1000 outputs of 1000 terms 9.5 us,
// 128-square tiles 15 us. While a step's MFMAs run from registers the next step's fragments are read.
constexpr int kDeepStages = 5, kDeepStageBytes = (64 + 2 * 32) * kStepR * 2;
template <typename T, int OA, int OB, int KIND>
MOE_DEV void deep_tile(const TileArgs& a, const TileIndex& x, uint16_t* lds) {
  constexpr int STAGES = kDeepStages, W = 4, HI = 64, HJ = 32;
  constexpr int kBytes = kDeepStageBytes;  // A, B0, B1
  typedef typename Operand<T>::v8 v8;
  constexpr int kCopies = OperandCopy<OA, HI, W>::kCopies + 2 * OperandCopy<OB, HJ, W>::kCopies;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave >> 1, wj = wave & 1;
  constexpr int JT = KIND == kEpiGated ? HJ : 2 * HJ;
  const int64_t i0 = (int64_t)x.ti * HI, j0 = (int64_t)x.tj * JT;

  const int steps = (a.R + kStepR - 1) / kStepR, total = steps * a.nseg;
  const int s_begin = (int)((int64_t)total * x.split / x.splits);
  const int count = (int)((int64_t)total * (x.split + 1) / x.splits) - s_begin;

  constexpr bool kSegs = OA == kRows && OB == kCols, kBatches = OA == kCols;
  OperandCopy<OA, HI, W> ca;
  OperandCopy<OB, HJ, W> cb[2];
  HalfStream<OA, HI, W, kSegs> sa;
  HalfStream<OB, HJ, W, kSegs> sb[2];
  ca.init(a.lda[0], wave, lane);
  sa.init(ca, kBatches && x.batch ? a.a[1] : a.a[0], a.a[1], a.lda[0], 0, i0, a.M, OA == kRows ? a.len_a : a.R, steps, s_begin,
          count);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    constexpr bool g = KIND == kEpiGated;
    cb[h].init(a.ldb[g ? h : 0], wave, lane);
    sb[h].init(cb[h], a.b[g ? h : 0], a.b[1], a.ldb[g ? h : 0], a.ldb[1], j0 + (g ? 0 : h * HJ), a.N,
               OB == kRows ? a.len_b : a.R, steps, s_begin, count);
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t*)lds;
  auto copy = [&](uint32_t to) {  // the next step into the stage at `to`
    sa.issue(ca, to + wave * 1024);
    sb[0].issue(cb[0], to + HI * kStepR * 2 + wave * 1024);
    sb[1].issue(cb[1], to + (HI + HJ) * kStepR * 2 + wave * 1024);
  };

  const uint32_t addr_a = frag_addr<OA, HI>(0, wi * 32, lane);
  const uint32_t addr_b = frag_addr<OB, HJ>(HI * kStepR * 2, wj * 16, lane);
  v8 fa[2][2][2], fb[2][2][2];  // [set][fragment or j half][kk]
  float4v acc[2][2] = {};       // [j half][i fragment]
  auto read = [&](auto S, uint32_t stage) {
    constexpr int set = decltype(S)::value;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int n = 0; n < 2; ++n) fa[set][n][kk] = read_frag<T, OA, HI>(stage + addr_a, n, kk, 0);
#pragma unroll
      for (int h = 0; h < 2; ++h) fb[set][h][kk] = read_frag<T, OB, HJ>(stage + addr_b, 0, kk, h * HJ * kStepR * 2);
    }
  };
  uint32_t here = lds0;  // stage of step k
  auto next = [&](uint32_t st) { return st == lds0 + (STAGES - 1) * kBytes ? lds0 : st + kBytes; };
  auto step = [&](auto S) {
    constexpr int set = decltype(S)::value;
    copies_barrier<(STAGES - 2) * kCopies>();  // step k + 1 has landed, and every wave has read step k
    __builtin_amdgcn_sched_barrier(0);
    copy(here);
    here = next(here);
    read(std::integral_constant<int, 1 - set>{}, here);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 2; ++n) acc[h][n] = Operand<T>::mma(fb[set][h][kk], fa[set][n][kk], acc[h][n]);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int k = 0; k < STAGES; ++k) copy(lds0 + k * kBytes);
  copies_barrier<(STAGES - 1) * kCopies>();
  read(std::integral_constant<int, 0>{}, lds0);
  int k = 0;
  for (; k + 1 < count; k += 2) {
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
  }
  if (k < count) step(std::integral_constant<int, 0>{});
  copies_barrier<0>();  // no copy may land after the workgroup has given its LDS back

  float4v s[1][2][2][1];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < 2; ++n) s[0][h][n][0] = acc[h][n];
  if constexpr (KIND == kEpiLoss)
    finish_loss<HI, 2>(a, x, i0 + wi * 32, 0, j0 + wj * 16, HJ, wj, s, (float*)lds, lane);
  else
    finish_blocks<T, KIND, OA>(a, x, i0 + wi * 32, 0, j0 + wj * 16, HJ, s, (float*)lds + wave * 1024, lane);
}

template <typename T, int OA, int OB, int KIND>
__global__ __launch_bounds__(256, 2) void k_tile_deep(TileArgs a) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[kDeepStages * kDeepStageBytes / 2];
  deep_tile<T, OA, OB, KIND>(a, tile_index<false>(a, blockIdx.x, gridDim.x), lds);
}

// A small backward pass in one launch: dx's tiles, dW's tiles, then the bias gradients' columns. Alone each of
// the two products leaves CUs idle, and a launch costs two to three microseconds (333 tokens, 1000 x 1357: 27.8
// us as separate launches).
template <typename T>
__global__ __launch_bounds__(256, 2) void k_backward_small(TileArgs dx, TileArgs dw, BiasSumArgs db, uint32_t n_dx, uint32_t n_dw) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[kDeepStages * kDeepStageBytes / 2];
  uint32_t id = blockIdx.x;
  if (id < n_dx) {
    deep_tile<T, kRows, kCols, kEpiStore>(dx, tile_index<false>(dx, id, n_dx), lds);
    return;
  }
  id -= n_dx;
  if (id < n_dw) {
    deep_tile<T, kCols, kCols, kEpiStore>(dw, tile_index<false>(dw, id, n_dw), lds);
    return;
  }
  bias_sum_block<T>(db, id - n_dw, (float*)lds);
}

// (2 WI FI 16) x (2 WJ FJ 16) tile, WI x WJ waves; a wave's quarter in (i half, j half) is FI x FJ fragments.
//
// Two LDS buffers of one step (64 reduction elements) each. A step is four phases, one per quarter, in the
// order (A0,B0) (A0,B1) (A1,B1) (A1,B0); while a phase's MFMAs run from registers, the wave reads the fragments
// that the next phase adds and issues copies of a later step's half tile into the LDS region that was read out
// last:
//     phase        MFMA    reads to registers     copies
//     1 of step k  A0 B0   B1 of k                B0 of k+2
//     2            A0 B1   A1 of k                B1 of k+2
//     3            A1 B1   A0 of k+1              A1 of k+2
//     4            A1 B0   B0 of k+1 (over B1)    A0 of k+3
// A half tile is thus read six to seven phases after its copies were issued, with one barrier per phase that
// waits only for the copies older than the last six half tiles.
//
// Bound by the feed from the L2 (64 KB a step and CU in 256-square tiles; half the barriers or deeper reads
// ahead changed nothing): 1.47 us a step, matrix cores busy 60 % of the cycles, and about 10 us per round of
// tiles for the first copies and the stores. 8192^3 bf16: forward 808-910 us (1,210-1,360 TFLOP/s), dx 824, dW
// 810 us. 128-square tiles, two workgroups per CU, where 256-square ones would leave CUs idle: 4096 x 2048
// outputs of 8192 terms 134 against 181 us.
constexpr int big_lds(int wi, int wj, int fi, int fj) { return 2 * 2 * 16 * (wi * fi + wj * fj) * kStepR; }  // elements
template <typename T, int OA, int OB, int KIND, int WI, int WJ, int FI, int FJ, bool HINT = false>
MOE_DEV void big_tile(const TileArgs& a, const TileIndex& x, uint16_t* lds) {
  constexpr int W = WI * WJ, HI = WI * FI * 16, HJ = WJ * FJ * 16;
  constexpr int kBuf = 2 * (HI + HJ) * kStepR;  // elements of one buffer: A0 A1 B0 B1
  typedef typename Operand<T>::v8 v8;
  constexpr int DA = OperandCopy<OA, HI, W>::kCopies, DB = OperandCopy<OB, HJ, W>::kCopies;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / WJ, wj = wave % WJ;
  constexpr int JT = KIND == kEpiGated ? HJ : 2 * HJ;
  const int64_t i0 = (int64_t)x.ti * 2 * HI, j0 = (int64_t)x.tj * JT;

  const int steps = (a.R + kStepR - 1) / kStepR, total = steps * a.nseg;
  const int s_begin = (int)((int64_t)total * x.split / x.splits);
  const int count = (int)((int64_t)total * (x.split + 1) / x.splits) - s_begin;

  constexpr bool kSegs = OA == kRows && OB == kCols, kBatches = OA == kCols;  // which products have them
  OperandCopy<OA, HI, W> ca;
  OperandCopy<OB, HJ, W> cb[2];
  HalfStream<OA, HI, W, kSegs> sa[2];
  HalfStream<OB, HJ, W, kSegs, HINT> sb[2];
  ca.init(a.lda[0], wave, lane);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    constexpr bool g = KIND == kEpiGated;
    sa[h].init(ca, kBatches && x.batch ? a.a[1] : a.a[0], a.a[1], a.lda[0], 0, i0 + h * HI, a.M, OA == kRows ? a.len_a : a.R,
               steps, s_begin, count);
    if constexpr (HINT) sb[h].once = a.b_once;
    cb[h].init(a.ldb[g ? h : 0], wave, lane);
    sb[h].init(cb[h], a.b[g ? h : 0], a.b[1], a.ldb[g ? h : 0], a.ldb[1], j0 + (g ? 0 : h * HJ), a.N,
               OB == kRows ? a.len_b : a.R, steps, s_begin, count);
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t*)lds;
  const uint32_t mine = lds0 + wave * 1024;
  // half tile h of its stream's next step, into LDS buffer `buf`
  auto copy_a = [&](int h, int buf) { sa[h].issue(ca, mine + 2 * (buf * kBuf + h * HI * kStepR)); };
  auto copy_b = [&](int h, int buf) { sb[h].issue(cb[h], mine + 2 * (buf * kBuf + (2 * HI + h * HJ) * kStepR)); };

  v8 fa[2][FI][2], fb[2][FJ][2];
  float4v acc[2][2][FI][FJ] = {};  // [i half][j half]
  uint32_t addr_a = frag_addr<OA, HI>(lds0, wi * FI * 16, lane);
  uint32_t addr_b = frag_addr<OB, HJ>(lds0 + 2 * 2 * HI * kStepR, wj * FJ * 16, lane);
  auto read_a = [&](v8 (&f)[FI][2], int h, int buf) {
    asm volatile("" : "+v"(addr_a));  // the addresses derived from it are formed here, not kept in registers
    const uint32_t base = addr_a + buf * kBuf * 2;
#pragma unroll
    for (int n = 0; n < FI; ++n)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) f[n][kk] = read_frag<T, OA, HI>(base, n, kk, h * HI * kStepR * 2);
  };
  auto read_b = [&](v8 (&f)[FJ][2], int h, int buf) {
    asm volatile("" : "+v"(addr_b));
    const uint32_t base = addr_b + buf * kBuf * 2;
#pragma unroll
    for (int n = 0; n < FJ; ++n)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) f[n][kk] = read_frag<T, OB, HJ>(base, n, kk, h * HJ * kStepR * 2);
  };
  auto multiply = [&](int h, int hj, const v8 (&xa)[FI][2], const v8 (&xb)[FJ][2]) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int f = 0; f < FI; ++f)
#pragma unroll
        for (int g = 0; g < FJ; ++g) acc[h][hj][f][g] = Operand<T>::mma(xb[g][kk], xa[f][kk], acc[h][hj][f][g]);
    __builtin_amdgcn_s_setprio(0);
  };
  // one step; `p` is the register set that holds B0 (B1 goes to the other one), equal to the LDS buffer
  auto step = [&](auto P) {
    constexpr int p = decltype(P)::value, q = 1 - p;
    copies_barrier<4 * DA + 2 * DB>();
    __builtin_amdgcn_sched_barrier(0);
    copy_b(0, p);
    read_b(fb[q], 1, p);
    __builtin_amdgcn_sched_barrier(0);
    multiply(0, 0, fa[0], fb[p]);
    __builtin_amdgcn_sched_barrier(0);
    copies_barrier<3 * DA + 3 * DB>();
    __builtin_amdgcn_sched_barrier(0);
    copy_b(1, p);
    read_a(fa[1], 1, p);
    __builtin_amdgcn_sched_barrier(0);
    multiply(0, 1, fa[0], fb[q]);
    __builtin_amdgcn_sched_barrier(0);
    copies_barrier<2 * DA + 4 * DB>();
    __builtin_amdgcn_sched_barrier(0);
    copy_a(1, p);
    read_a(fa[0], 0, q);
    __builtin_amdgcn_sched_barrier(0);
    multiply(1, 1, fa[1], fb[q]);
    __builtin_amdgcn_sched_barrier(0);
    copies_barrier<3 * DA + 3 * DB>();
    __builtin_amdgcn_sched_barrier(0);
    copy_a(0, q);
    read_b(fb[q], 0, q);
    __builtin_amdgcn_sched_barrier(0);
    multiply(1, 0, fa[1], fb[p]);
    __builtin_amdgcn_sched_barrier(0);
  };

  copy_a(0, 0);
  copy_b(0, 0);
  copy_b(1, 0);
  copy_a(1, 0);
  copy_a(0, 1);
  copy_b(0, 1);
  copy_b(1, 1);
  copy_a(1, 1);
  copies_barrier<3 * DA + 3 * DB>();
  read_a(fa[0], 0, 0);
  read_b(fb[0], 0, 0);
  copies_barrier<3 * DA + 3 * DB>();
  copy_a(0, 0);
  int k = 0;
  for (; k + 1 < count; k += 2) {
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
  }
  if (k < count) step(std::integral_constant<int, 0>{});
  copies_barrier<0>();  // no copy may land after the workgroup has given its LDS back

  if constexpr (KIND == kEpiLoss)
    finish_loss<2 * HI, WJ>(a, x, i0 + wi * FI * 16, HI, j0 + wj * FJ * 16, HJ, wj, acc, (float*)lds, lane);
  else
    finish_blocks<T, KIND, OA>(a, x, i0 + wi * FI * 16, HI, j0 + wj * FJ * 16, HJ, acc,
                           (float*)lds + wave * (KIND == kEpiGated ? 2 : 1) * FI * FJ * 256, lane);
}

template <typename T, int OA, int OB, int KIND, int WI, int WJ, int FI, int FJ>
__global__ __launch_bounds__(64 * WI * WJ, 2) void k_tile(TileArgs a) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[big_lds(WI, WJ, FI, FJ)];
  big_tile<T, OA, OB, KIND, WI, WJ, FI, FJ>(a, tile_index<true>(a, blockIdx.x, gridDim.x), lds);
}

// A line's chunks lie on 16-byte addresses. kRows: and end with the reduction (or with zeros past it: len
// counts them). kCols: a last chunk that is partly past the outputs only reaches sums that are not stored.
inline bool whole_chunks(int order, const void* p, int64_t ld, int64_t len) {
  return (uintptr_t)p % 16 == 0 && ld % 8 == 0 && (order == kCols || len % 8 == 0);
}

// The plan with the least estimated time, in microseconds. Measured at bf16 and 64 reduction elements per step:
// a CU draws 45 to 50 KB per microsecond from the L2 whatever is in flight, so a step of a lone workgroup on
// its CU takes 0.36 us with a 64 x 64 tile (16 KB), 0.63 us with 128 x 128, 1.5 us with 256 x 256; two
// workgroups side by side (which the two smaller tiles allow) take 0.52 and 0.92 us for a step of each. Per
// round of tiles the prologue and epilogue add 1, 2 and 5 us; a split reduction adds a launch and the traffic
// of its fp32 sums. A last round that would leave most CUs idle is filled by splitting its tiles' reductions:
// 2500 x 4096 outputs of 4096 terms 98.5 -> 89.8 us (640 tiles, two of them at a time on a CU: 512 whole, 128 in
// two parts), gated 2060 x 4096 outputs of 8192 terms 273 -> 224 us (256-square, 256 whole, 32 in eight).
struct TileCost {
  int kernel, tile;
  double lone, pair, round;
};
constexpr TileCost kWholeCosts[] = {{MOE_DENSE_TILE64, 64, 0.36, 0.52, 1.0},
                                    {MOE_DENSE_TILE128, 128, 0.63, 0.92, 2.0},
                                    {MOE_DENSE_TILE256, 256, 1.55, 3.1, 5.0}};
constexpr TileCost kAnyCosts[] = {{MOE_DENSE_ANY64, 64, 0.9, 1.1, 1.0}, {MOE_DENSE_ANY128, 128, 1.5, 2.2, 2.0}};

template <int OA, int KIND>
DensePlan plan_tile(const TileArgs& a, bool whole, double* us) {
  const int64_t steps = (int64_t)((a.R + kStepR - 1) / kStepR) * a.nseg;
  const int mats = KIND == kEpiGated ? 2 : a.nbatch;
  DensePlan best = {0, 1, 0};
  double& least = *us = 1e300;
  const TileCost* costs = whole ? kWholeCosts : kAnyCosts;
  for (int c = 0; c < (whole ? 3 : 2); ++c) {
    const TileCost& k = costs[c];
    const int ti = k.tile, tj = KIND == kEpiGated ? ti / 2 : ti;
    const int64_t tiles = (((int64_t)a.M + ti - 1) / ti) * (((int64_t)a.N + tj - 1) / tj) * a.nbatch;
    for (int splits = 1; splits <= kMaxSplits; ++splits) {
      const size_t part = split_bytes(splits, mats, a.M, a.N);
      if (splits > 1 && (part > a.part_bytes || tiles * splits > 512 || steps / splits < 4)) break;
      const int64_t per_cu = (tiles * splits + 255) / 256;
      double t = 3.0 + (per_cu / 2 * k.pair + per_cu % 2 * k.lone) * ((steps + splits - 1) / splits) + (per_cu + 1) / 2 * k.round;
      if (splits > 1) t += 2.5 + 2.0 * part / 4e6;
      if (t < least) {
        least = t;
        best = {k.kernel, splits, 0};
      }
    }
    // whole rounds of tiles by single workgroups, the rest's reductions split (measured up to 5 us beyond its
    // parts)
    if (!whole || k.kernel == MOE_DENSE_TILE64 || a.nbatch > 1 || g_dense_plan.splits) continue;
    const int64_t row = ((int64_t)a.N + tj - 1) / tj, slots = k.pair < 2 * k.lone ? 512 : 256;
    const int64_t rounds = tiles / slots, head = rounds * slots / row, tail = tiles - head * row;
    if (!head || !tail) continue;
    for (int splits = 2; splits <= kMaxSplits; ++splits) {
      const size_t part = split_bytes(splits, mats, a.M - head * ti, a.N);
      if (part > a.part_bytes || tail * splits > slots || steps / splits < 4) break;
      const double step = slots == 512 ? k.pair : k.lone, tail_step = tail * splits > 256 ? k.pair : k.lone;
      const double t = 3.0 + rounds * (step * steps + k.round) + tail_step * ((steps + splits - 1) / splits) + k.round +
                       7.5 + 2.0 * part / 4e6;
      if (t < least) {
        least = t;
        best = {k.kernel, splits, (int)head};
      }
    }
  }
  return best;
}

// Tiles of TI x TJ outputs; false if the launch would exceed a grid's limit.
template <int TI, int TJ, int THREADS>
bool set_tiles(TileArgs& a, int64_t* count) {
  a.tiles_i = (a.M + TI - 1) / TI;
  a.tiles_j = (a.N + TJ - 1) / TJ;
  *count = ((int64_t)(a.tiles_i - a.head) * a.splits + a.head) * a.tiles_j * a.nbatch;
  return *count <= (int64_t)0xFFFFFFFF / THREADS;
}

template <typename T, int OA, int OB, int KIND, int WI, int WJ, int FI, int FJ>
hipError_t start_tile(TileArgs a, hipStream_t st) {
  int64_t count;
  if (!set_tiles<2 * WI * FI * 16, (KIND == kEpiGated ? 1 : 2) * WJ * FJ * 16, 64 * WI * WJ>(a, &count))
    return hipErrorInvalidConfiguration;
  k_tile<T, OA, OB, KIND, WI, WJ, FI, FJ><<<dim3((uint32_t)count), dim3(64 * WI * WJ), 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int OA, int OB, int KIND>
hipError_t start_plan(TileArgs a, int kernel, hipStream_t st) {
  int64_t count;
  switch (kernel) {
    case MOE_DENSE_TILE64:
      if (!set_tiles<64, KIND == kEpiGated ? 32 : 64, 256>(a, &count)) return hipErrorInvalidConfiguration;
      k_tile_deep<T, OA, OB, KIND><<<dim3((uint32_t)count), dim3(256), 0, st>>>(a);
      return hipGetLastError();
    case MOE_DENSE_TILE128: return start_tile<T, OA, OB, KIND, 2, 2, 2, 2>(a, st);
    case MOE_DENSE_TILE256: return start_tile<T, OA, OB, KIND, 2, 4, 4, 2>(a, st);
    case MOE_DENSE_ANY64:
      if (!set_tiles<64, KIND == kEpiGated ? 32 : 64, 256>(a, &count)) return hipErrorInvalidConfiguration;
      k_tile_any<T, OA, OB, KIND, 1><<<dim3((uint32_t)count), dim3(256), 0, st>>>(a);
      return hipGetLastError();
    default:
      if (!set_tiles<128, KIND == kEpiGated ? 64 : 128, 256>(a, &count)) return hipErrorInvalidConfiguration;
      k_tile_any<T, OA, OB, KIND, 2><<<dim3((uint32_t)count), dim3(256), 0, st>>>(a);
      return hipGetLastError();
  }
}

// Gives the operands that lack them whole 16-byte chunks, by copies in the workspace, when that pays: the copy
// costs a launch and the operand's bytes twice, the other kernels run at about half the rate (4096 x 4096
// tokens and outputs of 4095 inputs: 206 us without copies, 138 with; whole rows 106).
template <int OA, int OB, int KIND>
bool pack_operands(TileArgs& a, bool whole_a, const bool (&whole_b)[2], hipStream_t st, hipError_t* err) {
  const int na = a.nseg > 1 || a.nbatch > 1 ? 2 : 1, nb = KIND == kEpiGated || a.nseg > 1 ? 2 : 1;
  PackArgs p{};
  double bytes = 0;
  auto add = [&](const void*& src, int64_t& ld, uint16_t* to, int64_t lines, int len) {
    if (!to || p.count == 3) return false;
    const int64_t to_ld = ((int64_t)len + 7) / 8 * 8;
    p.m[p.count++] = {(const uint16_t*)src, to, ld, to_ld, lines, len};
    bytes += 4.0 * lines * to_ld;
    src = to;
    ld = to_ld;
    return true;
  };
  TileArgs b = a;
  if (!whole_a) {
    if (na > 1 || !add(b.a[0], b.lda[0], a.pack_a, OA == kRows ? a.M : a.R, OA == kRows ? a.R : a.M)) return false;
    b.len_a = (a.R + 7) / 8 * 8;
  }
  b.len_b = OB == kRows && !(whole_b[0] && whole_b[1]) ? (a.R + 7) / 8 * 8 : a.R;
  for (int m = 0; m < nb; ++m) {
    if (!whole_b[m] && !add(b.b[m], b.ldb[m], a.pack_b[m], OB == kRows ? a.N : a.R, OB == kRows ? a.R : a.N)) return false;
  }
  if (a.nbatch > 1) b.b[1] = b.b[0], b.ldb[1] = b.ldb[0];
  double direct, packed;
  plan_tile<OA, KIND>(a, false, &direct);
  plan_tile<OA, KIND>(b, true, &packed);
  if (packed + 2.5 + bytes / 4e6 >= direct) return false;
  a = b;
  *err = launch_pack(p, st);
  return true;
}

// The operands as the kernels will read them (copied where that pays), and the plan with its estimate.
template <int OA, int OB, int KIND>
hipError_t prepare_tile(TileArgs& a, DensePlan& plan, double& us, hipStream_t st) {
  bool whole_a = true, whole_b[2] = {true, true};
  for (int m = 0; m < (a.nseg > 1 || a.nbatch > 1 ? 2 : 1); ++m)
    whole_a = whole_a && whole_chunks(OA, a.a[m], a.lda[m], a.len_a);
  for (int m = 0; m < (KIND == kEpiGated || a.nseg > 1 ? 2 : 1); ++m)
    whole_b[m] = whole_chunks(OB, a.b[m], a.ldb[m], a.R);
  bool whole = whole_a && whole_b[0] && whole_b[1];
  if (!whole && g_dense_plan.kernel < MOE_DENSE_ANY64) {
    hipError_t err = hipSuccess;
    whole = pack_operands<OA, OB, KIND>(a, whole_a, whole_b, st, &err);
    if (err != hipSuccess) return err;
  }
  plan = plan_tile<OA, KIND>(a, whole, &us);
  if (g_dense_plan.kernel != MOE_DENSE_AUTO && (whole || g_dense_plan.kernel >= MOE_DENSE_ANY64))
    plan = {g_dense_plan.kernel, 1, 0};
  if (g_dense_plan.splits) {
    plan.splits = g_dense_plan.splits;
    while (plan.splits > 1 && split_bytes(plan.splits, KIND == kEpiGated ? 2 : a.nbatch, a.M, a.N) > a.part_bytes)
      --plan.splits;
  }
  a.splits = plan.splits;
  a.head = plan.head;
  a.head_rows = plan.head * (plan.kernel == MOE_DENSE_TILE256 ? 256 : 128);
  a.epi.stream = 2.0 * a.M * a.N * a.nbatch >= 16e6;
  return hipSuccess;
}

template <typename T, int OA, int OB, int KIND>
hipError_t run_tile(const TileArgs& a, const DensePlan& plan, hipStream_t st) {
  const hipError_t e = start_plan<T, OA, OB, KIND>(a, plan.kernel, st);
  return e != hipSuccess || a.splits == 1 ? e : launch_finish(__is_same(T, __bf16) ? MOE_BF16 : MOE_F16, a, KIND, st);
}

template <typename T, int OA, int OB, int KIND>
hipError_t launch_tile_k(const TileArgs& args, hipStream_t st) {
  TileArgs a = args;
  DensePlan plan{};
  double us;
  const hipError_t e = prepare_tile<OA, OB, KIND>(a, plan, us, st);
  return e != hipSuccess ? e : run_tile<T, OA, OB, KIND>(a, plan, st);
}

// The products (and bias sums) of a backward pass; dx.nseg, dw.nbatch or db.runs 0: not wanted.
template <typename T>
hipError_t launch_backward_t(const TileArgs& dx_args, const TileArgs& dw_args, const BiasSumArgs& db, hipStream_t st) {
  TileArgs dx = dx_args, dw = dw_args;
  DensePlan px, pw;
  double ux = 0, uw = 0;
  hipError_t e;
  if (dx.nseg && (e = prepare_tile<kRows, kCols, kEpiStore>(dx, px, ux, st)) != hipSuccess) return e;
  if (dw.nbatch && (e = prepare_tile<kCols, kCols, kEpiStore>(dw, pw, uw, st)) != hipSuccess) return e;
  const bool small = [&] {  // both on 64 x 64 tiles by choice, and faster together unsplit
    if (!dx.nseg || !dw.nbatch || px.kernel != MOE_DENSE_TILE64 || pw.kernel != MOE_DENSE_TILE64) return false;
    if (g_dense_plan.splits > 1) return false;
    const TileCost& k = kWholeCosts[0];
    const int64_t nx = (int64_t)((dx.M + 63) / 64) * ((dx.N + 63) / 64), nw = (int64_t)((dw.M + 63) / 64) * ((dw.N + 63) / 64) * dw.nbatch;
    const int64_t sx = (int64_t)((dx.R + kStepR - 1) / kStepR) * dx.nseg, sw = (dw.R + kStepR - 1) / kStepR;
    const int64_t per_cu = (nx + nw + 255) / 256;
    const double each = per_cu > 1 ? k.pair / 2 : k.lone, mean = (double)(nx * sx + nw * sw) / 256 * each;
    const double longest = (sx > sw ? sx : sw) * k.lone;
    return 3.0 + (mean > longest ? mean : longest) + k.round * per_cu < ux + uw;
  }();
  if (small) {
    int64_t nx, nw;
    dx.splits = dw.splits = 1;
    if (!set_tiles<64, 64, 256>(dx, &nx) || !set_tiles<64, 64, 256>(dw, &nw)) return hipErrorInvalidConfiguration;
    const int64_t nb = db.runs ? ((int64_t)db.mats * db.N + 31) / 32 : 0;
    k_backward_small<T><<<dim3((uint32_t)(nx + nw + nb)), dim3(256), 0, st>>>(dx, dw, db, (uint32_t)nx, (uint32_t)nw);
    return hipGetLastError();
  }
  if (db.runs && (e = launch_bias_sum(__is_same(T, __bf16) ? MOE_BF16 : MOE_F16, db, st)) != hipSuccess) return e;
  if (dx.nseg && (e = run_tile<T, kRows, kCols, kEpiStore>(dx, px, st)) != hipSuccess) return e;
  return dw.nbatch ? run_tile<T, kCols, kCols, kEpiStore>(dw, pw, st) : hipSuccess;
}

template <typename T>
hipError_t launch_forward_t(const TileArgs& a, int kind, hipStream_t st) {
  return kind == kEpiGated ? launch_tile_k<T, kRows, kRows, kEpiGated>(a, st) : launch_tile_k<T, kRows, kRows, kEpiLinear>(a, st);
}

}  // namespace moe
