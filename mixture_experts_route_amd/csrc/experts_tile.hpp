// Tile products of the experts: the dense operators' tile kernels, each workgroup on one expert's rows.
//
// How many rows an expert has is known on the device only.  A launch over rows (forward, dx) takes the largest grid
// that any distribution of P rows over E experts can need, sum_e ceil(rows_e / tile) <= P / tile + min(E, P) rows of
// tiles; each wave finds its tile's expert from the offsets by itself (two loads' latency and two scans, about 1 us,
// where a launch that made a list of tiles would cost 2 to 3), and workgroups past the last tile leave at once.  The order
// of tiles goes by their true number, so that every XCD has the same share of them.
#pragma once

#include "dense_tile.hpp"
#include "experts.hpp"

namespace moe {

struct GroupTile {
  int e, tile, row0, rows;  // the expert, the tile among its own, its rows in the matrices
};

MOE_DEV int wave_scan(int v) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}
MOE_DEV int clamp_rows(int v, int P) { return v < 0 ? 0 : (v > P ? P : v); }

// Rows of tiles of TI rows over all experts, and this lane's share: experts lane * per .. + per - 1.  Offsets that do not
// ascend within 0 .. P are taken as clamped to it and an expert's negative rows as none: no row outside the matrices
// is ever named; one workgroup reports them.  Rows that such offsets name many times over would take the sums past 32 bits (1024
// experts of 2^28 rows each), so a lane counts no more tiles than good offsets can give it.
template <int TI>
MOE_DEV int count_tiles(const GroupArgs& g, int per, int& mine, int& incl) {
  const int lane = threadIdx.x & 63;
  const int first = lane * per;
  int prev = g.offsets[first < g.E ? first : g.E];
  bool bad = prev < 0 || prev > g.P;
  prev = clamp_rows(prev, g.P);
  mine = 0;
  for (int i = 0; i < per; i += 4) {
    int next[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) next[u] = g.offsets[first + i + u + 1 < g.E ? first + i + u + 1 : g.E];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i + u >= per) break;
      bad |= next[u] < prev || next[u] > g.P;
      const int at = clamp_rows(next[u], g.P);
      mine += at > prev ? (at - prev + TI - 1) / TI : 0;
      prev = at;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < 64 && bad) set_error(g.ctrl, MOE_DERR_ROWS);
  mine = mine < g.P / TI + per ? mine : g.P / TI + per;
  incl = wave_scan(mine);
  return __builtin_amdgcn_readlane(incl, 63);
}

// Tile `t` of all experts' rows of tiles; per, mine and incl as count_tiles has them.
template <int TI>
MOE_DEV GroupTile find_tile(const GroupArgs& g, int t, int per, int mine, int incl) {
  const int lane = threadIdx.x & 63;
  const int owner = __builtin_ctzll(__ballot(incl > t));
  t -= __builtin_amdgcn_readlane(incl - mine, owner);
  const int e = owner * per + lane;
  const bool own = lane < per && e < g.E;
  const int lo = clamp_rows(g.offsets[own ? e : 0], g.P), hi = clamp_rows(g.offsets[own ? e + 1 : 0], g.P);
  const int rows = own && hi > lo ? hi - lo : 0, tiles = (rows + TI - 1) / TI;
  const int scan = wave_scan(tiles);
  const int at = __builtin_ctzll(__ballot(scan > t));
  GroupTile x;
  x.e = owner * per + at;
  x.tile = t - __builtin_amdgcn_readlane(scan - tiles, at);
  x.row0 = __builtin_amdgcn_readlane(lo, at);
  x.rows = __builtin_amdgcn_readlane(rows, at);
  return x;
}

// This workgroup's tile of a product over rows, as arguments of its expert's product; false: there is none.
template <int TI>
MOE_DEV bool group_rows(const GroupArgs& g, TileArgs& a, TileIndex& x) {
  const int per = (g.E + 63) / 64;
  int mine, incl;
  a = g.tile;
  a.tiles_i = count_tiles<TI>(g, per, mine, incl);
  const uint32_t count = (uint32_t)a.tiles_i * (uint32_t)a.tiles_j;
  if (blockIdx.x >= count) return false;
  x = tile_index<false>(a, blockIdx.x, count);
  const GroupTile t = find_tile<TI>(g, x.ti, per, mine, incl);
  x.ti = t.tile;
  a.M = t.rows;
  a.b_once = t.rows <= TI;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    a.a[m] = (const uint16_t*)a.a[m] + t.row0 * a.lda[0];
    a.b[m] = (const uint16_t*)a.b[m] + t.e * g.stride;
    if (a.epi.pre[m]) a.epi.pre[m] = (uint16_t*)a.epi.pre[m] + t.row0 * a.epi.ldp[m];
  }
  a.epi.y[0] = (uint16_t*)a.epi.y[0] + t.row0 * a.epi.ldy[0];
  return true;
}

// Tiles of dW, whose reduction is an expert's rows.  A tile's time goes by its expert's rows, so each matrix's tiles are
// spread over all XCDs, each XCD taking a run of an eighth of them (a run of whole experts per XCD: 8 experts of 4096 rows
// on average, the longest three times that, 4096 x 4096, 2273 us; spread 922), along the shorter side first, which reads the
// fewest different operand columns.
struct DwTile {
  int e, m, ti, tj, row0, rows;
};
// Tile `id` of the launch's; false: there is none.
MOE_DEV bool dw_tile(const GroupArgs& g, uint32_t id, DwTile& x) {
  const uint32_t ti = (uint32_t)g.tile.tiles_i, tj = (uint32_t)g.tile.tiles_j;
  const uint32_t run = (ti * tj + 7) / 8, at = id / 8, me = at / run, in = id % 8 * run + (at - me * run);
  if (in >= ti * tj) return false;
  x.e = (int)(me / (uint32_t)g.mats);
  x.m = (int)(me - (uint32_t)x.e * g.mats);
  x.ti = (int)(ti < tj ? in % ti : in / tj);
  x.tj = (int)(ti < tj ? in / ti : in % tj);
  const int o0 = __builtin_amdgcn_readfirstlane(g.offsets[x.e]), o1 = __builtin_amdgcn_readfirstlane(g.offsets[x.e + 1]);
  const int lo = clamp_rows(o0, g.P), hi = clamp_rows(o1, g.P);
  if (in == 0 && threadIdx.x == 0 && (o0 != lo || o1 != hi || hi < lo)) set_error(g.ctrl, MOE_DERR_ROWS);
  x.row0 = lo;
  x.rows = hi > lo ? hi - lo : 0;
  return true;
}
// This workgroup's tile of dW, as arguments of its expert's product; false: there is none.
MOE_DEV bool group_sums(const GroupArgs& g, uint32_t id, TileArgs& a, TileIndex& x) {
  DwTile t;
  if (!dw_tile(g, id, t)) return false;
  a = g.tile;
  x = {0, t.ti, t.tj, 0, 1};
  a.R = t.rows;
  a.a[0] = (const uint16_t*)(t.m ? a.a[1] : a.a[0]) + t.row0 * a.lda[0];
  a.b[0] = (const uint16_t*)a.b[0] + t.row0 * a.ldb[0];
  a.epi.y[0] = (uint16_t*)(t.m ? a.epi.y[1] : a.epi.y[0]) + t.e * g.stride;
  return true;
}

// The dW of an expert without rows.
template <typename T, int THREADS>
MOE_DEV void zero_tile(const TileArgs& a, int64_t i0, int rows, int64_t j0, int cols) {
  const float zero[8] = {};
  const int chunks = cols / 8;
  for (int c = threadIdx.x; c < rows * chunks; c += THREADS) {
    const int64_t i = i0 + c / chunks, j = j0 + c % chunks * 8;
    if (i < a.M && j < a.N) store8<T>(a.epi.y[0], i * a.epi.ldy[0] + j, a.N - j < 8 ? (int)(a.N - j) : 8, zero, a.epi.stream);
  }
}

// The weights of an expert with one row of tiles are read once, and hinted so: 2048 x 768 gated, 512 experts, 256 tokens' ten
// 420 -> 389 us, 4096 tokens' 808 -> 790; hinted throughout, the popular experts' tiles miss each other's (4096: 812).  (Not
// in the 64-square kernel: one token 14.5 us, 15.1 hinted.)
template <typename T, int OA, int OB, int KIND, int WI, int WJ, int FI, int FJ>
__global__ __launch_bounds__(64 * WI * WJ, 2) void k_group_big(GroupArgs g) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[big_lds(WI, WJ, FI, FJ)];
  constexpr int TI = 2 * WI * FI * 16, TJ = 2 * WJ * FJ * 16;
  TileArgs a;
  TileIndex x;
  if constexpr (OA == kCols) {
    if (!group_sums(g, blockIdx.x, a, x)) return;
    if (a.R == 0) return zero_tile<T, 64 * WI * WJ>(a, (int64_t)x.ti * TI, TI, (int64_t)x.tj * TJ, TJ);
  } else if (!group_rows<TI>(g, a, x)) {
    return;
  }
  big_tile<T, OA, OB, KIND, WI, WJ, FI, FJ, OA == kRows>(a, x, lds);
}

template <typename T, int OA, int OB, int KIND>
__global__ __launch_bounds__(256, 2) void k_group_deep(GroupArgs g) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[kDeepStages * kDeepStageBytes / 2];
  TileArgs a;
  TileIndex x;
  if constexpr (OA == kCols) {
    if (!group_sums(g, blockIdx.x, a, x)) return;
    if (a.R == 0) return zero_tile<T, 256>(a, (int64_t)x.ti * 64, 64, (int64_t)x.tj * 64, 64);
  } else if (!group_rows<64>(g, a, x)) {
    return;
  }
  deep_tile<T, OA, OB, KIND>(a, x, lds);
}

template <typename T, int OA, int OB, int KIND, int F>
__global__ __launch_bounds__(256, 2) void k_group_any(GroupArgs g) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[any_lds(F)];
  constexpr int TT = 64 * F;
  TileArgs a;
  TileIndex x;
  if constexpr (OA == kCols) {
    if (!group_sums(g, blockIdx.x, a, x)) return;
    if (a.R == 0) return zero_tile<T, 256>(a, (int64_t)x.ti * TT, TT, (int64_t)x.tj * TT, TT);
  } else if (!group_rows<TT>(g, a, x)) {
    return;
  }
  any_tile<T, OA, OB, KIND, F>(a, x, lds);
}

// Mean rows of an expert up to which dW takes k_group_dw.  Against the best of the pipelined tiles, lengths spread
// exponentially, 768 x 2048: 512 experts of 20 rows 337 and 361 us, of 80 rows 467 and 483; 256 of 160 rows 296 and 306; 128
// of 320 rows 220 both; 64 of 512 rows 144 and 135, of 1024 rows 276 and 233.
constexpr int kShortRows = 320;

// dW of experts with few rows: 128 x 128 tile, 4 waves of 64 x 64.  A reduction of a step or two is over before a pipeline has
// filled, so there is none: a step's operands come into one LDS buffer of 32 KB, and the four workgroups that fit a CU
// cover each other's loads and stores.  A wave's results leave, through the same LDS, as whole 128-byte lines.  512 Zipf experts
// of 80 rows, 2 x 768 x 2048 (3.2 GB written): 935 us, 4.7 TB/s of what it reads and writes; of one matrix's 483 us the stores
// alone take 264 and everything else alone 180.  (Two workgroups per CU that walk over the tiles with the next one's operands
// on their way: 538; 128 x 256: 550.)
constexpr int kDwLds = (128 + 128) * kStepR;  // elements
template <typename T>
MOE_DEV void short_dw(const GroupArgs& g, uint32_t id, uint16_t* lds) {
  constexpr int HI = 128, HJ = 128, WJ = 2, W = 2 * WJ, F = 4;
  typedef typename Operand<T>::v8 v8;
  TileArgs a;
  TileIndex x;
  if (!group_sums(g, id, a, x)) return;
  const int64_t i0 = (int64_t)x.ti * HI, j0 = (int64_t)x.tj * HJ;
  if (a.R == 0) return zero_tile<T, 64 * W>(a, i0, HI, j0, HJ);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / WJ, wj = wave % WJ;
  const int steps = (a.R + kStepR - 1) / kStepR;
  OperandCopy<kCols, HI, W> ca;
  OperandCopy<kCols, HJ, W> cb;
  HalfStream<kCols, HI, W, false> sa;
  HalfStream<kCols, HJ, W, false> sb;
  ca.init(a.lda[0], wave, lane);
  cb.init(a.ldb[0], wave, lane);
  sa.init(ca, a.a[0], nullptr, a.lda[0], 0, i0, a.M, a.R, steps, 0, steps);
  sb.init(cb, a.b[0], nullptr, a.ldb[0], 0, j0, a.N, a.R, steps, 0, steps);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t*)lds;
  const uint32_t addr_a = frag_addr<kCols, HI>(lds0, wi * 64, lane);
  const uint32_t addr_b = frag_addr<kCols, HJ>(lds0 + 2 * HI * kStepR, wj * 64, lane);
  float4v acc[F][F] = {};
  for (int k = 0; k < steps; ++k) {
    sa.issue(ca, lds0 + wave * 1024);
    sb.issue(cb, lds0 + 2 * HI * kStepR + wave * 1024);
    copies_barrier<0>();
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      v8 fa[F], fb[F];
#pragma unroll
      for (int n = 0; n < F; ++n) {
        fa[n] = read_frag<T, kCols, HI>(addr_a, n, kk, 0);
        fb[n] = read_frag<T, kCols, HJ>(addr_b, n, kk, 0);
      }
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int n = 0; n < F; ++n) acc[f][n] = Operand<T>::mma(fb[n], fa[f], acc[f][n]);
    }
    copies_barrier<0>();  // every wave has read the step
  }
  store_block<T, F, F>(a.epi.y[0], a.epi.ldy[0], i0 + wi * 64, j0 + wj * 64, a.M, a.N, a.epi.stream, acc, lds + wave * 4096, lane);
}

template <typename T>
__global__ __launch_bounds__(256, 4) void k_group_dw(GroupArgs g) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[kDwLds];
  short_dw<T>(g, blockIdx.x, lds);
}

// dx's 128-square tiles up to which dx and dW are one launch: a round of them, two workgroups a CU.
constexpr uint32_t kOneRound = 512;

// A backward pass whose dx has few tiles: those first, dW's beside and behind them, in one launch.  dx alone leaves CUs idle,
// more so where few experts hold most rows, and a launch costs two to three microseconds (lengths spread exponentially: 8
// experts of 40 rows, gated 768 of 2048, 49.2 -> 40.9 us; 24 of 28 rows, 1360 of 1000, 50.3 -> 45.4; 64 of 64 rows, 512 of 512,
// 33 -> 24.7; 4 of 300 rows, 2048 of 2048, 61.8 -> 52.7).  Behind more than a round of dx's tiles, dW's run two to a CU here
// instead of k_group_dw's four: 32 experts of 40 rows, gated 768 of 2048, 107 alone and 113 joined; 256 experts, 768 of 2048,
// 392 and 460.  dx's 64-square tiles are only taken where 704 at most are needed, and gained throughout.
template <typename T, int TILE>
__global__ __launch_bounds__(256, 2) void k_group_backward(GroupArgs dx, GroupArgs dw, uint32_t n_dx) {
  constexpr int kLds = TILE == 64 ? kDeepStages * kDeepStageBytes / 2 : big_lds(2, 2, 2, 2);
  __shared__ __attribute__((aligned(1024))) uint16_t lds[kLds > kDwLds ? kLds : kDwLds];
  if (blockIdx.x >= n_dx) {
    short_dw<T>(dw, blockIdx.x - n_dx, lds);
    return;
  }
  TileArgs a;
  TileIndex x;
  if (!group_rows<TILE>(dx, a, x)) return;
  if constexpr (TILE == 64)
    deep_tile<T, kRows, kCols, kEpiStore>(a, x, lds);
  else
    big_tile<T, kRows, kCols, kEpiStore, 2, 2, 2, 2, true>(a, x, lds);
}

// The tile of a product over rows of whole 16-byte chunks.  How many rows an expert has is not known here: rows of tiles are taken
// as P / tile + half the experts that can have rows, but at least those.  128-square tiles carry everything but the ends:
// they draw the weights fastest even where an expert has two rows (16 tokens' ten of 512 experts, 2048 x 768: 56 us, 64-square
// 71), but below two for three CUs the 64-square ones' number counts for more (one token, 768 gated of 2048: 15.5 and 23.5 us;
// 24 experts of 28 rows, 1360 of 1000, 264 tiles: 21.6 and 16.9; near the limit it goes by the sizes: 140 tiles, 8 experts of 162
// rows, 1280 of 512: 8.3 and 9.9, 160 tiles of 200 rows 12.4 and 10.0, 216 tiles, 18 of 17 rows, 1536 of 2048: 22.8 and 26.0), and from 256 rows per expert on the 256-square ones'
// reuse does (128 experts of 320 rows, 2048 x 768: 176 us, 128-square 197; 256 of 160: 241 and 250, 512 Zipf ones of 160 980
// and 966).
template <int KIND>
int plan_rows_whole(const GroupArgs& g) {
  const int64_t active = g.E < g.P ? g.E : g.P;
  auto tiles = [&](int tile) {
    const int64_t rows = g.P / tile + active / 2, tj = KIND == kEpiGated ? tile / 2 : tile;
    return (rows > active ? rows : active) * ((g.tile.N + tj - 1) / tj);
  };
  if (tiles(128) <= 176) return MOE_DENSE_TILE64;
  return g.P >= 256 * active && tiles(256) >= 256 ? MOE_DENSE_TILE256 : MOE_DENSE_TILE128;
}

// Of the kernels for any alignment, and for dW of long reductions, the tile with the least estimated time by the costs
// measured for the dense products (TileCost).
template <int OA, int KIND>
int plan_group(const GroupArgs& g, bool whole) {
  if (OA == kRows && whole) return plan_rows_whole<KIND>(g);
  const int64_t active = g.E < g.P ? g.E : g.P;
  const TileCost* costs = whole ? kWholeCosts : kAnyCosts;
  int best = 0;
  double least = 1e300;
  for (int c = 0; c < (whole ? 3 : 2); ++c) {
    const TileCost& k = costs[c];
    const int64_t tj = KIND == kEpiGated ? k.tile / 2 : k.tile, cols = (g.tile.N + tj - 1) / tj;
    double tiles, steps;
    if (OA == kCols) {
      tiles = (double)g.E * g.mats * ((g.tile.M + k.tile - 1) / k.tile) * cols;
      steps = (double)g.P / active / kStepR + 0.5;
    } else {
      const double rows = (double)g.P / k.tile + 0.5 * active;
      tiles = (rows > active ? rows : active) * cols;
      steps = (double)((g.tile.R + kStepR - 1) / kStepR) * g.tile.nseg;
    }
    const double per_cu = tiles / 256, pairs = per_cu < 2 ? 1 : per_cu / 2;
    const double t = (per_cu <= 1 ? k.lone : k.pair) * steps * pairs + k.round * pairs;
    if (t < least) {
      least = t;
      best = k.kernel;
    }
  }
  return best;
}

// Rows of tiles that a launch must provide for.
inline int64_t most_tiles(const GroupArgs& g, int tile) { return g.P / tile + (g.E < g.P ? g.E : g.P); }

template <int OA, int KIND>
bool group_grid(GroupArgs& g, int tile, int threads, uint32_t* grid) {
  const int tj = KIND == kEpiGated ? tile / 2 : tile;
  g.tile.tiles_j = (g.tile.N + tj - 1) / tj;
  int64_t count;
  if (OA == kCols) {
    g.tile.tiles_i = (g.tile.M + tile - 1) / tile;
    count = (int64_t)g.E * g.mats * (((int64_t)g.tile.tiles_i * g.tile.tiles_j + 7) / 8) * 8;
  } else {
    count = most_tiles(g, tile) * g.tile.tiles_j;
  }
  *grid = (uint32_t)count;
  return count <= (int64_t)0xFFFFFFFF / threads;
}

// What a launch is made of beside its grid; returns the kernel (kShortDw: k_group_dw).
constexpr int kShortDw = 100;
template <int OA, int OB, int KIND>
int prepare_experts(GroupArgs& g) {
  bool whole = g.stride % 8 == 0 || OA == kCols;
  for (int m = 0; m < (OA == kCols ? g.mats : g.tile.nseg); ++m) whole = whole && whole_chunks(OA, g.tile.a[m], g.tile.lda[0], g.tile.len_a);
  for (int m = 0; m < (OA == kCols ? 1 : KIND == kEpiGated || g.tile.nseg > 1 ? 2 : 1); ++m)
    whole = whole && whole_chunks(OB, g.tile.b[m], g.tile.ldb[m], g.tile.R);
  g.tile.splits = 1;
  const double out = OA == kCols ? 2.0 * g.E * g.mats * g.tile.M * g.tile.N : 2.0 * g.P * g.tile.N;
  g.tile.epi.stream = out >= 16e6;
  const int kernel = g_dense_plan.kernel;
  if (kernel != MOE_DENSE_AUTO && (whole || kernel >= MOE_DENSE_ANY64)) return kernel;
  if (OA == kCols && whole && g.P <= kShortRows * (int64_t)g.E) return kShortDw;
  return plan_group<OA, KIND>(g, whole);
}

template <typename T, int OA, int OB, int KIND>
hipError_t run_experts(GroupArgs g, int kernel, hipStream_t st) {
  uint32_t grid;
  if constexpr (OA == kCols) {
    if (kernel == kShortDw) {
      if (!group_grid<OA, KIND>(g, 128, 256, &grid)) return hipErrorInvalidConfiguration;
      k_group_dw<T><<<grid, 256, 0, st>>>(g);
      return hipGetLastError();
    }
  }
  switch (kernel) {
    case MOE_DENSE_TILE64:
      if (!group_grid<OA, KIND>(g, 64, 256, &grid)) return hipErrorInvalidConfiguration;
      k_group_deep<T, OA, OB, KIND><<<grid, 256, 0, st>>>(g);
      break;
    case MOE_DENSE_TILE128:
      if (!group_grid<OA, KIND>(g, 128, 256, &grid)) return hipErrorInvalidConfiguration;
      k_group_big<T, OA, OB, KIND, 2, 2, 2, 2><<<grid, 256, 0, st>>>(g);
      break;
    case MOE_DENSE_TILE256:
      if (!group_grid<OA, KIND>(g, 256, 512, &grid)) return hipErrorInvalidConfiguration;
      k_group_big<T, OA, OB, KIND, 2, 4, 4, 2><<<grid, 512, 0, st>>>(g);
      break;
    case MOE_DENSE_ANY64:
      if (!group_grid<OA, KIND>(g, 64, 256, &grid)) return hipErrorInvalidConfiguration;
      k_group_any<T, OA, OB, KIND, 1><<<grid, 256, 0, st>>>(g);
      break;
    default:
      if (!group_grid<OA, KIND>(g, 128, 256, &grid)) return hipErrorInvalidConfiguration;
      k_group_any<T, OA, OB, KIND, 2><<<grid, 256, 0, st>>>(g);
  }
  return hipGetLastError();
}

template <typename T, int OA, int OB, int KIND>
hipError_t launch_experts(const GroupArgs& args, hipStream_t st) {
  GroupArgs g = args;
  const int kernel = prepare_experts<OA, OB, KIND>(g);
  return run_experts<T, OA, OB, KIND>(g, kernel, st);
}

// dx (tile.nseg 0: not wanted) and dW (mats 0: not wanted).
template <typename T>
hipError_t launch_experts_backward_t(const GroupArgs& dx_args, const GroupArgs& dw_args, hipStream_t st) {
  GroupArgs dx = dx_args, dw = dw_args;
  const int kx = dx.tile.nseg ? prepare_experts<kRows, kCols, kEpiStore>(dx) : 0;
  const int kw = dw.mats ? prepare_experts<kCols, kCols, kEpiStore>(dw) : 0;
  const int tile = kx == MOE_DENSE_TILE64 ? 64 : kx == MOE_DENSE_TILE128 ? 128 : 0;
  uint32_t nx, nw;
  if (tile && kw == kShortDw && group_grid<kRows, kEpiStore>(dx, tile, 256, &nx) && (tile == 64 || nx <= kOneRound) &&
      group_grid<kCols, kEpiStore>(dw, 128, 256, &nw) && nw <= 0x7FFFFFFF / 256) {
    nx = (nx + 7) / 8 * 8;  // dW's tiles keep their XCDs
    if (tile == 64) k_group_backward<T, 64><<<nx + nw, 256, 0, st>>>(dx, dw, nx);
    else k_group_backward<T, 128><<<nx + nw, 256, 0, st>>>(dx, dw, nx);
    return hipGetLastError();
  }
  hipError_t e = hipSuccess;
  if (kx) e = run_experts<T, kRows, kCols, kEpiStore>(dx, kx, st);
  return e != hipSuccess || !kw ? e : run_experts<T, kCols, kCols, kEpiStore>(dw, kw, st);
}

template <typename T>
hipError_t launch_experts_forward_t(const GroupArgs& g, int kind, hipStream_t st) {
  return kind == kEpiGated ? launch_experts<T, kRows, kRows, kEpiGated>(g, st) : launch_experts<T, kRows, kRows, kEpiStore>(g, st);
}

}  // namespace moe
