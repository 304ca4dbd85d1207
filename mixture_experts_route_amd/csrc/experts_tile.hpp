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
// is ever named; one workgroup reports them.
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
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    a.a[m] = (const uint16_t*)a.a[m] + t.row0 * a.lda[0];
    a.b[m] = (const uint16_t*)a.b[m] + t.e * g.stride;
    if (a.epi.pre[m]) a.epi.pre[m] = (uint16_t*)a.epi.pre[m] + t.row0 * a.epi.ldp[m];
  }
  a.epi.y[0] = (uint16_t*)a.epi.y[0] + t.row0 * a.epi.ldy[0];
  return true;
}

// This workgroup's tile of dW, its reduction the expert's rows.  Consecutive tiles are of one expert, and an XCD takes a
// run of them.
MOE_DEV void group_sums(const GroupArgs& g, TileArgs& a, TileIndex& x) {
  a = g.tile;
  const uint32_t each = (uint32_t)a.tiles_i * (uint32_t)a.tiles_j, count = gridDim.x;
  const uint32_t q = count / 8, rem = count % 8, xcd = blockIdx.x % 8;
  const uint32_t t = xcd * q + (xcd < rem ? xcd : rem) + blockIdx.x / 8;
  const uint32_t me = t / each, in = t - me * each;
  const int e = (int)(me / (uint32_t)g.mats), m = (int)(me - (uint32_t)e * g.mats);
  x = {0, (int)(in / (uint32_t)a.tiles_j), (int)(in % (uint32_t)a.tiles_j), 0, 1};
  const int o0 = g.offsets[e], o1 = g.offsets[e + 1];
  const int lo = clamp_rows(o0, g.P), hi = clamp_rows(o1, g.P);
  if (in == 0 && threadIdx.x == 0 && (o0 != lo || o1 != hi || hi < lo)) set_error(g.ctrl, MOE_DERR_ROWS);
  a.R = hi > lo ? hi - lo : 0;
  a.a[0] = (const uint16_t*)(m ? a.a[1] : a.a[0]) + lo * a.lda[0];
  a.b[0] = (const uint16_t*)a.b[0] + lo * a.ldb[0];
  a.epi.y[0] = (uint16_t*)(m ? a.epi.y[1] : a.epi.y[0]) + e * g.stride;
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

template <typename T, int OA, int OB, int KIND, int WI, int WJ, int FI, int FJ>
__global__ __launch_bounds__(64 * WI * WJ, 2) void k_group_big(GroupArgs g) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[big_lds(WI, WJ, FI, FJ)];
  constexpr int TI = 2 * WI * FI * 16, TJ = 2 * WJ * FJ * 16;
  TileArgs a;
  TileIndex x;
  if constexpr (OA == kCols) {
    group_sums(g, a, x);
    if (a.R == 0) return zero_tile<T, 64 * WI * WJ>(a, (int64_t)x.ti * TI, TI, (int64_t)x.tj * TJ, TJ);
  } else if (!group_rows<TI>(g, a, x)) {
    return;
  }
  big_tile<T, OA, OB, KIND, WI, WJ, FI, FJ>(a, x, lds);
}

template <typename T, int OA, int OB, int KIND>
__global__ __launch_bounds__(256, 2) void k_group_deep(GroupArgs g) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[kDeepStages * kDeepStageBytes / 2];
  TileArgs a;
  TileIndex x;
  if constexpr (OA == kCols) {
    group_sums(g, a, x);
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
    group_sums(g, a, x);
    if (a.R == 0) return zero_tile<T, 256>(a, (int64_t)x.ti * TT, TT, (int64_t)x.tj * TT, TT);
  } else if (!group_rows<TT>(g, a, x)) {
    return;
  }
  any_tile<T, OA, OB, KIND, F>(a, x, lds);
}

// The tile with the least estimated time, by the costs measured for the dense products (TileCost).  The rows of an
// expert are not known here: rows of tiles are taken as P / tile + half the experts that can have rows, but at least
// those.
template <int OA, int KIND>
int plan_group(const GroupArgs& g, bool whole) {
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
    count = (int64_t)g.E * g.mats * g.tile.tiles_i * g.tile.tiles_j;
  } else {
    count = most_tiles(g, tile) * g.tile.tiles_j;
  }
  *grid = (uint32_t)count;
  return count <= (int64_t)0xFFFFFFFF / threads;
}

template <typename T, int OA, int OB, int KIND>
hipError_t launch_experts(const GroupArgs& args, hipStream_t st) {
  GroupArgs g = args;
  bool whole = g.stride % 8 == 0 || OA == kCols;
  for (int m = 0; m < (OA == kCols ? g.mats : g.tile.nseg); ++m) whole = whole && whole_chunks(OA, g.tile.a[m], g.tile.lda[0], g.tile.len_a);
  for (int m = 0; m < (OA == kCols ? 1 : KIND == kEpiGated || g.tile.nseg > 1 ? 2 : 1); ++m)
    whole = whole && whole_chunks(OB, g.tile.b[m], g.tile.ldb[m], g.tile.R);
  int kernel = g_dense_plan.kernel;
  if (kernel == MOE_DENSE_AUTO || (!whole && kernel < MOE_DENSE_ANY64)) kernel = plan_group<OA, KIND>(g, whole);
  g.tile.splits = 1;
  const double out = OA == kCols ? 2.0 * g.E * g.mats * g.tile.M * g.tile.N : 2.0 * g.P * g.tile.N;
  g.tile.epi.stream = out >= 16e6;
  uint32_t grid;
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

template <typename T>
hipError_t launch_experts_forward_t(const GroupArgs& g, int kind, hipStream_t st) {
  return kind == kEpiGated ? launch_experts<T, kRows, kRows, kEpiGated>(g, st) : launch_experts<T, kRows, kRows, kEpiStore>(g, st);
}

}  // namespace moe
