// Group norm with an activation: which kernels a call takes, its workspace, and
// the sum of the parameters' partial gradients.
#include "group_norm.cuh"

namespace ssd {

namespace {

constexpr int kSms = 152;  // not asked for: a workspace's size may be, where there is no GPU

// Partials of one channel, 16 threads a channel: thread q adds partials q, q + 16, ... in order, then
// the 16 sums are added in order.
constexpr int kSumLanes = 16, kSumCols = gn::kThreads / kSumLanes;
__global__ void __launch_bounds__(gn::kThreads) param_sum_kernel(int C, int partials, const float *__restrict__ dwp,
                                                                 const float *__restrict__ dbp, float *dw, float *db) {
  __shared__ float acc[2][kSumLanes][kSumCols];
  const int cl = threadIdx.x % kSumCols, q = threadIdx.x / kSumCols, c = blockIdx.x * kSumCols + cl;
  float sw = 0.f, sb = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int t = q; t < partials; t += kSumLanes) {
      sw += dwp[(size_t)t * C + c];
      sb += dbp[(size_t)t * C + c];
    }
  }
  acc[0][q][cl] = sw;
  acc[1][q][cl] = sb;
  __syncthreads();
  if (q == 0 && c < C) {
    sw = sb = 0.f;
#pragma unroll
    for (int i = 0; i < kSumLanes; ++i) {
      sw += acc[0][i][cl];
      sb += acc[1][i][cl];
    }
    if (dw) dw[c] = sw;
    if (db) db[c] = sb;
  }
}

}  // namespace

void launch_gn_param_sum(int C, int partials, const float *dwp, const float *dbp, float *dw, float *db,
                         cudaStream_t s) {
  param_sum_kernel<<<(C + kSumCols - 1) / kSumCols, gn::kThreads, 0, s>>>(C, partials, dwp, dbp, dw, db);
}

GnPlan gn_plan(const GnProblem &p, bool backward, int widest) {
  GnPlan pl{};
  pl.vec = widest >= 8 && p.cg % 8 == 0 ? 8 : widest >= 2 && p.cg % 2 == 0 ? 2 : 1;
  const int ncol = p.cg / pl.vec, block_places = pl.vec == 8 ? (backward ? kBackwardPlaces : kForwardPlaces) : 12;
  // Widths: rows of 16 bytes where a group allows it; pairs of channels halve the accesses of groups that eight do
  // not divide (6 samples of 4099 rows of 32 groups of 10 channels, fp32: 51 us one by one, 37 us in pairs).
  // The narrowest team that holds a group; backward teams also need a thread to keep its column.
  if (p.m == 1 && ncol <= 32) {
    pl.team = ncol <= 4 ? 4 : ncol <= 8 ? 8 : ncol <= 16 ? 16 : 32;
    pl.places = 1;
  } else if (p.m <= gn::rows_of_team(ncol, 32, 4) && (!backward || ncol <= 32)) {
    pl.team = 32;
    pl.places = 4;
  } else {
    pl.team = gn::kThreads;
    pl.places = block_places;
    const long long rows = gn::rows_of_team(ncol, pl.team, pl.places);
    if (p.m > rows || (backward && ncol > pl.team)) {
      pl.tile_rows = (int)rows;
      const long long tiles = ncol <= pl.team ? (p.m + rows - 1) / rows
                                              : ((long long)p.m * ncol + pl.places * pl.team - 1) / (pl.places * pl.team);
      pl.tiles = (int)tiles;
      pl.cluster = ncol > pl.team ? 0 : tiles <= 2 ? 2 : tiles <= 4 ? 4 : tiles <= 8 ? 8 : 0;  // 8: the largest portable cluster
    }
  }
  pl.own_columns = ncol <= pl.team;
  if (pl.tiles == 0) {
    const int teams = gn::kThreads / pl.team;
    pl.groups_per_block = teams < p.G ? teams : p.G;
    // blocks that fill the GPU a few times over, but no fewer samples than a block's teams take at once
    const long long gblocks = (p.G + pl.groups_per_block - 1) / pl.groups_per_block, shares = teams / pl.groups_per_block;
    // (a backward block writes a partial row of dw and db, and as many are resident at once)
    const long long want = (backward ? (pl.places == 1 ? 3 : 2) : 8) * kSms;
    long long per = (p.n * gblocks + want - 1) / want;
    per = (per + shares - 1) / shares * shares;
    while ((p.n + per - 1) / per > 65535) per *= 2;
    pl.samples_per_block = (int)per;
  }
  if (backward)
    pl.partials = !pl.own_columns ? (int)(((long long)p.n * p.m + gn::kParamRows - 1) / gn::kParamRows)
                  : pl.tiles      ? p.n * pl.tiles
                                  : (p.n + pl.samples_per_block - 1) / pl.samples_per_block;
  size_t off = 256;  // never empty
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  pl.part = take((size_t)p.n * p.G * pl.tiles * 8);
  pl.dwp = take((size_t)pl.partials * p.C * 4);
  pl.dbp = take((size_t)pl.partials * p.C * 4);
  pl.total = off;
  return pl;
}

size_t gn_workspace(const GnProblem &p, bool backward) {
  size_t most = 0;
  for (int widest : {8, 2, 1}) {
    const size_t t = gn_plan(p, backward, widest).total;
    if (t > most) most = t;
  }
  return most;
}

}  // namespace ssd
