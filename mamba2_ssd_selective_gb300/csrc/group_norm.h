// Group norm with an activation, internal.
#pragma once

#include "launch.h"

namespace ssd {

struct GnProblem {
  int n, m, C, G, cg;  // samples, rows of a sample, channels, groups, channels of a group
  int act;             // ssd_activation
  const void *x, *z, *dy;
  void *y, *dx, *dz;
  int xs, zs, dys, ys, dxs, dzs;  // row strides (elements)
  const float *w, *b;                   // or null: 1 and 0
  float eps;
  float *mean, *rstd;  // (n, G): written by the forward pass (may be null), read by the backward pass
  float *dw, *db;      // (C), may be null
};

// Places of 8 channels of a thread whose block takes a group or a tile of one: forward keeps x alone (57 samples of 771 rows
// of 16 groups of 64 channels, bf16: 68 us with 8, 78 us with 4), backward three tensors and their gradients.
constexpr int kForwardPlaces = 8, kBackwardPlaces = 4;

// How a call is cut up.  The workspace's size does not depend on alignments: it
// suffices for any width of accesses.
struct GnPlan {
  int vec;                // channels of an access: 8 (16 bytes of bf16), 2 or 1
  int team, places;       // threads of a group's team and places of a thread
  int tiles, tile_rows;   // 0: a group fits its team; else tiles of rows of a sample
  int cluster;            // blocks of a cluster that holds a group's tiles, or 0: the tiles are read twice
  bool own_columns;       // a thread keeps one column of channels: dw and db come out of the gradient kernel
  int groups_per_block, samples_per_block;  // of a block of teams
  int partials;           // partial dw / db rows
  size_t part, dwp, dbp, total;  // workspace: (n, G, tiles, 2) and (partials, C) fp32 twice
};

// widest: channels that every tensor of the call allows at once (8, 2 or 1)
GnPlan gn_plan(const GnProblem &p, bool backward, int widest);
size_t gn_workspace(const GnProblem &p, bool backward);
template <typename T> void run_gn_forward(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s);
template <typename T> void run_gn_backward(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s);
template <> void run_gn_forward<float>(const GnProblem &, const GnPlan &, char *, cudaStream_t);
template <> void run_gn_forward<__nv_bfloat16>(const GnProblem &, const GnPlan &, char *, cudaStream_t);
template <> void run_gn_backward<float>(const GnProblem &, const GnPlan &, char *, cudaStream_t);
template <> void run_gn_backward<__nv_bfloat16>(const GnProblem &, const GnPlan &, char *, cudaStream_t);
// dw and db as sums of their partials, in order (gn_plan.cu)
void launch_gn_param_sum(int C, int partials, const float *dwp, const float *dbp, float *dw, float *db, cudaStream_t s);

}  // namespace ssd
