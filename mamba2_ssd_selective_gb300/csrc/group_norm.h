// Group norm with an activation, internal.
#pragma once

#include "launch.h"

namespace ssd {

struct GnProblem {
  int n, m, C, G, cg;  // samples, rows of a sample, channels, groups, channels of a group
  int act;             // ssd_activation
  int eb;              // bytes of an element
  const void *x, *z, *dy;
  void *y, *dx, *dz;
  long long xs, zs, dys, ys, dxs, dzs;  // row strides (elements)
  const float *w, *b;                   // or null: 1 and 0
  float eps;
  float *mean, *rstd;  // (n, G): written by the forward pass (may be null), read by the backward pass
  float *dw, *db;      // (C), may be null
};

struct GnPlan {
  int tiles;                 // row tiles that hold a partial dweight / dbias each
  size_t dwp, dbp, total;    // (tiles, C) fp32 each
};

GnPlan gn_plan(const GnProblem &p, bool backward);
template <typename T> void run_gn_forward(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s);
template <typename T> void run_gn_backward(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s);

}  // namespace ssd
