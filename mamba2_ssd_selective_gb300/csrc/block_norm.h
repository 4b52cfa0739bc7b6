// The join of a block's output with the residual stream, between its norms, internal: a call's description and the
// launchers.
//     u = x rstd_post post_weight (post_norm; else x),   t = u z sigmoid(z) (gate; else u)
//     h = residual + branch_scale t,   y = h rstd_pre pre_weight (pre_norm)
// rstd = 1 / sqrt(mean of squares of the row + eps).
#pragma once

#include "launch.h"

namespace ssd {

constexpr int kBnMaxChannels = 16384;  // 512 threads of 32 values

struct BnProblem {
  int rows, C;
  int post, gate, pre;
  const void *x, *z, *res;
  long long xs, zs, rs;  // row strides (elements)
  const float *pw, *sc, *w;  // or null: 1
  float eps;
  // forward
  void *h, *y;
  long long hs, ys;
  float *rstd_post, *rstd_pre;
  // backward: h is read; dh and dy may be null (zero)
  const void *dh, *dy;
  long long dhs, dys;
  void *dx, *dz, *dres;
  long long dxs, dzs, drs;
  float *dpw, *dsc, *dw;
  float *part;  // (blocks, 3, C) partial sums of dpw, dsc, dw
};

// threads of a row: whole warps whose threads have 8, 16 or 32 values each
struct BnTeam {
  int threads, per;  // per: units of 8 values a thread
};
BnTeam bn_team(int channels);
int bn_blocks_per_sm(const BnTeam &team, int vec);  // of the backward pass
int bn_blocks(int rows, int channels, int vec);     // likewise, all of them: one set of partial sums each (most with vec 8)

// T: x, z, y; R: the residual stream; vec: channels that the tensors' addresses and strides allow at once (8, 2, 1)
template <typename T, typename R> void launch_bn_forward(const BnProblem &p, int vec, cudaStream_t s);
template <typename T, typename R> void launch_bn_backward(const BnProblem &p, int vec, cudaStream_t s);
void launch_bn_sums(const BnProblem &p, int vec, cudaStream_t s);

}  // namespace ssd
