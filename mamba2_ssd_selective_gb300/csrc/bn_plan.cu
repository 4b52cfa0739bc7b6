// The join of a block's output with the residual stream: how a row is spread over threads, and the parameters' sums.
#include "block_norm.h"

namespace ssd {

BnTeam bn_team(int C) {
  const int units = (C + 7) / 8;
  if (units <= 32) return {32, 1};
  if (units <= 64) return {32, 2};
  if (units <= 128) return {32, 4};
  // a block of at most 512 threads
  auto warps = [](int n) { return (n + 31) / 32 * 32; };
  if (units <= 512) return {warps(units), 1};
  if (units <= 1024) return {warps((units + 1) / 2), 2};
  return {warps((units + 3) / 4), 4};
}

int bn_blocks(int rows, int C) {
  const BnTeam t = bn_team(C);
  // (a workspace's size may be asked for where there is no GPU: the SMs are not asked)
  const int most = 152 * 2;
  if (t.threads == 32) return 8 * ((rows + 7) / 8 < most ? (rows + 7) / 8 : most);
  return rows < most ? rows : most;
}

namespace {

// sums of the sets in order: 8 threads to a column, then their sums
__global__ void __launch_bounds__(256) bn_sums_kernel(const float *part, int sets, int C, float *dpw, float *dsc, float *dw) {
  __shared__ float sm[8][32];
  float *out = blockIdx.y == 0 ? dpw : blockIdx.y == 1 ? dsc : dw;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < C)
    for (int i = warp; i < sets; i += 8) s += part[((size_t)i * 3 + blockIdx.y) * C + c];
  sm[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < C) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sm[w][lane];
    out[c] = s;
  }
}

}  // namespace

void launch_bn_sums(const BnProblem &p, cudaStream_t s) {
  bn_sums_kernel<<<dim3((unsigned)((p.C + 31) / 32), 3), 256, 0, s>>>(p.part, bn_blocks(p.rows, p.C), p.C, p.dpw, p.dsc, p.dw);
}

}  // namespace ssd
