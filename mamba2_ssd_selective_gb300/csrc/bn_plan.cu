// The join of a block's output with the residual stream: how a row is spread over threads, and the parameters' sums.
#include "block_norm.h"

namespace ssd {

// What a row costs whatever its length is shared by 16 channels a thread where it is long (gradients of 8192 x 4096: 182 us
// with 8).
BnTeam bn_team(int C) {
  const int units = (C + 7) / 8;
  if (units <= 32) return {32, 1};
  if (units <= 64) return {32, 2};
  auto warps = [](int n) { return (n + 31) / 32 * 32; };
  if (units <= 256) return {warps(units), 1};
  if (units <= 1024) return {warps((units + 1) / 2), 2};
  return {warps((units + 3) / 4), 4};
}

// as registers allow: about 100 a thread with 8 channels, 200 with 16
int bn_blocks_per_sm(const BnTeam &t) { return t.threads > 256 || t.per > 1 ? 1 : t.threads > 128 ? 2 : 4; }

int bn_blocks(int rows, int C) {
  const BnTeam t = bn_team(C);
  // (a workspace's size may be asked for where there is no GPU: the SMs are not asked)
  const int most = 152 * (t.threads == 32 ? 2 : bn_blocks_per_sm(t)), wanted = t.threads == 32 ? (rows + 7) / 8 : rows;
  return wanted < most ? wanted : most;
}

namespace {

// sums of the sets: 32 threads to a column, each every 32nd set in order, then theirs
__global__ void __launch_bounds__(1024) bn_sums_kernel(const float *part, int sets, int C, float *dpw, float *dsc, float *dw) {
  __shared__ float sm[32][33];
  float *out = blockIdx.y == 0 ? dpw : blockIdx.y == 1 ? dsc : dw;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < C) {
#pragma unroll 4
    for (int i = warp; i < sets; i += 32) s += part[((size_t)i * 3 + blockIdx.y) * C + c];
  }
  sm[warp][lane] = s;
  __syncthreads();
  s = sm[lane][warp];  // column warp
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + warp < C) out[blockIdx.x * 32 + warp] = s;
}

}  // namespace

void launch_bn_sums(const BnProblem &p, cudaStream_t s) {
  bn_sums_kernel<<<dim3((unsigned)((p.C + 31) / 32), 3), 1024, 0, s>>>(p.part, bn_blocks(p.rows, p.C), p.C, p.dpw, p.dsc, p.dw);
}

}  // namespace ssd
