// The join of a block's output with the residual stream: how a row is spread over threads, and the parameters' sums.
#include "block_norm.h"

namespace ssd {

// What a row costs whatever its length is shared by 16 channels a thread where it is long (gradients of 8192 x 4096: 182 us
// with 8), and rows of more than 256 channels are a block's (gradients of 16384 x 512: 107 us with a warp of 16 channels a
// thread, 46 with two warps).
BnTeam bn_team(int C) {
  const int units = (C + 7) / 8;
  if (units <= 32) return {32, 1};
  auto warps = [](int n) { return (n + 31) / 32 * 32; };
  if (units <= 256) return {warps(units), 1};
  if (units <= 1024) return {warps((units + 1) / 2), 2};
  return {warps((units + 3) / 4), 4};
}

// as registers allow: 128 a thread with 8 channels, 255 with 16, or with 8 that move one by one (bn_resident)
int bn_blocks_per_sm(const BnTeam &t, int vec) {
  const int most = t.threads > 256 || t.per > 1 ? 1 : t.threads > 128 ? 2 : t.threads > 64 ? 4 : 8;
  return vec == 1 && most > 1 ? most / 2 : most;
}

int bn_blocks(int rows, int C, int vec) {
  const BnTeam t = bn_team(C);
  // (a workspace's size may be asked for where there is no GPU: the SMs are not asked)
  const int most = 152 * (t.threads == 32 ? 2 : bn_blocks_per_sm(t, vec)), wanted = t.threads == 32 ? (rows + 7) / 8 : rows;
  return wanted < most ? wanted : most;
}

namespace {

// Sums of the sets: a block has COLS columns, 512 / COLS threads to each, which take a set each in turn; then theirs.
template <int COLS>
__global__ void __launch_bounds__(512) bn_sums_kernel(const float *part, int sets, int C, float *dpw, float *dsc, float *dw) {
  constexpr int kLanes = 512 / COLS;
  __shared__ float sm[kLanes][COLS + 1];
  float *out = blockIdx.y == 0 ? dpw : blockIdx.y == 1 ? dsc : dw;
  if (!out) return;
  const int first = blockIdx.x * COLS, col = threadIdx.x % COLS, at = threadIdx.x / COLS;
  float s = 0.f;
  if (first + col < C) {
    const float *from = part + (size_t)blockIdx.y * C + first + col;
    for (int i = at; i < sets; i += 10 * kLanes) {  // ten at once
      float v[10];
#pragma unroll
      for (int j = 0; j < 10; ++j) v[j] = i + j * kLanes < sets ? from[(size_t)(i + j * kLanes) * 3 * C] : 0.f;
#pragma unroll
      for (int j = 0; j < 10; ++j) s += v[j];
    }
  }
  sm[at][col] = s;
  __syncthreads();
  const int lane = threadIdx.x % kLanes, mine = threadIdx.x / kLanes;
  s = sm[lane][mine];
#pragma unroll
  for (int o = kLanes / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && first + mine < C) out[first + mine] = s;
}

}  // namespace

// wide columns where they are blocks enough
void launch_bn_sums(const BnProblem &p, int vec, cudaStream_t s) {
  const int sets = bn_blocks(p.rows, p.C, vec);
  if (p.C > 2048)
    bn_sums_kernel<32><<<dim3((unsigned)((p.C + 31) / 32), 3), 512, 0, s>>>(p.part, sets, p.C, p.dpw, p.dsc, p.dw);
  else
    bn_sums_kernel<16><<<dim3((unsigned)((p.C + 15) / 16), 3), 512, 0, s>>>(p.part, sets, p.C, p.dpw, p.dsc, p.dw);
}

}  // namespace ssd
