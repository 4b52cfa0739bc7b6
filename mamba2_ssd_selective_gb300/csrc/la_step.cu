// Linear attention with a decay for each head, one token of each row against a
// cache of states:
//     S[slot] = lam S[slot] + k^T v,   o = scale q S[slot]
// The state is read and written once, and that traffic is the bound.  A block
// of 256 threads takes 32 columns of one state: 8 threads span a row of 128
// bytes, 32 rows at a time, all of a thread's rows loaded before the first is
// used; the sum over rows goes through the warps' lanes, then shared memory, in
// a fixed order.  The columns are split over blocks so that a single row's few
// states still spread over many SMs.
#include "retention.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kCols = 32;
constexpr int kRows = kThreads / (kCols / 4);  // state rows of one sweep

template <typename T> __device__ __forceinline__ float load1(const T *p) { return to_f<T>(*p); }

// SWEEPS * 32 rows cover the state's dk
template <typename T, int SWEEPS>
__global__ void __launch_bounds__(kThreads) la_step_kernel(LaPass p, float *__restrict__ states, int nslots,
                                                           const int *__restrict__ slot_idx) {
  __shared__ float part[kThreads / 32][kCols];
  const int r = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int c = blockIdx.z * kCols + 4 * (tid & 7), a0 = tid >> 3;
  const bool col = c < p.dv;
  const int slot = slot_idx ? __ldg(slot_idx + r) : r;
  const bool live = slot >= 0 && slot < nslots;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (live && col) {
    float *st = states + ((size_t)slot * p.H + h) * ((size_t)p.dk * p.dv) + c;
    const T *q = static_cast<const T *>(p.q) + r * p.qs + (h / p.gq) * p.dk;
    const T *k = static_cast<const T *>(p.k) + r * p.ks + (h / p.gk) * p.dk;
    const T *v = static_cast<const T *>(p.v) + r * p.vs + (h / p.gv) * p.dv + c;
    float4 x[SWEEPS];
    float qv[SWEEPS], kv[SWEEPS];
#pragma unroll
    for (int i = 0; i < SWEEPS; ++i) {
      const int a = a0 + kRows * i;
      if (a < p.dk) {
        x[i] = *reinterpret_cast<const float4 *>(st + (size_t)a * p.dv);
        qv[i] = load1(q + a);
        kv[i] = load1(k + a);
      }
    }
    const float vv[4] = {load1(v), load1(v + 1), load1(v + 2), load1(v + 3)};
    const float lam = expf(__ldg(p.g + h));
#pragma unroll
    for (int i = 0; i < SWEEPS; ++i) {
      const int a = a0 + kRows * i;
      if (a < p.dk) {
        x[i].x = fmaf(lam, x[i].x, kv[i] * vv[0]);
        x[i].y = fmaf(lam, x[i].y, kv[i] * vv[1]);
        x[i].z = fmaf(lam, x[i].z, kv[i] * vv[2]);
        x[i].w = fmaf(lam, x[i].w, kv[i] * vv[3]);
        *reinterpret_cast<float4 *>(st + (size_t)a * p.dv) = x[i];
        acc[0] = fmaf(qv[i], x[i].x, acc[0]);
        acc[1] = fmaf(qv[i], x[i].y, acc[1]);
        acc[2] = fmaf(qv[i], x[i].z, acc[2]);
        acc[3] = fmaf(qv[i], x[i].w, acc[3]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 8);
    acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 16);
  }
  if ((tid & 31) < 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[tid >> 5][4 * (tid & 7) + j] = acc[j];
  __syncthreads();
  if (tid < kCols && blockIdx.z * kCols + tid < p.dv) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) o += part[w][tid];
    static_cast<T *>(p.o)[r * p.os + (long long)h * p.dv + blockIdx.z * kCols + tid] = from_f<T>(o * p.o_scale);
  }
}

}  // namespace

template <typename T>
void launch_la_step(const LaPass &p, int rows, float *states, int nslots, const int *slot_idx, cudaStream_t s) {
  const dim3 grid(rows, p.H, (p.dv + kCols - 1) / kCols);
  if (p.dk <= 2 * kRows)
    la_step_kernel<T, 2><<<grid, kThreads, 0, s>>>(p, states, nslots, slot_idx);
  else if (p.dk <= 4 * kRows)
    la_step_kernel<T, 4><<<grid, kThreads, 0, s>>>(p, states, nslots, slot_idx);
  else
    la_step_kernel<T, 8><<<grid, kThreads, 0, s>>>(p, states, nslots, slot_idx);
}

template void launch_la_step<float>(const LaPass &, int, float *, int, const int *, cudaStream_t);
template void launch_la_step<__nv_bfloat16>(const LaPass &, int, float *, int, const int *, cudaStream_t);

}  // namespace ssd
