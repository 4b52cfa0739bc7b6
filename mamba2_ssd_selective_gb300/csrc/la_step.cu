// Linear attention with a decay for each head, one token of each row against a
// cache of states:
//     S[slot] = lam S[slot] + k^T v,   o = scale q S[slot]
// The state is read and written once, and that traffic is the bound.  A block
// of 256 threads takes 64 or 32 columns of one state, all of a thread's elements
// loaded before the first is used; the sum over rows goes through the warps'
// lanes, then shared memory, in a fixed order.  Blocks of one state are
// neighbours in the grid, so that its memory is read as one piece (with rows of the cache next to one
// another instead: 209 us where it was 199).  By the time of a row's next token its state has left the L2 cache in
// any case, so it takes no place of others there (ldcs, stcs).  256 rows, 32 heads of 128 x 128 (1.07 GB): 163 us
// (6.6 TB/s), without the hints 173 us; 64 rows, 8 heads of 256 x 256: 48 us and 51 us; 300 rows, 32 heads of 24 x 128: 67 us
// and 69 us; a state of 67 MB stepped again at once, from the cache: 19 us and 15 us.
// Before the hints 64 columns took 178 us for the 256 rows, 32 columns 202 us, 128 columns 223 us, which leave a thread
// 16 loads and the SM few warps; dk of 256 takes 32 columns for the same reason (211 us against 509).  Where 64
// columns leave SMs without a block, 32 spread a single row's few states over more of them (16 heads: 8.3 us against 9.0).
#include "retention.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;

template <typename T> __device__ __forceinline__ float load1(const T *p) { return to_f<T>(*p); }

template <int COLS> constexpr int kRows = kThreads / (COLS / 4);  // state rows of one sweep

// SWEEPS sweeps cover the state's dk
template <typename T, int COLS, int SWEEPS>
__global__ void __launch_bounds__(kThreads) la_step_kernel(LaPass p, float *__restrict__ states, int nslots,
                                                           const int *__restrict__ slot_idx) {
  constexpr int kLanes = COLS / 4;  // threads of a state row
  __shared__ float part[kThreads / 32][COLS];
  const int nz = (p.dv + COLS - 1) / COLS, r = blockIdx.x / nz, h = blockIdx.y, tid = threadIdx.x;
  const int z = blockIdx.x - r * nz, c = z * COLS + 4 * (tid % kLanes), a0 = tid / kLanes;
  const bool col = c < p.dv;
  const float g = __ldg(p.g + h);
  const int slot = slot_idx ? __ldg(slot_idx + r) : r;
  const bool live = slot >= 0 && slot < nslots;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  float4 x[SWEEPS];
  float qv[SWEEPS], kv[SWEEPS], vv[4];
  if (live && col) {
    float *st = states + ((size_t)slot * p.H + h) * ((size_t)p.dk * p.dv) + c;
    const T *q = static_cast<const T *>(p.q) + r * p.qs + (h / p.gq) * p.dk;
    const T *k = static_cast<const T *>(p.k) + r * p.ks + (h / p.gk) * p.dk;
    const T *v = static_cast<const T *>(p.v) + r * p.vs + (h / p.gv) * p.dv + c;
#pragma unroll
    for (int i = 0; i < SWEEPS; ++i) {
      const int a = a0 + kRows<COLS> * i;
      if (a < p.dk) {
        x[i] = __ldcs(reinterpret_cast<const float4 *>(st + (size_t)a * p.dv));
        qv[i] = load1(q + a);
        kv[i] = load1(k + a);
      }
    }
    vv[0] = load1(v), vv[1] = load1(v + 1), vv[2] = load1(v + 2), vv[3] = load1(v + 3);
  }
  const float2 lam = step_decay(g);
  if (live && col) {
    float *st = states + ((size_t)slot * p.H + h) * ((size_t)p.dk * p.dv) + c;
#pragma unroll
    for (int i = 0; i < SWEEPS; ++i) {
      const int a = a0 + kRows<COLS> * i;
      if (a < p.dk) {
        x[i].x = fmaf(x[i].x, lam.x, fmaf(x[i].x, lam.y, kv[i] * vv[0]));
        x[i].y = fmaf(x[i].y, lam.x, fmaf(x[i].y, lam.y, kv[i] * vv[1]));
        x[i].z = fmaf(x[i].z, lam.x, fmaf(x[i].z, lam.y, kv[i] * vv[2]));
        x[i].w = fmaf(x[i].w, lam.x, fmaf(x[i].w, lam.y, kv[i] * vv[3]));
        __stcs(reinterpret_cast<float4 *>(st + (size_t)a * p.dv), x[i]);
        acc[0] = fmaf(qv[i], x[i].x, acc[0]);
        acc[1] = fmaf(qv[i], x[i].y, acc[1]);
        acc[2] = fmaf(qv[i], x[i].z, acc[2]);
        acc[3] = fmaf(qv[i], x[i].w, acc[3]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int o = kLanes; o < 32; o *= 2) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
  if ((tid & 31) < kLanes)
    *reinterpret_cast<float4 *>(&part[tid >> 5][4 * (tid % kLanes)]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (tid < COLS && z * COLS + tid < p.dv) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) o += part[w][tid];
    static_cast<T *>(p.o)[r * p.os + (long long)h * p.dv + z * COLS + tid] = from_f<T>(o * p.o_scale);
  }
}

template <typename T, int COLS, int SWEEPS>
void run_step(const LaPass &p, int rows, float *states, int nslots, const int *slot_idx, cudaStream_t s) {
  static_assert(SWEEPS <= 8, "registers");
  const dim3 grid((unsigned)rows * ((p.dv + COLS - 1) / COLS), p.H);
  la_step_kernel<T, COLS, SWEEPS><<<grid, kThreads, 0, s>>>(p, states, nslots, slot_idx);
}

}  // namespace

template <typename T>
void launch_la_step(const LaPass &p, int rows, float *states, int nslots, const int *slot_idx, cudaStream_t s) {
  const bool wide = p.dv > 32 && p.dk <= 128 && (long long)rows * p.H * ((p.dv + 63) / 64) >= 152;
  if (p.dk <= 64)
    wide ? run_step<T, 64, 4>(p, rows, states, nslots, slot_idx, s) : run_step<T, 32, 2>(p, rows, states, nslots, slot_idx, s);
  else if (p.dk <= 128)
    wide ? run_step<T, 64, 8>(p, rows, states, nslots, slot_idx, s) : run_step<T, 32, 4>(p, rows, states, nslots, slot_idx, s);
  else
    run_step<T, 32, 8>(p, rows, states, nslots, slot_idx, s);
}

template void launch_la_step<float>(const LaPass &, int, float *, int, const int *, cudaStream_t);
template void launch_la_step<__nv_bfloat16>(const LaPass &, int, float *, int, const int *, cudaStream_t);

}  // namespace ssd
