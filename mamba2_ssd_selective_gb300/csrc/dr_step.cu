// The gated delta rule, one token of each row against a cache of states:
//     S' = a S[slot],   d = beta (v - k S'),   S[slot] = S' + k^T d,   o = scale q S[slot]
// The state is read and written once, and that traffic is the bound; the layout is that of la_step.cu: a block takes
// 64 or 32 columns of one state, all of a thread's elements in registers.  Both sums over the state's rows
// (k S' and q S') are taken in one pass before the update, since q S[slot] = q S' + (q.k) d; the lengths of q and k
// and q.k ride along.
#include "delta.h"

namespace ssd {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <typename T> __device__ __forceinline__ float load1(const T *p) { return to_f<T>(*p); }

// SWEEPS sweeps of kThreads / (COLS / 4) rows cover the state's dk
template <typename T, int COLS, int SWEEPS>
__global__ void __launch_bounds__(kThreads) dr_step_kernel(DrProblem p, T *__restrict__ o, long long os,
                                                           float *__restrict__ states, int nslots,
                                                           const int *__restrict__ slot_idx) {
  constexpr int kLanes = COLS / 4, kRows = kThreads / kLanes;  // threads of a state row, state rows of a sweep
  __shared__ __align__(16) float part[2][kWarps][COLS];
  __shared__ float dots[kWarps][4];
  const int nz = (p.dv + COLS - 1) / COLS, r = blockIdx.x / nz, h = blockIdx.y, tid = threadIdx.x;
  const int z = blockIdx.x - r * nz, lc = tid % kLanes, c = z * COLS + 4 * lc, a0 = tid / kLanes;
  const bool col = c < p.dv;
  const int slot = slot_idx ? __ldg(slot_idx + r) : r;
  const bool live = slot >= 0 && slot < nslots;
  T *out = o + r * os + (size_t)h * p.dv;
  if (!live) {
    if (tid < COLS && z * COLS + tid < p.dv) out[z * COLS + tid] = from_f<T>(0.f);
    return;
  }
  float *st = states + ((size_t)slot * p.H + h) * ((size_t)p.dk * p.dv) + c;
  const T *q = static_cast<const T *>(p.q) + r * p.qs + (size_t)(h / p.group) * p.dk;
  const T *k = static_cast<const T *>(p.k) + r * p.ks + (size_t)(h / p.group) * p.dk;
  const T *v = static_cast<const T *>(p.v) + r * p.vs + (size_t)h * p.dv + c;
  float4 x[SWEEPS];
  float kv[SWEEPS], vv[4] = {0.f, 0.f, 0.f, 0.f};
  float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f}, kk = 0.f, qk = 0.f, qq = 0.f;
#pragma unroll
  for (int i = 0; i < SWEEPS; ++i) {
    const int a = a0 + kRows * i;
    x[i] = a < p.dk && col ? __ldcs(reinterpret_cast<const float4 *>(st + (size_t)a * p.dv)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float g = load1(static_cast<const T *>(p.g) + r * p.gs + h), beta = load1(static_cast<const T *>(p.b) + r * p.bs + h);
  if (col) {
#pragma unroll
    for (int e = 0; e < 4; ++e) vv[e] = load1(v + e);
  }
#pragma unroll
  for (int i = 0; i < SWEEPS; ++i) {
    const int a = a0 + kRows * i;
    const float qv = a < p.dk ? load1(q + a) : 0.f;
    kv[i] = a < p.dk ? load1(k + a) : 0.f;
    kk = fmaf(kv[i], kv[i], kk);
    qk = fmaf(kv[i], qv, qk);
    qq = fmaf(qv, qv, qq);
    sk[0] = fmaf(kv[i], x[i].x, sk[0]), sk[1] = fmaf(kv[i], x[i].y, sk[1]);
    sk[2] = fmaf(kv[i], x[i].z, sk[2]), sk[3] = fmaf(kv[i], x[i].w, sk[3]);
    sq[0] = fmaf(qv, x[i].x, sq[0]), sq[1] = fmaf(qv, x[i].y, sq[1]);
    sq[2] = fmaf(qv, x[i].z, sq[2]), sq[3] = fmaf(qv, x[i].w, sq[3]);
  }
#pragma unroll
  for (int s = kLanes; s < 32; s *= 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sk[j] += __shfl_xor_sync(0xffffffffu, sk[j], s);
      sq[j] += __shfl_xor_sync(0xffffffffu, sq[j], s);
    }
    kk += __shfl_xor_sync(0xffffffffu, kk, s);
    qk += __shfl_xor_sync(0xffffffffu, qk, s);
    qq += __shfl_xor_sync(0xffffffffu, qq, s);
  }
  if ((tid & 31) < kLanes) {
    *reinterpret_cast<float4 *>(&part[0][tid >> 5][4 * lc]) = make_float4(sk[0], sk[1], sk[2], sk[3]);
    *reinterpret_cast<float4 *>(&part[1][tid >> 5][4 * lc]) = make_float4(sq[0], sq[1], sq[2], sq[3]);
  }
  if ((tid & 31) == 0) {
    dots[tid >> 5][0] = kk;
    dots[tid >> 5][1] = qk;
    dots[tid >> 5][2] = qq;
  }
  __syncthreads();
  kk = qk = qq = 0.f;
  float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    kk += dots[w][0];
    qk += dots[w][1];
    qq += dots[w][2];
    const float4 y = *reinterpret_cast<const float4 *>(&part[0][w][4 * lc]);
    k4.x += y.x, k4.y += y.y, k4.z += y.z, k4.w += y.w;
  }
  const float rk = p.norm ? 1.f / sqrtf(kk + p.eps) : 1.f, rq = p.norm ? 1.f / sqrtf(qq + p.eps) : 1.f;
  const float2 lam = step_decay(g);
  auto low = [&](float y) { return fmaf(y, lam.x, y * lam.y); };
  const float d[4] = {beta * (vv[0] - rk * low(k4.x)), beta * (vv[1] - rk * low(k4.y)), beta * (vv[2] - rk * low(k4.z)),
                      beta * (vv[3] - rk * low(k4.w))};
  if (col) {
#pragma unroll
    for (int i = 0; i < SWEEPS; ++i) {
      const int a = a0 + kRows * i;
      if (a < p.dk) {
        const float u = rk * kv[i];
        x[i].x = fmaf(x[i].x, lam.x, fmaf(x[i].x, lam.y, u * d[0]));
        x[i].y = fmaf(x[i].y, lam.x, fmaf(x[i].y, lam.y, u * d[1]));
        x[i].z = fmaf(x[i].z, lam.x, fmaf(x[i].z, lam.y, u * d[2]));
        x[i].w = fmaf(x[i].w, lam.x, fmaf(x[i].w, lam.y, u * d[3]));
        __stcs(reinterpret_cast<float4 *>(st + (size_t)a * p.dv), x[i]);
      }
    }
  }
  if (tid < kLanes && col) {  // the first row's threads, which have their columns' d
    float4 q4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4 *>(&part[1][w][4 * lc]);
      q4.x += y.x, q4.y += y.y, q4.z += y.z, q4.w += y.w;
    }
    const float f = rk * qk, s = p.scale * rq;
    const float y[4] = {s * (low(q4.x) + f * d[0]), s * (low(q4.y) + f * d[1]), s * (low(q4.z) + f * d[2]), s * (low(q4.w) + f * d[3])};
#pragma unroll
    for (int e = 0; e < 4; ++e) out[c + e] = from_f<T>(y[e]);
  }
}

template <typename T, int COLS, int SWEEPS>
void run_step(const DrProblem &p, void *o, long long os, float *states, int nslots, const int *slot_idx, cudaStream_t s) {
  const dim3 grid((unsigned)p.nseq * ((p.dv + COLS - 1) / COLS), p.H);
  dr_step_kernel<T, COLS, SWEEPS><<<grid, kThreads, 0, s>>>(p, static_cast<T *>(o), os, states, nslots, slot_idx);
}

}  // namespace

template <typename T>
void launch_dr_step(const DrProblem &p, void *o, long long os, float *states, int nslots, const int *slot_idx, cudaStream_t s) {
  const bool wide = p.dv > 32 && p.dk <= 128 && (long long)p.nseq * p.H * ((p.dv + 63) / 64) >= 152;
  if (p.dk <= 64)
    wide ? run_step<T, 64, 4>(p, o, os, states, nslots, slot_idx, s) : run_step<T, 32, 2>(p, o, os, states, nslots, slot_idx, s);
  else if (p.dk <= 128)
    wide ? run_step<T, 64, 8>(p, o, os, states, nslots, slot_idx, s) : run_step<T, 32, 4>(p, o, os, states, nslots, slot_idx, s);
  else
    run_step<T, 32, 8>(p, o, os, states, nslots, slot_idx, s);
}

template void launch_dr_step<float>(const DrProblem &, void *, long long, float *, int, const int *, cudaStream_t);
template void launch_dr_step<__nv_bfloat16>(const DrProblem &, void *, long long, float *, int, const int *, cudaStream_t);

}  // namespace ssd
