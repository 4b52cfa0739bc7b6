// What the chunks of the gated delta rule need before the state is known: the rows' factors, N and P.
//
// A block takes a chunk and a head of q and k.  K K^T and Q K^T are made once and serve every state that shares the
// head.  N = (I + A diag(b))^-1 A column by column, a thread to a column, its 64 values in registers: once row m
// is final, b_m N_mj times column m of A leaves the rows below.
// The tensor-core chains have dr_prep_tc.cu.
#include "delta.h"
#include "dr_rows.cuh"
#include "simt_gemm.cuh"

namespace ssd {

namespace {

constexpr int kThreads = 256, kRowLd = kDrC + 4;

template <typename T> __device__ __forceinline__ float load1(const T *p) { return to_f<T>(*p); }

struct PrepShared {
  float kk[kDrC][kRowLd], qk[kDrC][kRowLd];
  float at[kDrC][kRowLd];  // A transposed: column m as a row; before, the products' staging
  DrRows rows;
  float rk[kDrC], rq[kDrC];
  int nan_at;
};
static_assert(sizeof(float) * kGemmSmemFloats <= sizeof(float) * kDrC * kRowLd, "staging");

template <typename T>
__global__ void __launch_bounds__(kThreads) dr_prep_kernel(DrProblem p) {
  extern __shared__ __align__(16) uint8_t raw[];
  PrepShared &sm = *reinterpret_cast<PrepShared *>(raw);
  const int slot = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x, tm = tid >> 4, tn = tid & 15;
  int t0, n;
  if (slot == 0 && hk == 0 && tid == 0) *p.status = 0;
  dr_chunk(p, slot, t0, n);
  if (n == 0) return;
  const T *q = static_cast<const T *>(p.q) + (size_t)t0 * p.qs + (size_t)hk * p.dk;
  const T *k = static_cast<const T *>(p.k) + (size_t)t0 * p.ks + (size_t)hk * p.dk;
  float *stage = &sm.at[0][0];
  auto kr = [&](int i, int c) { return load1(k + i * p.ks + c); };
  auto kc = [&](int c, int i) { return load1(k + i * p.ks + c); };
  auto qr = [&](int i, int c) { return load1(q + i * p.qs + c); };
  float acc[4][4];
  zero_acc(acc);
  gemm_tile<true, false>(acc, 0, n, 0, n, 0, p.dk, kr, kc, stage);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sm.kk[tm * 4 + i][tn * 4 + j] = acc[i][j];
  zero_acc(acc);
  gemm_tile<true, false>(acc, 0, n, 0, n, 0, p.dk, qr, kc, stage);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sm.qk[tm * 4 + i][tn * 4 + j] = acc[i][j];
  __syncthreads();
  if (tid < kDrC) {
    sm.rk[tid] = p.norm ? 1.f / sqrtf(sm.kk[tid][tid] + p.eps) : 1.f;
    float qq = 0.f;
    if (p.norm && tid < n)
      for (int c = 0; c < p.dk; ++c) qq = fmaf(qr(tid, c), qr(tid, c), qq);
    sm.rq[tid] = p.norm ? 1.f / sqrtf(qq + p.eps) : 1.f;
  }
  for (int h = hk * p.group; h < (hk + 1) * p.group; ++h) {
    __syncthreads();
    if (tid < 32) {
      const DrSums sums = dr_sums(dr_load_gates<T>(p, h, t0, n, tid), tid);
      dr_put_rows(sm.rows, sums, sm.rk, sm.rq, p.scale, n, tid);
      if (tid == 0) sm.nan_at = sums.first_nan;
    }
    __syncthreads();
    const size_t at = (size_t)slot * p.H + h;
    const float nan = __int_as_float(0x7fffffff);
    for (int e = tid; e < kDrC * kDrC; e += kThreads) {
      const int i = e >> 6, j = e & 63;
      float l = j <= i ? expf((sm.rows.ghi[i] - sm.rows.ghi[j]) + (sm.rows.glo[i] - sm.rows.glo[j])) : 0.f;
      if (j <= i && i >= sm.nan_at && j < sm.nan_at) l = nan;
      const float rk = sm.rows.rk[j];
      p.P[at * (kDrC * kDrC) + e] = j <= i ? l * sm.qk[i][j] * (sm.rows.rq[i] * rk * p.scale) : 0.f;
      const float a = j < i ? l * sm.kk[i][j] * (sm.rows.rk[i] * rk) : 0.f;
      sm.at[j][i] = a;
      if (p.A) p.A[at * (kDrC * kDrC) + e] = a;
    }
    const uint32_t *from = reinterpret_cast<const uint32_t *>(&sm.rows);
    uint32_t *to = reinterpret_cast<uint32_t *>(p.rows + at);
    for (int e = tid; e < (int)(sizeof(DrRows) / 4); e += kThreads) to[e] = from[e];
    __syncthreads();
    if (tid < kDrC) {  // column tid of N
      float x[kDrC];
#pragma unroll
      for (int i = 0; i < kDrC; i += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(&sm.at[tid][i]);
        x[i] = a.x, x[i + 1] = a.y, x[i + 2] = a.z, x[i + 3] = a.w;
      }
#pragma unroll
      for (int m = 1; m < kDrC - 1; ++m) {
        const float f = -sm.rows.beta[m] * x[m];
#pragma unroll
        for (int i = (m + 1) & ~3; i < kDrC; i += 4) {
          const float4 a = *reinterpret_cast<const float4 *>(&sm.at[m][i]);  // zeros up to row m
          x[i] = fmaf(f, a.x, x[i]);
          x[i + 1] = fmaf(f, a.y, x[i + 1]);
          x[i + 2] = fmaf(f, a.z, x[i + 2]);
          x[i + 3] = fmaf(f, a.w, x[i + 3]);
        }
      }
#pragma unroll
      for (int i = 0; i < kDrC; ++i) p.N[at * (kDrC * kDrC) + i * kDrC + tid] = x[i];
    }
  }
}

}  // namespace

template <typename T> void launch_dr_prep(const DrProblem &p, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(dr_prep_kernel<T>), sizeof(PrepShared), allowed);
  dr_prep_kernel<T><<<dim3((unsigned)p.slots, (unsigned)p.Hk), kThreads, sizeof(PrepShared), s>>>(p);
}

template void launch_dr_prep<float>(const DrProblem &, cudaStream_t);
template void launch_dr_prep<__nv_bfloat16>(const DrProblem &, cudaStream_t);

}  // namespace ssd
