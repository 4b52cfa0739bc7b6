// What the chunks of the gated delta rule need before the state is known: the rows' factors, N and P.
//
// A block takes a chunk and a head of q and k.  K K^T and Q K^T are made once and serve every state that shares the
// head.  N = (I + A diag(b))^-1 A column by column, a thread to a column, its 64 values in registers: once row m
// is final, b_m N_mj times column m of A leaves the rows below.
// Sums of log decays are whole numbers of 2^-32, so that differences between tokens are exact however much was forgotten
// before them; what is below -256 is taken as -256 (e^-256 is 0 in fp32).
#include "delta.h"
#include "simt_gemm.cuh"

namespace ssd {

namespace {

constexpr int kThreads = 256, kRowLd = kDrC + 4;
constexpr float kUnit = 4294967296.f, kLowest = -256.f;

template <typename T> __device__ __forceinline__ float load1(const T *p) { return to_f<T>(*p); }

struct PrepShared {
  float kk[kDrC][kRowLd], qk[kDrC][kRowLd];
  float at[kDrC][kRowLd];  // A transposed: column m as a row; before, the products' staging
  DrRows rows;
  float rk[kDrC], rq[kDrC];
  int nan_at;
};
static_assert(sizeof(float) * kGemmSmemFloats <= sizeof(float) * kDrC * kRowLd, "staging");

// G of one head by one warp, and everything of a row
template <typename T>
__device__ __forceinline__ void fill_rows(const DrProblem &p, PrepShared &sm, int h, int t0, int n, int lane) {
  const T *g = static_cast<const T *>(p.g), *b = static_cast<const T *>(p.b);
  long long x[2];
  float beta[2];
  unsigned nan_lanes[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * lane + e;
    const float v = i < n ? load1(g + (t0 + i) * p.gs + h) : 0.f;
    beta[e] = i < n ? load1(b + (t0 + i) * p.bs + h) : 0.f;
    x[e] = __float2ll_rn(fminf(fmaxf(v, kLowest), -kLowest) * kUnit);
    nan_lanes[e] = __ballot_sync(0xffffffffu, v != v);
  }
  x[1] += x[0];
  long long before = x[1];
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  const long long whole = __shfl_sync(0xffffffffu, before, 31);
  before -= x[1];
  // the first token whose log decay is not a number: nothing that passes it is
  int nan_at = kDrC;
  if (nan_lanes[0]) nan_at = min(nan_at, 2 * (__ffs(nan_lanes[0]) - 1));
  if (nan_lanes[1]) nan_at = min(nan_at, 2 * (__ffs(nan_lanes[1]) - 1) + 1);
  const float nan = __int_as_float(0x7fffffff);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * lane + e;
    const long long G = before + x[e];
    const float hi = __ll2float_rn(G), lo = __ll2float_rn(G - __float2ll_rn(hi));
    const float in = expf(hi * (1.f / kUnit)) + (i >= nan_at ? nan : 0.f);
    const float out = expf(__ll2float_rn(whole - G) * (1.f / kUnit)) + (nan_at < kDrC && i < n ? nan : 0.f);
    const bool live = i < n;
    sm.rows.ghi[i] = hi * (1.f / kUnit);
    sm.rows.glo[i] = lo * (1.f / kUnit);
    sm.rows.kin[i] = live ? in * sm.rk[i] : 0.f;
    sm.rows.kout[i] = live ? out * sm.rk[i] : 0.f;
    sm.rows.qin[i] = live ? in * sm.rq[i] * p.scale : 0.f;
    sm.rows.beta[i] = beta[e];
    sm.rows.rk[i] = live ? sm.rk[i] : 0.f;
    sm.rows.rq[i] = live ? sm.rq[i] : 0.f;
  }
  if (lane == 0) {
    const float gall = __ll2float_rn(whole) * (1.f / kUnit), em = expm1f(gall), hi = 1.f + em;
    sm.rows.all_hi = nan_at < kDrC ? nan : hi;
    // hi is 0 or tiny where em is near -1: the rest is then e^gall itself
    sm.rows.all_lo = nan_at < kDrC ? nan : gall < -0.5f ? expf(gall) - hi : em - (hi - 1.f);
    sm.rows.pad[0] = sm.rows.pad[1] = 0.f;
    sm.nan_at = nan_at;
  }
}

// a value as two bf16 terms, element (i, j) of their tiles in the 128-byte swizzle
__device__ __forceinline__ void store_terms(uint8_t *tile, int i, int j, float v) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(v);
  const uint32_t at = sm100::sw128_offset(i, j);
  *reinterpret_cast<__nv_bfloat16 *>(tile + at) = hi;
  *reinterpret_cast<__nv_bfloat16 *>(tile + kDrTile + at) = __float2bfloat16_rn(v - __bfloat162float(hi));
}

template <typename T, bool TC>
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
    if (tid < 32) fill_rows<T>(p, sm, h, t0, n, tid);
    __syncthreads();
    const size_t at = (size_t)slot * p.H + h;
    const float nan = __int_as_float(0x7fffffff);
    uint8_t *tiles = reinterpret_cast<uint8_t *>(p.N) + at * (4 * kDrTile);
    for (int e = tid; e < kDrC * kDrC; e += kThreads) {
      const int i = e >> 6, j = e & 63;
      float l = j <= i ? expf((sm.rows.ghi[i] - sm.rows.ghi[j]) + (sm.rows.glo[i] - sm.rows.glo[j])) : 0.f;
      if (j <= i && i >= sm.nan_at && j < sm.nan_at) l = nan;
      const float rk = sm.rows.rk[j];
      const float w = j <= i ? l * sm.qk[i][j] * (sm.rows.rq[i] * rk * p.scale) : 0.f;
      if (TC)
        store_terms(tiles + 2 * kDrTile, i, j, w);
      else
        p.P[at * (kDrC * kDrC) + e] = w;
      sm.at[j][i] = j < i ? l * sm.kk[i][j] * (sm.rows.rk[i] * rk) : 0.f;
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
      for (int i = 0; i < kDrC; ++i) {
        if (TC)
          store_terms(tiles, i, tid, x[i]);
        else
          p.N[at * (kDrC * kDrC) + i * kDrC + tid] = x[i];
      }
    }
  }
}

template <typename T, bool TC> void run_prep(const DrProblem &p, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(dr_prep_kernel<T, TC>), sizeof(PrepShared), allowed);
  dr_prep_kernel<T, TC><<<dim3((unsigned)p.slots, (unsigned)p.Hk), kThreads, sizeof(PrepShared), s>>>(p);
}

}  // namespace

template <typename T> void launch_dr_prep(const DrProblem &p, bool tc, cudaStream_t s) {
  if (sizeof(T) == 2 && tc)
    run_prep<__nv_bfloat16, true>(p, s);
  else
    run_prep<T, false>(p, s);
}

template void launch_dr_prep<float>(const DrProblem &, bool, cudaStream_t);
template void launch_dr_prep<__nv_bfloat16>(const DrProblem &, bool, cudaStream_t);

}  // namespace ssd
