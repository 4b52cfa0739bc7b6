// The factors of a chunk's rows (DrRows in delta.h), made by one warp.
//
// Sums of log decays are whole numbers of 2^-32, so that differences between tokens are exact however much was forgotten
// before them; what is below -256 is taken as -256 (e^-256 is 0 in fp32).
#pragma once

#include "delta.h"

namespace ssd {

namespace {

// G of one head and everything of a row, by one warp; rk, rq: 1 / |k|, 1 / |q|; first_nan: the first token whose log decay is
// not a number, or 64
template <typename T>
__device__ __forceinline__ void dr_fill_rows(const DrProblem &p, DrRows &rows, const float *rk, const float *rq, int &first_nan,
                                             int h, int t0, int n, int lane) {
  constexpr float kUnit = 4294967296.f, kLowest = -256.f;
  const T *g = static_cast<const T *>(p.g), *b = static_cast<const T *>(p.b);
  long long x[2];
  float beta[2];
  unsigned nan_lanes[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * lane + e;
    const float v = i < n ? to_f<T>(g[(t0 + i) * p.gs + h]) : 0.f;
    beta[e] = i < n ? to_f<T>(b[(t0 + i) * p.bs + h]) : 0.f;
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
    rows.ghi[i] = hi * (1.f / kUnit);
    rows.glo[i] = lo * (1.f / kUnit);
    rows.kin[i] = live ? in * rk[i] : 0.f;
    rows.kout[i] = live ? out * rk[i] : 0.f;
    rows.qin[i] = live ? in * rq[i] * p.scale : 0.f;
    rows.beta[i] = beta[e];
    rows.rk[i] = live ? rk[i] : 0.f;
    rows.rq[i] = live ? rq[i] : 0.f;
  }
  if (lane == 0) {
    const float gall = __ll2float_rn(whole) * (1.f / kUnit), em = expm1f(gall), hi = 1.f + em;
    rows.all_hi = nan_at < kDrC ? nan : hi;
    // hi is 0 or tiny where em is near -1: the rest is then e^gall itself
    rows.all_lo = nan_at < kDrC ? nan : gall < -0.5f ? expf(gall) - hi : em - (hi - 1.f);
    rows.pad[0] = rows.pad[1] = 0.f;
    first_nan = nan_at;
  }
}

}  // namespace

}  // namespace ssd
