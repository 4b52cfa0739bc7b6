// The factors of a chunk's rows (DrRows in delta.h), made by one warp.
//
// Sums of log decays are whole numbers of 2^-32, so that differences between tokens are exact however much was forgotten
// before them; what is below -256 is taken as -256 (e^-256 is 0 in fp32).  They go to and from fp32 as a whole part and a
// signed rest of 32 bits each: conversions of 64 bits are slow here (with them a chunk's factors took 7400 cycles).
#pragma once

#include "delta.h"

namespace ssd {

namespace {

// What a head's log decays and strengths give, a warp's lane having rows 2 lane and 2 lane + 1
struct DrSums {
  float in[2], out[2], hi[2], lo[2], beta[2];  // e^G, e^(Gall - G), G as two values
  float all_hi, all_lo;                        // e^Gall, likewise
  int first_nan;                               // the first token whose log decay is not a number, or 64
};
struct DrGates {
  float g[2], b[2];
};
template <typename T> __device__ __forceinline__ DrGates dr_load_gates(const DrProblem &p, int h, int t0, int n, int lane) {
  const T *g = static_cast<const T *>(p.g) + (size_t)t0 * p.gs + h, *b = static_cast<const T *>(p.b) + (size_t)t0 * p.bs + h;
  DrGates v;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * lane + e;
    v.g[e] = i < n ? to_f<T>(g[i * p.gs]) : 0.f;
    v.b[e] = i < n ? to_f<T>(b[i * p.bs]) : 0.f;
  }
  return v;
}
// a sum as the nearest whole number and the rest
__device__ __forceinline__ void dr_parts(long long G, float &whole, float &rest) {
  const int I = (int)((G + 0x80000000LL) >> 32);
  whole = (float)I;
  rest = (float)(int)(G - ((long long)I << 32)) * (1.f / 4294967296.f);
}
__device__ __forceinline__ DrSums dr_sums(const DrGates &gates, int lane) {
  constexpr float kLowest = -256.f;
  const float *v = gates.g;
  DrSums s;
  s.beta[0] = gates.b[0], s.beta[1] = gates.b[1];
  long long x[2];
  s.first_nan = kDrC;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float c = fminf(fmaxf(v[e], kLowest), -kLowest), whole = rintf(c);
    x[e] = ((long long)(int)whole << 32) + __float2int_rn((c - whole) * 4294967296.f);
    const unsigned nans = __ballot_sync(0xffffffffu, v[e] != v[e]);
    if (nans) s.first_nan = min(s.first_nan, 2 * (__ffs(nans) - 1) + e);
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
  // nothing that passes a log decay that is not a number is one
  const float nan = __int_as_float(0x7fffffff);
  const bool bad = s.first_nan < kDrC;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * lane + e;
    const long long G = before + x[e];
    float hi, lo;
    dr_parts(whole - G, hi, lo);
    s.out[e] = bad ? nan : expf(hi + lo);
    dr_parts(G, s.hi[e], s.lo[e]);
    s.in[e] = i < s.first_nan ? expf(s.hi[e] + s.lo[e]) : nan;
  }
  float gw, gr;
  dr_parts(whole, gw, gr);
  const float gall = gw + gr, em = expm1f(gall), hi = 1.f + em;
  s.all_hi = bad ? nan : hi;
  // far from 1 the sum 1 + em has lost digits of e^gall, not of em
  s.all_lo = bad ? nan : gall < -0.5f ? expf(gall) - hi : em - (hi - 1.f);
  return s;
}
// The rows' factors, rk and rq being 1 / |k| and 1 / |q|; rows from n on get zeros.
__device__ __forceinline__ void dr_put_rows(DrRows &rows, const DrSums &s, const float *rk, const float *rq, float scale, int n,
                                            int lane) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * lane + e;
    const float k = i < n ? rk[i] : 0.f, q = i < n ? rq[i] : 0.f;
    rows.ghi[i] = s.hi[e];
    rows.glo[i] = s.lo[e];
    rows.kin[i] = i < n ? s.in[e] * k : 0.f;
    rows.kout[i] = i < n ? s.out[e] * k : 0.f;
    rows.qin[i] = i < n ? s.in[e] * q * scale : 0.f;
    rows.beta[i] = s.beta[e];
    rows.rk[i] = k;
    rows.rq[i] = q;
  }
  if (lane == 0) {
    rows.all_hi = s.all_hi;
    rows.all_lo = s.all_lo;
    rows.pad[0] = rows.pad[1] = 0.f;
  }
}

}  // namespace

}  // namespace ssd
