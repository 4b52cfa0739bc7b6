// Kernels of the join of a block's output with the residual stream (block_norm.h), by type and direction in
// bn_*.cu.
//
// Bytes bound them: every tensor is read and written once, a row's values wait in its threads' registers from
// the first sum to the last store.  A row is a warp's (up to 1024 channels) or a block's.
#pragma once

#include <type_traits>

#include "block_norm.h"

namespace ssd {

namespace {

constexpr int kBnWarpRows = 8;  // rows of a block whose warps have a row each

template <int VEC, typename T> struct alignas(VEC * sizeof(T) > 16 ? 16 : VEC * sizeof(T)) BnVec {
  T v[VEC];
};

// the channel of a thread's e-th value
template <int VEC> __device__ __forceinline__ int bn_channel(int e, int tid, int team) {
  return ((e / VEC) * team + tid) * VEC + e % VEC;
}

template <int N, int VEC, typename T>
__device__ __forceinline__ void bn_load(T (&v)[N], const void *base, size_t at, int C, int tid, int team) {
  const T *p = static_cast<const T *>(base) + at;
#pragma unroll
  for (int e = 0; e < N; e += VEC) {
    const int c = bn_channel<VEC>(e, tid, team);
    if (c < C) {
      const BnVec<VEC, T> t = *reinterpret_cast<const BnVec<VEC, T> *>(p + c);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[e + j] = t.v[j];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[e + j] = from_f<T>(0.f);
    }
  }
}
template <int N, int VEC, typename T>
__device__ __forceinline__ void bn_store(void *base, size_t at, const float (&v)[N], int C, int tid, int team) {
  T *p = static_cast<T *>(base) + at;
#pragma unroll
  for (int e = 0; e < N; e += VEC) {
    const int c = bn_channel<VEC>(e, tid, team);
    if (c < C) {
      BnVec<VEC, T> t;
#pragma unroll
      for (int j = 0; j < VEC; ++j) t.v[j] = from_f<T>(v[e + j]);
      *reinterpret_cast<BnVec<VEC, T> *>(p + c) = t;
    }
  }
}
// a weight times the values, or nothing where there is none
template <int N, int VEC>
__device__ __forceinline__ void bn_weigh(float (&v)[N], const float *w, int C, int tid, int team) {
  if (!w) return;
#pragma unroll
  for (int e = 0; e < N; e += VEC) {
    const int c = bn_channel<VEC>(e, tid, team);
    if (c < C) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[e + j] *= __ldg(w + c + j);
    }
  }
}

// Sum over a row's threads, in a fixed order; every thread gets it.  `buf`: 32 floats that the last two sums did not use.
template <bool WARP> __device__ __forceinline__ float bn_sum(float v, float *buf) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (WARP) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = lane < warps ? buf[lane] : 0.f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float bn_silu(float z) { return z * sigmoid_f(z); }

template <typename T, typename R, int PER, int VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kBnWarpRows : 512) bn_forward_kernel(const BnProblem p) {
  constexpr int N = 8 * PER;
  __shared__ float sums[2][32];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, team = WARP ? 32 : blockDim.x;
  const int row = WARP ? blockIdx.x * kBnWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.rows) return;
  T x[N], z[N];
  R res[N];
  bn_load<N, VEC>(x, p.x, (size_t)row * p.xs, p.C, tid, team);
  if (p.gate) bn_load<N, VEC>(z, p.z, (size_t)row * p.zs, p.C, tid, team);
  if (p.res) bn_load<N, VEC>(res, p.res, (size_t)row * p.rs, p.C, tid, team);
  float h[N];
#pragma unroll
  for (int e = 0; e < N; ++e) h[e] = to_f<T>(x[e]);
  if (p.post) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) s = fmaf(h[e], h[e], s);
    const float r = 1.f / sqrtf(bn_sum<WARP>(s, sums[0]) / (float)p.C + p.eps);
    if (tid == 0 && p.rstd_post) p.rstd_post[row] = r;
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] *= r;
    bn_weigh<N, VEC>(h, p.pw, p.C, tid, team);
  }
  if (p.gate) {
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] *= bn_silu(to_f<T>(z[e]));
  }
  bn_weigh<N, VEC>(h, p.sc, p.C, tid, team);
  if (p.res) {
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] += to_f<R>(res[e]);
  }
  if (p.h) bn_store<N, VEC, R>(p.h, (size_t)row * p.hs, h, p.C, tid, team);
  if (p.pre) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) s = fmaf(h[e], h[e], s);
    const float r = 1.f / sqrtf(bn_sum<WARP>(s, sums[1]) / (float)p.C + p.eps);
    if (tid == 0 && p.rstd_pre) p.rstd_pre[row] = r;
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] *= r;
    bn_weigh<N, VEC>(h, p.w, p.C, tid, team);
    bn_store<N, VEC, T>(p.y, (size_t)row * p.ys, h, p.C, tid, team);
  }
}

// A block goes through rows blockIdx.x, + gridDim.x, ...; the parameters' sums stay in registers and go out once.
// Teams of a warp: the block's warps have partial sums of their own.
template <typename T, typename R, int PER, int VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kBnWarpRows : 512) bn_backward_kernel(const BnProblem p) {
  constexpr int N = 8 * PER;
  __shared__ float sums[4][32];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, team = WARP ? 32 : blockDim.x;
  const int first = WARP ? blockIdx.x * kBnWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  const int step = WARP ? gridDim.x * kBnWarpRows : gridDim.x;
  const float per_c = 1.f / (float)p.C;
  float dpw[N], dsc[N], dw[N];
#pragma unroll
  for (int e = 0; e < N; ++e) dpw[e] = dsc[e] = dw[e] = 0.f;
  const bool uses_x = p.post || p.gate || p.dsc;
  int turn = 0;
  for (int row = first; row < p.rows; row += step) {
    float d[N];
    {
      R dh[N];
      if (p.dh) bn_load<N, VEC>(dh, p.dh, (size_t)row * p.dhs, p.C, tid, team);
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = p.dh ? to_f<R>(dh[e]) : 0.f;
    }
    T x[N], z[N];
    if (uses_x) bn_load<N, VEC>(x, p.x, (size_t)row * p.xs, p.C, tid, team);
    if (p.gate) bn_load<N, VEC>(z, p.z, (size_t)row * p.zs, p.C, tid, team);
    if (p.pre && p.dy) {
      R h[N];
      T dy[N];
      bn_load<N, VEC>(h, p.h, (size_t)row * p.hs, p.C, tid, team);
      bn_load<N, VEC>(dy, p.dy, (size_t)row * p.dys, p.C, tid, team);
      const float r = __ldg(p.rstd_pre + row);
      float g[N], s = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] = to_f<T>(dy[e]);
#pragma unroll
      for (int e = 0; e < N; ++e) dw[e] = fmaf(g[e], to_f<R>(h[e]) * r, dw[e]);
      bn_weigh<N, VEC>(g, p.w, p.C, tid, team);
#pragma unroll
      for (int e = 0; e < N; ++e) s = fmaf(g[e], to_f<R>(h[e]), s);
      s = bn_sum<WARP>(s, sums[turn]) * per_c * r * r;
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = fmaf(r, g[e] - to_f<R>(h[e]) * s, d[e]);
    }
    if (p.dres) bn_store<N, VEC, R>(p.dres, (size_t)row * p.drs, d, p.C, tid, team);
    float u[N];  // the normed x, before its weight
    const float rp = p.post ? __ldg(p.rstd_post + row) : 1.f;
    if (uses_x) {
#pragma unroll
      for (int e = 0; e < N; ++e) u[e] = to_f<T>(x[e]) * rp;
    }
    if (p.gate || p.dsc) {
      float t[N];  // weighted
#pragma unroll
      for (int e = 0; e < N; ++e) t[e] = u[e];
      if (p.post) bn_weigh<N, VEC>(t, p.pw, p.C, tid, team);
      if (p.dsc) {
#pragma unroll
        for (int e = 0; e < N; ++e) dsc[e] = fmaf(d[e], p.gate ? t[e] * bn_silu(to_f<T>(z[e])) : t[e], dsc[e]);
      }
      bn_weigh<N, VEC>(d, p.sc, p.C, tid, team);
      if (p.gate) {
        float dz[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float zz = to_f<T>(z[e]), q = sigmoid_f(zz);
          dz[e] = d[e] * t[e] * (q * (1.f + zz * (1.f - q)));
          d[e] *= zz * q;
        }
        bn_store<N, VEC, T>(p.dz, (size_t)row * p.dzs, dz, p.C, tid, team);
      }
    } else {
      bn_weigh<N, VEC>(d, p.sc, p.C, tid, team);
    }
    if (p.post) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) dpw[e] = fmaf(d[e], u[e], dpw[e]);
      bn_weigh<N, VEC>(d, p.pw, p.C, tid, team);
#pragma unroll
      for (int e = 0; e < N; ++e) s = fmaf(d[e], u[e], s);
      s = bn_sum<WARP>(s, sums[turn + 1]) * per_c;
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = rp * (d[e] - u[e] * s);
    }
    bn_store<N, VEC, T>(p.dx, (size_t)row * p.dxs, d, p.C, tid, team);
    turn ^= 2;
  }
  const size_t set = WARP ? (size_t)first : blockIdx.x;
  auto put = [&](int which, const float *wanted, const float(&v)[N]) {
    if (!wanted) return;
    float *to = p.part + (set * 3 + which) * p.C;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int c = bn_channel<VEC>(e, tid, team);
      if (c < p.C) to[c] = v[e];
    }
  };
  put(0, p.dpw, dpw);
  put(1, p.dsc, dsc);
  put(2, p.dw, dw);
}

template <typename T, typename R, int PER, int VEC> void run_forward(const BnProblem &p, int threads, cudaStream_t s) {
  if (threads == 32)
    bn_forward_kernel<T, R, PER, VEC, true><<<(p.rows + kBnWarpRows - 1) / kBnWarpRows, 32 * kBnWarpRows, 0, s>>>(p);
  else
    bn_forward_kernel<T, R, PER, VEC, false><<<p.rows, threads, 0, s>>>(p);
}
template <typename T, typename R, int PER, int VEC> void run_backward(const BnProblem &p, int threads, cudaStream_t s) {
  const int sets = bn_blocks(p.rows, p.C);
  if (threads == 32)
    bn_backward_kernel<T, R, PER, VEC, true><<<sets / kBnWarpRows, 32 * kBnWarpRows, 0, s>>>(p);
  else
    bn_backward_kernel<T, R, PER, VEC, false><<<sets, threads, 0, s>>>(p);
}

template <typename T, typename R, int PER, class Run> void by_vec(int vec, const Run &run) {
  if (vec == 8)
    run(std::integral_constant<int, PER>(), std::integral_constant<int, 8>());
  else if (vec == 2)
    run(std::integral_constant<int, PER>(), std::integral_constant<int, 2>());
  else
    run(std::integral_constant<int, PER>(), std::integral_constant<int, 1>());
}
template <typename T, typename R, class Run> void by_team(int per, int vec, const Run &run) {
  if (per == 1)
    by_vec<T, R, 1>(vec, run);
  else if (per == 2)
    by_vec<T, R, 2>(vec, run);
  else
    by_vec<T, R, 4>(vec, run);
}

}  // namespace

template <typename T, typename R> void launch_bn_forward(const BnProblem &p, int vec, cudaStream_t s) {
  const BnTeam team = bn_team(p.C);
  by_team<T, R>(team.per, vec, [&](auto per, auto v) { run_forward<T, R, decltype(per)::value, decltype(v)::value>(p, team.threads, s); });
}
template <typename T, typename R> void launch_bn_backward(const BnProblem &p, int vec, cudaStream_t s) {
  const BnTeam team = bn_team(p.C);
  by_team<T, R>(team.per, vec, [&](auto per, auto v) { run_backward<T, R, decltype(per)::value, decltype(v)::value>(p, team.threads, s); });
}

}  // namespace ssd
