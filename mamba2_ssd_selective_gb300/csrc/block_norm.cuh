// Kernels of the join of a block's output with the residual stream (block_norm.h), by type and direction in
// bn_*.cu.
//
// Bytes bound them: every tensor is read and written once, a row's values wait in its threads' registers from
// the first sum to the last store.  A row is a warp's (up to 256 channels) or a block's.  Blocks whose rows can be
// moved as whole 16-byte units go through many rows, with the next ones on their way into shared memory by bulk copies.
// All parts, bf16: 16384 x 4096 forward 128 us (5.2 TB/s), gradients of 8192 x 4096 with an fp32 stream 172 us, and 8 us
// for the parameters' sums (177 together, 4.2 TB/s).  What is left: backward has a block of 256 threads to an SM (255
// registers), whose sums over the row have nothing beside them.  From 4097 channels on it has 512 threads of 128
// registers, which spill: 4096 x 8192 take 368 us, 6554 x 5120 426.
#pragma once

#include <type_traits>

#include "block_norm.h"
#include "tc_pipe.cuh"

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

// A weight of a block that goes through many rows: in registers where HOLD says so (what bulk copies leave of the L1 cache
// does not hold them: 16384 x 4096 forward 299 us, read again for each row)
template <int N, int VEC, bool HOLD> struct BnWeight {
  const float *p;
  float v[HOLD ? N : 1];
  __device__ BnWeight(const float *w, int C, int tid, int team) : p(w) {
    if (!HOLD || !w) return;
#pragma unroll
    for (int e = 0; e < (HOLD ? N : 1); ++e) {
      const int c = bn_channel<VEC>(e, tid, team);
      v[e] = c < C ? __ldg(w + c) : 0.f;
    }
  }
  __device__ __forceinline__ void weigh(float (&x)[N], int C, int tid, int team) const {
    if (!HOLD) {
      bn_weigh<N, VEC>(x, p, C, tid, team);
    } else if (p) {
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] *= v[HOLD ? e : 0];
    }
  }
};

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

// sigmoid: of bf16 values on the fast intrinsics (relative error ~1e-6; infinities of the sum give 0)
template <typename T> __device__ __forceinline__ float bn_sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
template <> __device__ __forceinline__ float bn_sigmoid<float>(float z) { return sigmoid_f(z); }

// Where a block's rows come from: global memory, or (kRing) a ring of stages in shared memory that bulk copies fill.
enum { kWarp, kBlock, kRing };
struct BnTensor {
  const void *p;
  long long stride;
  int eb;  // bytes of an element
};
template <int MODE, int NT> struct BnRows {
  const BnTensor (&t)[NT];  // null where there is none
  uint8_t *ring;
  uint64_t *full;
  int rows, C, step, stages, stage_bytes;
  int next;  // the row that is copied next (thread 0)
  __device__ BnRows(const BnTensor (&tensors)[NT], uint8_t *smem, int rows_, int C_, int first, int step_, int stages_)
      : t(tensors), ring(smem + 64), full(reinterpret_cast<uint64_t *>(smem)), rows(rows_), C(C_), step(step_), stages(stages_), next(first) {
    stage_bytes = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) stage_bytes += t[i].p ? C * t[i].eb : 0;
    if (MODE != kRing) return;
    if (threadIdx.x == 0) {
      for (int s = 0; s < stages; ++s) sm100::mbar_init(&full[s], 1);
      sm100::fence_mbar_init();
    }
    __syncthreads();
    for (int s = 0; s < stages; ++s) fetch(s);
  }
  // the next row on its way into stage s, which every thread has read (a __syncthreads since)
  __device__ void fetch(int s) {
    if (MODE != kRing) return;
    if (threadIdx.x == 0 && next < rows) {
      sm100::mbar_expect_tx(&full[s], (uint32_t)stage_bytes);
      uint8_t *to = ring + (size_t)s * stage_bytes;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (t[i].p) {
          pipe::bulk_load(to, static_cast<const uint8_t *>(t[i].p) + (size_t)next * t[i].stride * t[i].eb, (uint32_t)(C * t[i].eb), &full[s]);
          to += C * t[i].eb;
        }
    }
    next += step;
  }
  // tensor `which` of a row, the it-th of the block
  template <int N, int VEC, typename X> __device__ void get(X (&v)[N], int which, int row, int it, int tid, int team) const {
    if (MODE == kRing) {
      const uint8_t *from = ring + (size_t)(it % stages) * stage_bytes;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (i < which && t[i].p) from += C * t[i].eb;
      bn_load<N, VEC>(v, from, 0, C, tid, team);
    } else {
      bn_load<N, VEC>(v, t[which].p, (size_t)row * t[which].stride, C, tid, team);
    }
  }
  __device__ void wait(int it) const {
    if (MODE == kRing) sm100::mbar_wait_drain(&full[it % stages], (it / stages) & 1);
  }
};

template <typename T, typename R, int PER, int VEC, int MODE>
__global__ void __launch_bounds__(MODE == kWarp ? 32 * kBnWarpRows : 512, 1) bn_forward_kernel(const BnProblem p, int stages) {
  constexpr int N = 8 * PER;
  constexpr bool WARP = MODE == kWarp;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sums[4][32];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, team = WARP ? 32 : blockDim.x;
  const int first = WARP ? blockIdx.x * kBnWarpRows + (threadIdx.x >> 5) : blockIdx.x, step = WARP ? gridDim.x * kBnWarpRows : gridDim.x;
  const float per_c = 1.f / (float)p.C;
  const BnTensor tensors[3] = {{p.x, p.xs, sizeof(T)}, {p.gate ? p.z : nullptr, p.zs, sizeof(T)}, {p.res, p.rs, sizeof(R)}};
  BnRows<MODE, 3> in(tensors, smem, p.rows, p.C, first, step, stages);
  constexpr bool kHold = MODE == kRing && N <= 16;
  const BnWeight<N, VEC, kHold> pw(p.pw, p.C, tid, team), sc(p.sc, p.C, tid, team), w(p.w, p.C, tid, team);
  int it = 0;
  for (int row = first; row < p.rows; row += step, ++it) {
    T x[N], z[N];
    R res[N];
    in.wait(it);
    in.template get<N, VEC>(x, 0, row, it, tid, team);
    if (p.gate) in.template get<N, VEC>(z, 1, row, it, tid, team);
    if (p.res) in.template get<N, VEC>(res, 2, row, it, tid, team);
    float h[N];
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = to_f<T>(x[e]);
    if (p.post) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) s = fmaf(h[e], h[e], s);
      const float r = 1.f / sqrtf(bn_sum<WARP>(s, sums[2 * (it & 1)]) * per_c + p.eps);
      if (tid == 0 && p.rstd_post) p.rstd_post[row] = r;
#pragma unroll
      for (int e = 0; e < N; ++e) h[e] *= r;
      pw.weigh(h, p.C, tid, team);
    } else if (MODE == kRing && !p.pre) {
      __syncthreads();
    }
    if (p.post || !p.pre) in.fetch(it % (MODE == kRing ? stages : 1));
    if (p.gate) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float g = to_f<T>(z[e]);
        h[e] *= g * bn_sigmoid<T>(g);
      }
    }
    sc.weigh(h, p.C, tid, team);
    if (p.res) {
#pragma unroll
      for (int e = 0; e < N; ++e) h[e] += to_f<R>(res[e]);
    }
    if (p.h) bn_store<N, VEC, R>(p.h, (size_t)row * p.hs, h, p.C, tid, team);
    if (p.pre) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) s = fmaf(h[e], h[e], s);
      const float r = 1.f / sqrtf(bn_sum<WARP>(s, sums[2 * (it & 1) + 1]) * per_c + p.eps);
      if (!p.post) in.fetch(it % (MODE == kRing ? stages : 1));
      if (tid == 0 && p.rstd_pre) p.rstd_pre[row] = r;
#pragma unroll
      for (int e = 0; e < N; ++e) h[e] *= r;
      w.weigh(h, p.C, tid, team);
      bn_store<N, VEC, T>(p.y, (size_t)row * p.ys, h, p.C, tid, team);
    }
  }
}

// The parameters' sums stay in registers and go out once: a set of partial sums for each block (teams of a warp: the
// block's warps add up in shared memory).
// As many blocks to an SM as bn_blocks() counts on: with the registers that the compiler takes otherwise (133 to 220) some
// of them waited, 8192 x 1000 64 us for 48, 16384 x 256 45 for 30.  Not where channels move one by one, whose addresses take
// up to 243: with 128 they spill, and 8192 x 1003 took 165 us for 98.
constexpr int bn_resident(int mode, int threads, int per, int vec) {
  return per > 1 || vec == 1 ? 1 : mode == kWarp || threads == 256 ? 2 : threads == 128 ? 4 : 1;
}
template <typename T, typename R, int PER, int VEC, int MODE, int THREADS>
__global__ void __launch_bounds__(MODE == kWarp ? 32 * kBnWarpRows : THREADS, bn_resident(MODE, THREADS, PER, VEC)) bn_backward_kernel(const BnProblem p, int stages) {
  constexpr int N = 8 * PER;
  constexpr bool WARP = MODE == kWarp;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sums[4][32];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, team = WARP ? 32 : blockDim.x;
  const int first = WARP ? blockIdx.x * kBnWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  const int step = WARP ? gridDim.x * kBnWarpRows : gridDim.x;
  const float per_c = 1.f / (float)p.C;
  float dpw[N], dsc[N], dw[N];
#pragma unroll
  for (int e = 0; e < N; ++e) dpw[e] = dsc[e] = dw[e] = 0.f;
  const bool uses_x = p.post || p.gate || p.dsc, pre = p.pre && p.dy;
  const BnTensor tensors[5] = {{uses_x ? p.x : nullptr, p.xs, sizeof(T)}, {p.gate ? p.z : nullptr, p.zs, sizeof(T)}, {pre ? p.dy : nullptr, p.dys, sizeof(T)},
                               {pre ? p.h : nullptr, p.hs, sizeof(R)}, {p.dh, p.dhs, sizeof(R)}};
  BnRows<MODE, 5> in(tensors, smem, p.rows, p.C, first, step, stages);
  constexpr bool kHold = MODE == kRing && N * THREADS <= 16 * 256;
  const BnWeight<N, VEC, kHold> pw(p.pw, p.C, tid, team), sc(p.sc, p.C, tid, team), w(p.w, p.C, tid, team);
  int it = 0;
  for (int row = first; row < p.rows; row += step, ++it) {
    float d[N];
    T x[N], z[N];
    in.wait(it);
    if (uses_x) in.template get<N, VEC>(x, 0, row, it, tid, team);
    if (p.gate) in.template get<N, VEC>(z, 1, row, it, tid, team);
    const float rp = p.post ? __ldg(p.rstd_post + row) : 1.f, r = pre ? __ldg(p.rstd_pre + row) : 1.f;
    {
      R dh[N];
      if (p.dh) in.template get<N, VEC>(dh, 4, row, it, tid, team);
      float g[N], s = 0.f;
      R h[N];
      if (pre) {
        T dy[N];
        in.template get<N, VEC>(dy, 2, row, it, tid, team);
        in.template get<N, VEC>(h, 3, row, it, tid, team);
#pragma unroll
        for (int e = 0; e < N; ++e) g[e] = to_f<T>(dy[e]);
#pragma unroll
        for (int e = 0; e < N; ++e) dw[e] = fmaf(g[e], to_f<R>(h[e]) * r, dw[e]);
        w.weigh(g, p.C, tid, team);
#pragma unroll
        for (int e = 0; e < N; ++e) s = fmaf(g[e], to_f<R>(h[e]), s);
        s = bn_sum<WARP>(s, sums[2 * (it & 1)]) * per_c * r * r;
      } else if (MODE == kRing) {
        __syncthreads();
      }
      in.fetch(it % (MODE == kRing ? stages : 1));
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = p.dh ? to_f<R>(dh[e]) : 0.f;
      if (pre) {
#pragma unroll
        for (int e = 0; e < N; ++e) d[e] = fmaf(r, g[e] - to_f<R>(h[e]) * s, d[e]);
      }
    }
    if (p.dres) bn_store<N, VEC, R>(p.dres, (size_t)row * p.drs, d, p.C, tid, team);
    float u[N];  // the normed x, before its weight
    if (uses_x) {
#pragma unroll
      for (int e = 0; e < N; ++e) u[e] = to_f<T>(x[e]) * rp;
    }
    if (p.gate || p.dsc) {
      float t[N];  // weighted
#pragma unroll
      for (int e = 0; e < N; ++e) t[e] = u[e];
      if (p.post) pw.weigh(t, p.C, tid, team);
      if (p.gate) {
        float s[N];
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = bn_sigmoid<T>(to_f<T>(z[e]));
        if (p.dsc) {
#pragma unroll
          for (int e = 0; e < N; ++e) dsc[e] = fmaf(d[e], t[e] * (to_f<T>(z[e]) * s[e]), dsc[e]);
        }
        sc.weigh(d, p.C, tid, team);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float zz = to_f<T>(z[e]);
          t[e] *= d[e] * (s[e] * fmaf(zz, 1.f - s[e], 1.f));
          d[e] *= zz * s[e];
        }
        bn_store<N, VEC, T>(p.dz, (size_t)row * p.dzs, t, p.C, tid, team);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) dsc[e] = fmaf(d[e], t[e], dsc[e]);
        sc.weigh(d, p.C, tid, team);
      }
    } else {
      sc.weigh(d, p.C, tid, team);
    }
    if (p.post) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) dpw[e] = fmaf(d[e], u[e], dpw[e]);
      pw.weigh(d, p.C, tid, team);
#pragma unroll
      for (int e = 0; e < N; ++e) s = fmaf(d[e], u[e], s);
      s = bn_sum<WARP>(s, sums[2 * (it & 1) + 1]) * per_c;
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = rp * (d[e] - u[e] * s);
    }
    bn_store<N, VEC, T>(p.dx, (size_t)row * p.dxs, d, p.C, tid, team);
  }
  auto put = [&](int which, const float *wanted, const float(&v)[N]) {
    if (!wanted) return;
    float *to = p.part + ((size_t)blockIdx.x * 3 + which) * p.C;
    if (WARP) {  // one warp after another
      float *acc = reinterpret_cast<float *>(smem);
      for (int w = 0; w < kBnWarpRows; ++w) {
        __syncthreads();
        if ((int)(threadIdx.x >> 5) == w) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const int c = bn_channel<VEC>(e, tid, team);
            if (c < p.C) acc[c] = w == 0 ? v[e] : acc[c] + v[e];
          }
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < p.C; c += blockDim.x) to[c] = acc[c];
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int c = bn_channel<VEC>(e, tid, team);
        if (c < p.C) to[c] = v[e];
      }
    }
  };
  put(0, p.dpw, dpw);
  put(1, p.dsc, dsc);
  put(2, p.dw, dw);
}

// Bytes of a row that a ring would move, and how many stages of them a block may have (fewer than 2: no ring)
template <typename T, typename R> int bn_stages(const BnProblem &p, bool backward, int blocks_per_sm, int &stage) {
  const bool pre = p.pre && p.dy;
  if (backward)
    stage = p.C * ((p.post || p.gate || p.dsc ? (int)sizeof(T) : 0) + (p.gate ? (int)sizeof(T) : 0) + (pre ? (int)(sizeof(T) + sizeof(R)) : 0) + (p.dh ? (int)sizeof(R) : 0));
  else
    stage = p.C * ((int)sizeof(T) * (p.gate ? 2 : 1) + (p.res ? (int)sizeof(R) : 0));
  const int most = stage ? (220 * 1024 / blocks_per_sm - 1024) / stage : 0;
  return most < 4 ? most : 4;
}

template <typename T, typename R, int PER, int VEC> void run_forward(const BnProblem &p, const BnTeam &team, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  int stage = 0;
  const int sms = device_sm_count();
  if constexpr (PER == 1) {
    if (team.threads == 32) {
      bn_forward_kernel<T, R, 1, VEC, kWarp><<<(p.rows + kBnWarpRows - 1) / kBnWarpRows, 32 * kBnWarpRows, 0, s>>>(p, 1);
      return;
    }
  }
  // two blocks of 256 threads to an SM, more of smaller ones; rows enough for some to be on their way
  const int per_sm = team.threads > 256 ? 1 : team.threads > 128 ? 2 : team.threads > 64 ? 4 : 8, grid = sms * per_sm;
  const int stages = VEC == 8 ? bn_stages<T, R>(p, false, per_sm, stage) : 0;
  if (VEC == 8 && stages >= 2 && p.rows >= 2 * grid) {
    allow_smem(reinterpret_cast<const void *>(bn_forward_kernel<T, R, PER, 8, kRing>), 220 * 1024, allowed);
    bn_forward_kernel<T, R, PER, 8, kRing><<<grid, team.threads, 64 + stages * stage, s>>>(p, stages);
  } else {
    bn_forward_kernel<T, R, PER, VEC, kBlock><<<p.rows, team.threads, 0, s>>>(p, 1);
  }
}
template <typename T, typename R, int PER, int VEC, int THREADS> void run_backward_blocks(const BnProblem &p, const BnTeam &team, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  const int sets = bn_blocks(p.rows, p.C, VEC);
  int stage = 0;
  const int stages = VEC == 8 ? bn_stages<T, R>(p, true, bn_blocks_per_sm(team, VEC), stage) : 0;
  if (VEC == 8 && stages >= 2 && p.rows >= 2 * sets) {
    allow_smem(reinterpret_cast<const void *>(bn_backward_kernel<T, R, PER, 8, kRing, THREADS>), 220 * 1024, allowed);
    bn_backward_kernel<T, R, PER, 8, kRing, THREADS><<<sets, team.threads, 64 + stages * stage, s>>>(p, stages);
  } else {
    bn_backward_kernel<T, R, PER, VEC, kBlock, THREADS><<<sets, team.threads, 0, s>>>(p, 1);
  }
}
template <typename T, typename R, int PER, int VEC> void run_backward(const BnProblem &p, const BnTeam &team, cudaStream_t s) {
  if constexpr (PER == 1) {  // at most 2048 channels
    if (team.threads == 32)
      bn_backward_kernel<T, R, 1, VEC, kWarp, 256><<<bn_blocks(p.rows, p.C, VEC), 32 * kBnWarpRows, p.C * 4, s>>>(p, 1);
    else if (VEC > 1 && team.threads <= 128)
      run_backward_blocks<T, R, 1, VEC == 1 ? 2 : VEC, 128>(p, team, s);
    else
      run_backward_blocks<T, R, 1, VEC, 256>(p, team, s);
  } else if (PER == 2 && team.threads <= 256) {
    run_backward_blocks<T, R, 2, VEC, 256>(p, team, s);
  } else {
    run_backward_blocks<T, R, PER, VEC, 512>(p, team, s);
  }
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
  by_team<T, R>(team.per, vec, [&](auto per, auto v) { run_forward<T, R, decltype(per)::value, decltype(v)::value>(p, team, s); });
}
template <typename T, typename R> void launch_bn_backward(const BnProblem &p, int vec, cudaStream_t s) {
  const BnTeam team = bn_team(p.C);
  by_team<T, R>(team.per, vec, [&](auto per, auto v) { run_backward<T, R, decltype(per)::value, decltype(v)::value>(p, team, s); });
}

}  // namespace ssd
