// Group norm with an activation, channels last.  Per sample and group, over its
// m rows and cg channels (M = m cg values):
//     xhat = (x - mean) rstd,  u = xhat w + b,  y = u | u sigmoid(u) | u z sigmoid(z)
// and backwards, with du the gradient of u:
//     dx = rstd (du w - A / M - xhat B / M),  A = sum du w,  B = sum du w xhat
//     dw = sum du xhat,  db = sum du,  dz = dy u silu'(z)
// Memory traffic bounds all of it.  A thread owns W consecutive channels (16 bytes
// of bf16) of every RP-th row of a group's slab, so that its channels, and its
// part of dw and db, stay in registers.
//
// A group that fits the registers of its team of NT threads (a part of a warp, a
// warp, or a block) is read once: its mean, then its squared deviations, are
// summed from registers.  With one row to a sample, a team is the narrowest
// part of a warp that spans the group.  A larger group is cut into tiles of
// rows, a block each.  Up to eight tiles are a cluster, whose blocks keep their
// tile in registers while they exchange its mean and squared deviations (or its
// part of A and B) through distributed shared memory.  Beyond that a first kernel
// writes what a tile gives, and dz, and a second one joins the tiles, in order,
// and reads its own again, from L2 where the tensor fits it.
// dw and db are sums of per-block partials in a fixed order.
//
// Measured (kernel times): 32768 rows of 32 groups of 128 channels with a gate, bf16 (805 MB): 132 us, 6.1 TB/s;
// the backward pass of 16384 rows (671 MB): 116 us and 8 us for the parameters' sums.  Both are near HBM's rate
// once enough loads are in flight (the next samples' values in registers instead of shared memory: 141 us
// and 135 us).  Groups of a cluster are bound by instructions and the latency of their phases, not by memory (DRAM
// 15% of its rate): 6 samples of 4099 rows of 32 groups of 10 channels, fp32 (63 MB): 27 us (two kernels: 37 us);
// the backward pass of 8 samples of 2048 rows of 32 groups of 16, bf16 (50 MB): 31 us and 6 us for the
// parameters' sums (two kernels: 44 us).  Clusters that stay and copy their next group's tile ahead took 42 us and
// 35 us: the GPU holds fewer of them, and 192 or 256 groups do not fill their rounds.
#pragma once

#include <type_traits>

#include <cooperative_groups.h>

#include "group_norm.h"
#include "sm100.cuh"

namespace ssd {
namespace gn {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- vectors of W channels
template <int W>
__device__ __forceinline__ void load_vec(const __nv_bfloat16 *p, float (&v)[W]) {
  if constexpr (W == 8) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else if constexpr (W == 2) {
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(p));
    v[0] = __uint_as_float(u << 16);
    v[1] = __uint_as_float(u & 0xffff0000u);
  } else {
    v[0] = __bfloat162float(*p);
  }
}
template <int W>
__device__ __forceinline__ void load_vec(const float *p, float (&v)[W]) {
  if constexpr (W == 8) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(p + i));
      v[i] = a.x;
      v[i + 1] = a.y;
      v[i + 2] = a.z;
      v[i + 3] = a.w;
    }
  } else if constexpr (W == 2) {
    const float2 a = __ldg(reinterpret_cast<const float2 *>(p));
    v[0] = a.x;
    v[1] = a.y;
  } else {
    v[0] = __ldg(p);
  }
}
// W channels as they lie in memory: half the registers for bf16
template <typename T, int W>
struct Raw {
  float f[W];
  __device__ __forceinline__ void load(const T *p) { load_vec<W>(p, f); }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < W; ++e) f[e] = 0.f;
  }
  __device__ __forceinline__ void get(float (&v)[W]) const {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = f[e];
  }
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = __ldg(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <int W>
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float (&v)[W]) {
  if constexpr (W == 8) {
    uint4 u;
    uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = u;
  } else if constexpr (W == 2) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[1]);
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}
template <int W>
__device__ __forceinline__ void store_vec(float *p, const float (&v)[W]) {
  if constexpr (W == 8) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else if constexpr (W == 2) {
    *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  } else {
    p[0] = v[0];
  }
}
// ---------------------------------------------------------------- arithmetic on W channels
// Eight channels go two to an instruction (packed fp32): once enough loads are in
// flight, instructions bound these kernels before memory does.
template <int W>
struct Vec {
  static constexpr int kPairs = (W + 1) / 2;
  uint64_t q[kPairs];
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ explicit Vec(float c) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) q[i] = sm100::pk2(c, c);
  }
  __device__ __forceinline__ explicit Vec(const float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) q[i] = sm100::pk2(v[2 * i], W == 1 ? 0.f : v[2 * i + (W > 1)]);
  }
  __device__ __forceinline__ void get(float (&v)[W]) const {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float a, b;
      sm100::upk2(q[i], a, b);
      v[2 * i] = a;
      if (W > 1) v[2 * i + (W > 1)] = b;
    }
  }
  __device__ __forceinline__ float sum() const {
    uint64_t t = q[0];
#pragma unroll
    for (int i = 1; i < kPairs; ++i) t = sm100::add2(t, q[i]);
    float a, b;
    sm100::upk2(t, a, b);
    return W == 1 ? a : a + b;
  }
};
template <int W> __device__ __forceinline__ Vec<W> operator+(const Vec<W> &a, const Vec<W> &b) {
  Vec<W> r;
#pragma unroll
  for (int i = 0; i < Vec<W>::kPairs; ++i) r.q[i] = sm100::add2(a.q[i], b.q[i]);
  return r;
}
template <int W> __device__ __forceinline__ Vec<W> operator*(const Vec<W> &a, const Vec<W> &b) {
  Vec<W> r;
#pragma unroll
  for (int i = 0; i < Vec<W>::kPairs; ++i) r.q[i] = sm100::mul2(a.q[i], b.q[i]);
  return r;
}
template <int W> __device__ __forceinline__ Vec<W> fma(const Vec<W> &a, const Vec<W> &b, const Vec<W> &c) {
  Vec<W> r;
#pragma unroll
  for (int i = 0; i < Vec<W>::kPairs; ++i) r.q[i] = sm100::fma2(a.q[i], b.q[i], c.q[i]);
  return r;
}
// 1 / (1 + e^-v) on the special-function unit: 2^x and 1 / x, each to about 2^-22
template <int W> __device__ __forceinline__ Vec<W> sigmoid(const Vec<W> &v) {
  float t[W];
  (v * Vec<W>(-1.44269504f)).get(t);
#pragma unroll
  for (int e = 0; e < W; ++e) t[e] = sm100::ex2_approx(t[e]);
  (Vec<W>(t) + Vec<W>(1.f)).get(t);
#pragma unroll
  for (int e = 0; e < W; ++e) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t[e]));
  return Vec<W>(t);
}
// (a sigmoid(a))' given s = sigmoid(a)
template <int W> __device__ __forceinline__ Vec<W> silu_grad(const Vec<W> &a, const Vec<W> &s) {
  return s * fma(a, fma(s, Vec<W>(-1.f), Vec<W>(1.f)), Vec<W>(1.f));
}

// Vec of what lies in a Raw
template <typename T, int W>
__device__ __forceinline__ Vec<W> vec_of(const Raw<T, W> &r) {
  float v[W];
  r.get(v);
  return Vec<W>(v);
}
// W parameters of consecutive channels (c a multiple of W), or a constant where there are none
template <int W>
__device__ __forceinline__ Vec<W> load_param(const float *p, int c, float none) {
  float v[W];
  if (W == 8 && p && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    load_vec<W>(p + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = p ? __ldg(p + c + e) : none;
  }
  return Vec<W>(v);
}

// ---------------------------------------------------------------- sums over a team of NT threads
// (`fresh`: the scratch has not been used since a barrier)
template <int NT>
__device__ __forceinline__ float team_sum(float a, float *scratch, bool fresh = false) {
#pragma unroll
  for (int o = (NT < 32 ? NT : 32) / 2; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if constexpr (NT > 32) {
    if (!fresh) __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) a += scratch[w];
  }
  return a;
}
// two sums at once; scratch of 16 values
template <int NT>
__device__ __forceinline__ float2 team_sum2(float a, float b, float *scratch, bool fresh = false) {
#pragma unroll
  for (int o = (NT < 32 ? NT : 32) / 2; o >= 1; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (NT > 32) {
    if (!fresh) __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      scratch[threadIdx.x >> 5] = a;
      scratch[8 + (threadIdx.x >> 5)] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      a += scratch[w];
      b += scratch[8 + w];
    }
  }
  return make_float2(a, b);
}

// ---------------------------------------------------------------- a thread's places in a slab
// V places among a group's rows [r0, rows): column vectors of W channels.  With at most
// NT columns a thread keeps one column and takes every (NT / columns)-th row; with
// more the group is one sequence of vectors, taken from e0 on.
template <int W, int NT, int V>
struct Places {
  int row[V], col[V];  // row < 0: no such place
  __device__ __forceinline__ Places(int tid, int ncol, int r0, long long e0, int rows) {
    if constexpr (V == 1) {  // one row of at most NT columns
      row[0] = rows > 0 && tid < ncol ? 0 : -1;
      col[0] = tid * W;
    } else if (ncol <= NT) {
      const int rp = NT / ncol, ph = tid / ncol;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int r = r0 + ph + k * rp;
        row[k] = ph < rp && r < rows ? r : -1;
        col[k] = (tid - ph * ncol) * W;
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const long long e = e0 + tid + k * NT, r = e / ncol;
        row[k] = r < rows ? (int)r : -1;
        col[k] = (int)(e - r * ncol) * W;
      }
    }
  }
};
// The same with at most NT columns, without arrays: a thread's live places are the first `n`, `step` rows apart.
template <int W, int NT, int V>
struct ColumnPlaces {
  int row, step, col, n;
  __device__ __forceinline__ ColumnPlaces(int tid, int ncol, int r0, int rows) {
    step = NT / ncol;
    const int ph = tid / ncol;
    row = r0 + ph;
    col = (tid - ph * ncol) * W;
    n = ph < step && row < rows ? min(V, (rows - row + step - 1) / step) : 0;
  }
  // a tensor's pointer at place k
  template <typename U> __device__ __forceinline__ U *at(U *slab, int stride, int k) const {
    return slab + ((long long)row * stride + col) + (long long)k * ((long long)step * stride);
  }
};
// rows that fit a team's places (0: not one)
inline long long rows_of_team(int ncol, int nt, int v) {
  return ncol <= nt ? (long long)v * (nt / ncol) : (long long)v * nt / ncol;
}
// Tile t of a group: rows [t tile_rows, ...) or, where a row has more columns than a block has threads,
// vectors [t V NT, ...); and its number of values.  (A cluster's last blocks may have no tile: no rows.)
template <int W, int V>
struct Tile {
  int n, g, t;
  Places<W, kThreads, V> at;
  __device__ __forceinline__ Tile(const GnProblem &p, const GnPlan &pl)
      : n(pl.cluster ? blockIdx.x / pl.cluster / p.G : blockIdx.x / p.G / pl.tiles),
        g(pl.cluster ? blockIdx.x / pl.cluster % p.G : blockIdx.x % p.G),
        t(pl.cluster ? blockIdx.x % pl.cluster : blockIdx.x / p.G % pl.tiles),
        at(threadIdx.x, p.cg / W, t * pl.tile_rows, (long long)t * (V * kThreads), limit(p, pl)) {}
  // (in rows mode a thread's last places may lie in the next tile)
  __device__ __forceinline__ int limit(const GnProblem &p, const GnPlan &pl) const {
    return pl.own_columns ? min(p.m, (t + 1) * pl.tile_rows) : p.m;
  }
  static __device__ __forceinline__ float count(const GnProblem &p, const GnPlan &pl, int i) {
    if (pl.own_columns) return (float)max(0, min(pl.tile_rows, p.m - i * pl.tile_rows)) * p.cg;
    const long long left = (long long)p.m * (p.cg / W) - (long long)i * (V * kThreads);
    return (float)max(0LL, left < V * kThreads ? left : (long long)(V * kThreads)) * W;
  }
};

// u -> y
template <int W, bool GATE>
__device__ __forceinline__ Vec<W> activate(const Vec<W> &u, const Vec<W> &z, bool silu) {
  if (GATE) return u * (z * sigmoid(z));
  return silu ? u * sigmoid(u) : u;
}
// dy -> du, and dz with the gate
template <int W, bool GATE>
__device__ __forceinline__ Vec<W> activate_grad(const Vec<W> &dy, const Vec<W> &u, const Vec<W> &z, bool silu, Vec<W> &dz) {
  if (GATE) {
    const Vec<W> s = sigmoid(z);
    dz = dy * u * silu_grad(z, s);
    return dy * (z * s);
  }
  return silu ? dy * silu_grad(u, sigmoid(u)) : dy;
}

__device__ __forceinline__ long long off(int row, int stride) { return (long long)row * stride; }

// one group of one sample: pointers to its first row's first channel
template <typename T>
struct Slab {
  const T *x, *z, *dy;
  T *y, *dx, *dz;
  __device__ __forceinline__ Slab(const GnProblem &p, int n, int g) {
    const long long r = (long long)n * p.m;
    const int c = g * p.cg;
    x = static_cast<const T *>(p.x) + r * p.xs + c;
    z = static_cast<const T *>(p.z) + r * p.zs + c;
    dy = static_cast<const T *>(p.dy) + r * p.dys + c;
    y = static_cast<T *>(p.y) + r * p.ys + c;
    dx = static_cast<T *>(p.dx) + r * p.dxs + c;
    dz = static_cast<T *>(p.dz) + r * p.dzs + c;
  }
};

template <typename T, int W, bool GATE>
__device__ __forceinline__ void write_y(const GnProblem &p, T *to, const Vec<W> &w, const Vec<W> &b, const Vec<W> &x,
                                        const Raw<T, W> &z, float mean, float rstd) {
  const Vec<W> u = fma((x + Vec<W>(-mean)) * Vec<W>(rstd), w, b);
  float y[W];
  activate<W, GATE>(u, GATE ? vec_of<T, W>(z) : u, p.act == SSD_ACT_SILU).get(y);
  store_vec<W>(to, y);
}
// sum of (x - mean)^2
template <int W>
__device__ __forceinline__ float deviations(const Vec<W> &x, float mean) {
  const Vec<W> d = x + Vec<W>(-mean);
  return (d * d).sum();
}

// ---------------------------------------------------------------- a thread's own values on their way
// COUNT slots in shared memory for a thread's W channels, which it copies and reads for itself alone (no barrier), so
// that loads in flight do not cost registers.
template <typename T, int W, int COUNT>
struct Slots {
  static constexpr int kPiece = W * (int)sizeof(T), kStep = kPiece < 16 ? kPiece : 16, kChunks = kPiece / kStep;
  static constexpr int kBytes = COUNT * kPiece * kThreads;
  unsigned char *base;
  __device__ __forceinline__ explicit Slots(void *smem) : base(static_cast<unsigned char *>(smem)) {}
  __device__ __forceinline__ unsigned char *at(int i, int c) const {
    return base + ((i * kChunks + c) * kThreads + threadIdx.x) * kStep;
  }
  __device__ __forceinline__ void load(int i, const T *from) const {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      unsigned char *to = at(i, c);
      const unsigned char *src = reinterpret_cast<const unsigned char *>(from) + c * kStep;
      if constexpr (kStep == 16)
        sm100::cp_async16(sm100::smem_u32(to), src);
      else if constexpr (kStep >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(sm100::smem_u32(to)), "l"(src), "n"(kStep) : "memory");
      else  // less than an asynchronous copy moves
        *reinterpret_cast<T *>(to) = *from;
    }
  }
  __device__ __forceinline__ void get(int i, Raw<T, W> &to) const {
    if constexpr (W == 8) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) reinterpret_cast<uint4 *>(&to)[c] = *reinterpret_cast<const uint4 *>(at(i, c));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < W; ++e) to.f[e] = reinterpret_cast<const float *>(at(i, 0))[e];
    } else if constexpr (W == 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t *>(at(i, 0));
      to.f[0] = __uint_as_float(u << 16);
      to.f[1] = __uint_as_float(u & 0xffff0000u);
    } else {
      to.f[0] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(at(i, 0)));
    }
  }
};
// Teams of one place keep their next samples' values in a ring of stages.
// (forward with a gate: 131 us with 4 stages, 136 us with 6; backward: 117 us with 3, 118 us with 4)
template <typename T, int W, int TENSORS>
constexpr int kRingStages = TENSORS * Slots<T, W, 1>::kChunks <= 2 ? 4 : 3;
template <typename T, int W, int TENSORS>
struct Ring : Slots<T, W, kRingStages<T, W, TENSORS> * TENSORS> {
  using Base = Slots<T, W, kRingStages<T, W, TENSORS> * TENSORS>;
  static constexpr int kStages = kRingStages<T, W, TENSORS>;
  using Base::Base;
  __device__ __forceinline__ void load(int stage, int t, const T *from) const { Base::load(stage * TENSORS + t, from); }
  __device__ __forceinline__ void get(int stage, int t, Raw<T, W> &to) const { Base::get(stage * TENSORS + t, to); }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // all but the last kStages - 2 groups have landed
  static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory"); }
};

// ---------------------------------------------------------------- forward, groups that fit a team
// Teams that each keep one group and walk over samples; block (groups of the block, samples of the block).
// With one place to a thread the next samples' values are on their way while one is worked on.
template <int V>
constexpr int min_blocks(int one) { return V == 1 ? one : 1; }
template <typename T, int W, int NT, int V, bool GATE>
__global__ void __launch_bounds__(kThreads, min_blocks<V>(sizeof(T) == 2 ? 4 : 3))
    team_forward_kernel(GnProblem p, GnPlan pl) {
  constexpr int kTeams = kThreads / NT;
  __shared__ float red[16];
  const int team = threadIdx.x / NT, tid = threadIdx.x % NT, gpb = pl.groups_per_block, shares = kTeams / gpb;
  const int share = team / gpb, g = blockIdx.x * gpb + team % gpb;
  const bool has = g < p.G && share < shares;
  const int n0 = blockIdx.y * pl.samples_per_block + share;
  const int n1 = min(p.n, (blockIdx.y + 1) * pl.samples_per_block), c0 = (has ? g : 0) * p.cg;
  const int turns = (n1 - (int)blockIdx.y * pl.samples_per_block + shares - 1) / shares;
  const float inv = 1.f / ((float)p.m * p.cg);
  const Places<W, NT, V> at(tid, p.cg / W, 0, 0, has ? p.m : 0);
  Vec<W> w, b;
  if (pl.own_columns && has && at.row[0] >= 0) {
    w = load_param<W>(p.w, c0 + at.col[0], 1.f);
    b = load_param<W>(p.b, c0 + at.col[0], 0.f);
  }
  using R = Ring<T, W, GATE ? 2 : 1>;
  extern __shared__ uint4 ring_smem[];
  const R ring(ring_smem);
  auto ahead = [&](int i) {  // turn i's values on their way
    const int n = n0 + i * shares;
    if (has && n < n1 && at.row[0] >= 0) {
      const Slab<T> s(p, n, g);
      ring.load(i % R::kStages, 0, s.x + at.col[0]);
      if (GATE) ring.load(i % R::kStages, 1, s.z + at.col[0]);
    }
    R::commit();
  };
  if constexpr (V == 1)
    for (int i = 0; i < R::kStages - 1; ++i) ahead(i);
  // every thread of a warp makes the same number of turns (the sums are warp or block wide)
  for (int i = 0; i < turns; ++i) {
    const int n = n0 + i * shares;
    const bool live = has && n < n1;
    const Slab<T> s(p, live ? n : 0, has ? g : 0);
    Vec<W> x[V];
    Raw<T, W> z[V];
    if constexpr (V == 1) R::wait();
#pragma unroll
    for (int k = 0; k < V; ++k) {
      Raw<T, W> xr;
      if (live && at.row[k] >= 0) {
        if constexpr (V == 1) {
          ring.get(i % R::kStages, 0, xr);
          if (GATE) ring.get(i % R::kStages, 1, z[0]);
        } else {
          xr.load(s.x + off(at.row[k], p.xs) + at.col[k]);
          if (GATE) z[k].load(s.z + off(at.row[k], p.zs) + at.col[k]);
        }
      } else {
        xr.clear();
      }
      x[k] = vec_of<T, W>(xr);
    }
    if constexpr (V == 1) ahead(i + R::kStages - 1);
    float sum = 0.f, dev = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) sum += x[k].sum();
    const float mean = team_sum<NT>(sum, red) * inv;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (live && at.row[k] >= 0) dev += deviations<W>(x[k], mean);
    const float rstd = 1.f / sqrtf(team_sum<NT>(dev, red) * inv + p.eps);
    if (live && tid == 0) {
      if (p.mean) p.mean[n * p.G + g] = mean;
      if (p.rstd) p.rstd[n * p.G + g] = rstd;
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (live && at.row[k] >= 0) {
        if (!pl.own_columns) {
          w = load_param<W>(p.w, c0 + at.col[k], 1.f);
          b = load_param<W>(p.b, c0 + at.col[k], 0.f);
        }
        write_y<T, W, GATE>(p, s.y + off(at.row[k], p.ys) + at.col[k], w, b, x[k], z[k], mean, rstd);
      }
  }
}

// weight and bias of a thread's places: loaded once where it keeps its column
template <int W>
struct Params {
  Vec<W> wv, bv;
  bool own;
  __device__ __forceinline__ Params(const GnProblem &p, const GnPlan &pl, int c0, int col, bool live)
      : wv(1.f), bv(0.f), own(pl.own_columns) {
    if (own && live) {
      wv = load_param<W>(p.w, c0 + col, 1.f);
      bv = load_param<W>(p.b, c0 + col, 0.f);
    }
  }
  __device__ __forceinline__ Vec<W> w(const GnProblem &p, int c0, int col) const {
    return own ? wv : load_param<W>(p.w, c0 + col, 1.f);
  }
  __device__ __forceinline__ Vec<W> b(const GnProblem &p, int c0, int col) const {
    return own ? bv : load_param<W>(p.b, c0 + col, 0.f);
  }
};

// ---------------------------------------------------------------- forward, groups in tiles of rows
// Block (tile, group, sample): the tile's count, mean and squared deviations, joined over the threads
// as pairs (each thread's from its own values, twice over registers).
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads) tile_stats_kernel(GnProblem p, GnPlan pl, float *part) {
  __shared__ float red[16];
  const Tile<W, V> tile(p, pl);
  const Places<W, kThreads, V> &at = tile.at;
  const int n = tile.n, g = tile.g, t = tile.t;
  const Slab<T> s(p, n, g);
  Raw<T, W> xr[V];
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (at.row[k] >= 0)
      xr[k].load(s.x + off(at.row[k], p.xs) + at.col[k]);
    else
      xr[k].clear();
  float sum = 0.f, dev = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) sum += vec_of<T, W>(xr[k]).sum();
  const float mean = team_sum<kThreads>(sum, red) / Tile<W, V>::count(p, pl, t);
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (at.row[k] >= 0) dev += deviations<W>(vec_of<T, W>(xr[k]), mean);
  dev = team_sum<kThreads>(dev, red);
  if (threadIdx.x == 0) {
    float *q = part + 2 * (((size_t)n * p.G + g) * pl.tiles + t);
    q[0] = mean;
    q[1] = dev;
  }
}

// The joined mean and 1 / sqrt(variance + eps) of a group's tiles, whose own means and squared deviations come
// from get(tile): the tiles' means by their counts, then the deviations about the joined mean.  A warp's lanes take
// up to 32 tiles, each warp for itself; more go to the block's threads.
template <int W, int V, class GET>
__device__ __forceinline__ float2 join_stats(const GnProblem &p, const GnPlan &pl, float *red, GET get) {
  const float inv = 1.f / ((float)p.m * p.cg);
  if (pl.tiles <= 32) {
    const int i = threadIdx.x & 31;
    const float2 q = i < pl.tiles ? get(i) : make_float2(0.f, 0.f);
    const float c = i < pl.tiles ? Tile<W, V>::count(p, pl, i) : 0.f, base = __shfl_sync(0xffffffffu, q.x, 0);
    const float off = team_sum<32>((q.x - base) * c, red) * inv, d = (q.x - base) - off;
    return make_float2(base + off, 1.f / sqrtf(team_sum<32>(fmaf(d * d, c, q.y), red) * inv + p.eps));
  }
  const float base = get(0).x;
  float sum = 0.f, dev = 0.f;
  for (int i = threadIdx.x; i < pl.tiles; i += kThreads) sum += (get(i).x - base) * Tile<W, V>::count(p, pl, i);
  const float off = team_sum<kThreads>(sum, red) * inv;
  for (int i = threadIdx.x; i < pl.tiles; i += kThreads) {
    const float2 q = get(i);
    const float d = (q.x - base) - off;
    dev += fmaf(d * d, Tile<W, V>::count(p, pl, i), q.y);
  }
  return make_float2(base + off, 1.f / sqrtf(team_sum<kThreads>(dev, red) * inv + p.eps));
}

// Before a block of a cluster ends, the others have to have read its shared memory: they arrive after their
// reads (which orders nothing else: no waiting for stores) and wait at their end.
__device__ __forceinline__ void cluster_done_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;"); }
__device__ __forceinline__ void cluster_done_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// A cluster of blocks per group: loaded once, the tiles' statistics exchanged between the blocks.
template <typename T, int W, int V, bool GATE>
__global__ void __launch_bounds__(kThreads) cluster_forward_kernel(GnProblem p, GnPlan pl) {
  namespace cg = cooperative_groups;
  __shared__ float red[2][8];
  __shared__ float2 mine;
  const cg::cluster_group cluster = cg::this_cluster();
  const int pair = blockIdx.x / pl.cluster, t = blockIdx.x % pl.cluster, n = pair / p.G, g = pair % p.G;
  const ColumnPlaces<W, kThreads, V> at(threadIdx.x, p.cg / W, t * pl.tile_rows, min(p.m, (t + 1) * pl.tile_rows));
  const Slab<T> s(p, n, g);
  Raw<T, W> xr[V], zr[V];
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < at.n) {
      xr[k].load(at.at(s.x, p.xs, k));
      if (GATE) zr[k].load(at.at(s.z, p.zs, k));
    } else {
      xr[k].clear();
    }
  Vec<W> w(1.f), b(0.f);
  if (at.n > 0) {
    w = load_param<W>(p.w, g * p.cg + at.col, 1.f);
    b = load_param<W>(p.b, g * p.cg + at.col, 0.f);
  }
  float sum = 0.f, dev = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) sum += vec_of<T, W>(xr[k]).sum();
  const float own = team_sum<kThreads>(sum, red[0], true) / fmaxf(Tile<W, V>::count(p, pl, t), 1.f);
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < at.n) dev += deviations<W>(vec_of<T, W>(xr[k]), own);
  dev = team_sum<kThreads>(dev, red[1], true);
  if (threadIdx.x == 0) mine = make_float2(own, dev);
  cluster.sync();
  const float2 st = join_stats<W, V>(p, pl, red[0], [&](int i) { return *cluster.map_shared_rank(&mine, i); });
  __syncwarp();
  cluster_done_arrive();
  if (t == 0 && threadIdx.x == 0) {
    if (p.mean) p.mean[pair] = st.x;
    if (p.rstd) p.rstd[pair] = st.y;
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < at.n) write_y<T, W, GATE>(p, at.at(s.y, p.ys, k), w, b, vec_of<T, W>(xr[k]), zr[k], st.x, st.y);
  cluster_done_wait();
}

template <typename T, int W, int V, bool GATE>
__global__ void __launch_bounds__(kThreads) tile_forward_kernel(GnProblem p, GnPlan pl, const float *part) {
  __shared__ float red[16];
  const Tile<W, V> tile(p, pl);
  const Places<W, kThreads, V> &at = tile.at;
  const int n = tile.n, g = tile.g, t = tile.t, c0 = g * p.cg;
  const Slab<T> s(p, n, g);
  const Params<W> params(p, pl, c0, at.col[0], at.row[0] >= 0);
  Raw<T, W> xr[V], zr[V];
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (at.row[k] >= 0) {
      xr[k].load(s.x + off(at.row[k], p.xs) + at.col[k]);
      if (GATE) zr[k].load(s.z + off(at.row[k], p.zs) + at.col[k]);
    }
  const float2 *q = reinterpret_cast<const float2 *>(part) + ((size_t)n * p.G + g) * pl.tiles;
  const float2 st = join_stats<W, V>(p, pl, red, [&](int i) { return q[i]; });
  const float mean = st.x, rstd = st.y;
  if (t == 0 && threadIdx.x == 0) {
    if (p.mean) p.mean[n * p.G + g] = mean;
    if (p.rstd) p.rstd[n * p.G + g] = rstd;
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (at.row[k] >= 0)
      write_y<T, W, GATE>(p, s.y + off(at.row[k], p.ys) + at.col[k], params.w(p, c0, at.col[k]), params.b(p, c0, at.col[k]),
                          vec_of<T, W>(xr[k]), zr[k], mean, rstd);
}

// ---------------------------------------------------------------- backward
// What a place gives: du w (gradient of xhat) and xhat, its part of dw and db, and dz, which is stored if asked for.
template <typename T, int W, bool GATE>
__device__ __forceinline__ void place_grad(const GnProblem &p, const Raw<T, W> &xr, const Raw<T, W> &zr,
                                           const Raw<T, W> &dyr, const Vec<W> &w, const Vec<W> &b, float mean, float rstd,
                                           Vec<W> &dxh, Vec<W> &xh, Vec<W> &dw, Vec<W> &db, T *dz_to) {
  Vec<W> dz;
  xh = (vec_of<T, W>(xr) + Vec<W>(-mean)) * Vec<W>(rstd);
  const Vec<W> dy = vec_of<T, W>(dyr);
  const Vec<W> du =
      activate_grad<W, GATE>(dy, fma(xh, w, b), GATE ? vec_of<T, W>(zr) : dy, p.act == SSD_ACT_SILU, dz);
  dw = fma(du, xh, dw);
  db = db + du;
  dxh = du * w;
  if (GATE && dz_to) {
    float v[W];
    dz.get(v);
    store_vec<W>(dz_to, v);
  }
}
// dx = rstd (dxh - a - xh b)
template <typename T, int W>
__device__ __forceinline__ void write_dx(T *to, const Vec<W> &dxh, const Vec<W> &xh, float a, float b, float rstd) {
  float v[W];
  (Vec<W>(rstd) * fma(xh, Vec<W>(-b), dxh + Vec<W>(-a))).get(v);
  store_vec<W>(to, v);
}
template <typename T, int W, bool GATE>
__device__ __forceinline__ void load_place(const GnProblem &p, const Slab<T> &s, int row, int col, Raw<T, W> &x,
                                           Raw<T, W> &z, Raw<T, W> &dy) {
  x.load(s.x + off(row, p.xs) + col);
  dy.load(s.dy + off(row, p.dys) + col);
  if (GATE) z.load(s.z + off(row, p.zs) + col);
}

// dw and db of a block's `channels` channels: each is held by `holders` threads (thread_of(channel, holder), element
// channel % W of theirs) and added over them in a fixed order: in up to kThreads / channels runs, then the runs.
template <int W, class TH, class WR>
__device__ __forceinline__ void sum_params(float (&acc)[2][kThreads * W], int channels, int holders, TH thread_of,
                                           WR write) {
  __shared__ float run[2][kThreads];
  __syncthreads();
  const int runs = min(holders, max(1, kThreads / channels)), per = (holders + runs - 1) / runs;
  for (int c0 = 0; c0 < channels; c0 += kThreads) {
    const int c = c0 + threadIdx.x % min(channels, kThreads), q = threadIdx.x / min(channels, kThreads);
    float sw = 0.f, sb = 0.f;
    if (c < channels && q < runs)
      for (int j = q * per; j < min(holders, (q + 1) * per); ++j) {
        const int at = thread_of(c, j) * W + c % W;
        sw += acc[0][at];
        sb += acc[1][at];
      }
    if (runs > 1) {  // then all channels are in this one turn
      run[0][threadIdx.x] = sw;
      run[1][threadIdx.x] = sb;
      __syncthreads();
      if (q == 0)
        for (int i = 1; i < runs; ++i) {
          sw += run[0][i * channels + c];
          sb += run[1][i * channels + c];
        }
    }
    if (q == 0 && c < channels) write(c, sw, sb);
  }
}

template <int W>
__device__ __forceinline__ void keep_params(float (&acc)[2][kThreads * W], const Vec<W> &dw, const Vec<W> &db) {
  float a[W], b[W];
  dw.get(a);
  db.get(b);
#pragma unroll
  for (int e = 0; e < W; ++e) {
    acc[0][threadIdx.x * W + e] = a[e];
    acc[1][threadIdx.x * W + e] = b[e];
  }
}

// As the forward's teams; dw and db of the block's samples at the end.
template <typename T, int W, int NT, int V, bool GATE>
__global__ void __launch_bounds__(kThreads, min_blocks<V>(sizeof(T) == 2 ? 3 : 2))
    team_backward_kernel(GnProblem p, GnPlan pl, float *dwp, float *dbp) {
  constexpr int kTeams = kThreads / NT;
  __shared__ float red[16];
  using R = Ring<T, W, GATE ? 3 : 2>;
  using Acc = float[2][kThreads * W];
  extern __shared__ uint4 ring_smem[];  // the ring, then what the threads have of dw and db
  const R ring(ring_smem);
  Acc &acc = *reinterpret_cast<Acc *>(ring_smem);
  const int team = threadIdx.x / NT, tid = threadIdx.x % NT, gpb = pl.groups_per_block, shares = kTeams / gpb;
  const int gl = team % gpb, share = team / gpb, g = blockIdx.x * gpb + gl, ncol = p.cg / W;
  const bool has = g < p.G && share < shares;
  const int n0 = blockIdx.y * pl.samples_per_block + share;
  const int n1 = min(p.n, (blockIdx.y + 1) * pl.samples_per_block), c0 = (has ? g : 0) * p.cg;
  const int turns = (n1 - (int)blockIdx.y * pl.samples_per_block + shares - 1) / shares;
  const float inv = 1.f / ((float)p.m * p.cg);
  const Places<W, NT, V> at(tid, ncol, 0, 0, has ? p.m : 0);
  Vec<W> w(0.f), b(0.f), dw(0.f), db(0.f);  // with at most NT columns a thread keeps one
  const int col = at.col[0];
  if (has && at.row[0] >= 0) {
    w = load_param<W>(p.w, c0 + col, 1.f);
    b = load_param<W>(p.b, c0 + col, 0.f);
  }
  float mean_r = 0.f, rstd_r = 0.f;
  auto stats = [&](int n) {
    if (has && n < n1) {
      mean_r = __ldg(p.mean + n * p.G + g);
      rstd_r = __ldg(p.rstd + n * p.G + g);
    }
  };
  auto ahead = [&](int i) {  // turn i's values on their way
    const int n = n0 + i * shares;
    if (has && n < n1 && at.row[0] >= 0) {
      const Slab<T> s(p, n, g);
      ring.load(i % R::kStages, 0, s.x + col);
      ring.load(i % R::kStages, 1, s.dy + col);
      if (GATE) ring.load(i % R::kStages, 2, s.z + col);
    }
    R::commit();
  };
  if constexpr (V == 1) {
    for (int i = 0; i < R::kStages - 1; ++i) ahead(i);
    stats(n0);
  }
  for (int i = 0; i < turns; ++i) {
    const int n = n0 + i * shares;
    const bool live = has && n < n1;
    if (V > 1) stats(n);
    const float mean = mean_r, rstd = rstd_r;
    Raw<T, W> xr, zr, dyr;
    if constexpr (V == 1) {
      R::wait();
      if (live && at.row[0] >= 0) {
        ring.get(i % R::kStages, 0, xr);
        ring.get(i % R::kStages, 1, dyr);
        if (GATE) ring.get(i % R::kStages, 2, zr);
      }
      ahead(i + R::kStages - 1);
      stats(n + shares);
    }
    const Slab<T> s(p, live ? n : 0, has ? g : 0);
    Vec<W> dxh[V], xh[V];
    float sa = 0.f, sb = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (live && at.row[k] >= 0) {
        if (V > 1) load_place<T, W, GATE>(p, s, at.row[k], col, xr, zr, dyr);
        place_grad<T, W, GATE>(p, xr, zr, dyr, w, b, mean, rstd, dxh[k], xh[k], dw, db,
                               s.dz + off(at.row[k], p.dzs) + col);
        sa += dxh[k].sum();
        sb += (dxh[k] * xh[k]).sum();
      }
    const float2 ab = team_sum2<NT>(sa, sb, red);
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (live && at.row[k] >= 0)
        write_dx<T, W>(s.dx + off(at.row[k], p.dxs) + col, dxh[k], xh[k], ab.x * inv, ab.y * inv, rstd);
  }
  if (!dwp) return;
  if constexpr (V == 1) {  // the ring is done with
    sm100::cp_async_wait_all();
    __syncthreads();
  }
  // the threads of a block that hold the same channels: the teams of a group, each team's row phases
  keep_params<W>(acc, dw, db);
  const int phases = V == 1 ? 1 : NT / ncol;
  sum_params<W>(
      acc, gpb * p.cg, shares * phases,
      [&](int c, int j) { return (j / phases * gpb + c / p.cg) * NT + j % phases * ncol + c % p.cg / W; },
      [&](int c, float sw, float sb) {
        const int ch = blockIdx.x * gpb * p.cg + c;
        if (ch < p.C) {
          dwp[(size_t)blockIdx.y * p.C + ch] = sw;
          dbp[(size_t)blockIdx.y * p.C + ch] = sb;
        }
      });
}

// Tiles, first kernel: the tile's parts of A and B, of dw and db (when a thread keeps its column), and dz.
template <typename T, int W, int V, bool GATE>
__global__ void __launch_bounds__(kThreads) tile_sums_kernel(GnProblem p, GnPlan pl, float *part, float *dwp,
                                                             float *dbp) {
  __shared__ float red[16];
  __shared__ float acc[2][kThreads * W];
  const Tile<W, V> tile(p, pl);
  const Places<W, kThreads, V> &at = tile.at;
  const int n = tile.n, g = tile.g, t = tile.t, c0 = g * p.cg, ncol = p.cg / W;
  const Slab<T> s(p, n, g);
  const float mean = __ldg(p.mean + n * p.G + g), rstd = __ldg(p.rstd + n * p.G + g);
  const Params<W> params(p, pl, c0, at.col[0], at.row[0] >= 0);
  Raw<T, W> xr[V], zr[V], dyr[V];
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (at.row[k] >= 0) load_place<T, W, GATE>(p, s, at.row[k], at.col[k], xr[k], zr[k], dyr[k]);
  Vec<W> dw(0.f), db(0.f);
  float sa = 0.f, sb = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (at.row[k] >= 0) {
      Vec<W> dxh, xh;
      place_grad<T, W, GATE>(p, xr[k], zr[k], dyr[k], params.w(p, c0, at.col[k]),
                             params.b(p, c0, at.col[k]), mean, rstd, dxh, xh, dw, db,
                             s.dz + off(at.row[k], p.dzs) + at.col[k]);
      sa += dxh.sum();
      sb += (dxh * xh).sum();
    }
  const float2 ab = team_sum2<kThreads>(sa, sb, red);
  if (threadIdx.x == 0) {
    float *q = part + 2 * (((size_t)n * p.G + g) * pl.tiles + t);
    q[0] = ab.x;
    q[1] = ab.y;
  }
  if (!dwp) return;
  keep_params<W>(acc, dw, db);
  sum_params<W>(
      acc, p.cg, kThreads / ncol, [&](int c, int j) { return j * ncol + c / W; },
      [&](int c, float sw, float sd) {
        const size_t to = ((size_t)n * pl.tiles + t) * p.C + c0 + c;
        dwp[to] = sw;
        dbp[to] = sd;
      });
}

// A cluster of blocks per group: loaded once, the parts of A and B exchanged between the blocks.
// The inputs wait in shared memory, so that three blocks fit an SM: 57 samples of 771 rows of 16 groups of 64
// channels, bf16, 127 us (in registers, two blocks: 140 us; 8 samples of 2048 rows of 32 groups of 16: 31 us and 29 us).
template <typename T, int W, int V, bool GATE>
__global__ void __launch_bounds__(kThreads, W == 8 && sizeof(T) == 4 ? 2 : 3) cluster_backward_kernel(GnProblem p, GnPlan pl, float *dwp, float *dbp) {
  namespace cg = cooperative_groups;
  __shared__ float red[16];
  __shared__ float2 mine;
  __shared__ float acc[2][kThreads * W];
  extern __shared__ uint4 slot_smem[];
  const Slots<T, W, (GATE ? 3 : 2) * V> slots(slot_smem);  // x, dy, z of each place
  const cg::cluster_group cluster = cg::this_cluster();
  const int pair = blockIdx.x / pl.cluster, t = blockIdx.x % pl.cluster, n = pair / p.G, g = pair % p.G;
  const int c0 = g * p.cg, ncol = p.cg / W;
  const ColumnPlaces<W, kThreads, V> at(threadIdx.x, ncol, t * pl.tile_rows, min(p.m, (t + 1) * pl.tile_rows));
  const Slab<T> s(p, n, g);
  const float mean = __ldg(p.mean + pair), rstd = __ldg(p.rstd + pair);
  const float inv = 1.f / ((float)p.m * p.cg);
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < at.n) {
      slots.load(k, at.at(s.x, p.xs, k));
      slots.load(V + k, at.at(s.dy, p.dys, k));
      if (GATE) slots.load(2 * V + k, at.at(s.z, p.zs, k));
    }
  Vec<W> w(1.f), b(0.f);
  if (at.n > 0) {
    w = load_param<W>(p.w, c0 + at.col, 1.f);
    b = load_param<W>(p.b, c0 + at.col, 0.f);
  }
  Vec<W> dw(0.f), db(0.f), dxh[V];
  float sa = 0.f, sb = 0.f;
  sm100::cp_async_wait_all();
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < at.n) {
      Vec<W> xh;
      Raw<T, W> x, z, dy;
      slots.get(k, x);
      slots.get(V + k, dy);
      if (GATE) slots.get(2 * V + k, z);
      place_grad<T, W, GATE>(p, x, z, dy, w, b, mean, rstd, dxh[k], xh, dw, db,
                             at.at(s.dz, p.dzs, k));
      sa += dxh[k].sum();
      sb += (dxh[k] * xh).sum();
    }
  const float2 own = team_sum2<kThreads>(sa, sb, red, true);
  if (threadIdx.x == 0) mine = own;
  if (dwp) keep_params<W>(acc, dw, db);
  cluster.sync();
  const int lane = threadIdx.x & 31;  // each warp for itself
  const float2 q = lane < pl.tiles ? *cluster.map_shared_rank(&mine, lane) : make_float2(0.f, 0.f);
  const float2 ab = team_sum2<32>(q.x, q.y, red);
  __syncwarp();
  cluster_done_arrive();
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < at.n) {
      Raw<T, W> x;
      slots.get(k, x);
      write_dx<T, W>(at.at(s.dx, p.dxs, k), dxh[k], (vec_of<T, W>(x) + Vec<W>(-mean)) * Vec<W>(rstd), ab.x * inv,
                     ab.y * inv, rstd);
    }
  if (dwp && t < pl.tiles) {
    sum_params<W>(
        acc, p.cg, kThreads / ncol, [&](int c, int j) { return j * ncol + c / W; },
        [&](int c, float sw, float sd) {
          const size_t to = ((size_t)n * pl.tiles + t) * p.C + c0 + c;
          dwp[to] = sw;
          dbp[to] = sd;
        });
  }
  cluster_done_wait();
}

template <typename T, int W, int V, bool GATE>
__global__ void __launch_bounds__(kThreads) tile_backward_kernel(GnProblem p, GnPlan pl, const float *part) {
  __shared__ float red[16];
  const Tile<W, V> tile(p, pl);
  const Places<W, kThreads, V> &at = tile.at;
  const int n = tile.n, g = tile.g, t = tile.t, c0 = g * p.cg;
  const Slab<T> s(p, n, g);
  const float mean = __ldg(p.mean + n * p.G + g), rstd = __ldg(p.rstd + n * p.G + g);
  const Params<W> params(p, pl, c0, at.col[0], at.row[0] >= 0);
  Raw<T, W> xr[V], zr[V], dyr[V];
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (at.row[k] >= 0) load_place<T, W, GATE>(p, s, at.row[k], at.col[k], xr[k], zr[k], dyr[k]);
  const float *q = part + 2 * ((size_t)n * p.G + g) * pl.tiles;
  float sa = 0.f, sb = 0.f;
  for (int i = threadIdx.x; i < pl.tiles; i += kThreads) {
    sa += q[2 * i];
    sb += q[2 * i + 1];
  }
  const float inv = 1.f / ((float)p.m * p.cg);
  const float2 ab = team_sum2<kThreads>(sa, sb, red);
  Vec<W> dw(0.f), db(0.f);
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (at.row[k] >= 0) {
      Vec<W> dxh, xh;
      place_grad<T, W, GATE>(p, xr[k], zr[k], dyr[k], params.w(p, c0, at.col[k]),
                             params.b(p, c0, at.col[k]), mean, rstd, dxh, xh, dw, db,
                             static_cast<T *>(nullptr));
      write_dx<T, W>(s.dx + off(at.row[k], p.dxs) + at.col[k], dxh, xh, ab.x * inv, ab.y * inv, rstd);
    }
}

// dw and db of rows of groups wider than a block (a thread then has no column of its own): a thread per
// channel, a tile of rows per block
constexpr int kParamRows = 256;
template <typename T, bool GATE>
__global__ void __launch_bounds__(kThreads) param_kernel(GnProblem p, float *dwp, float *dbp) {
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= p.C) return;
  const int g = c / p.cg;
  const long long r0 = (long long)blockIdx.x * kParamRows, r1 = min((long long)p.n * p.m, r0 + kParamRows);
  const Vec<1> w = load_param<1>(p.w, c, 1.f), b = load_param<1>(p.b, c, 0.f);
  Vec<1> sw(0.f), sb(0.f);
  for (long long r = r0; r < r1; ++r) {
    const size_t at = (size_t)(r / p.m) * p.G + g;
    Raw<T, 1> x, z, dy;
    Vec<1> dxh, xh;
    x.load(static_cast<const T *>(p.x) + r * p.xs + c);
    dy.load(static_cast<const T *>(p.dy) + r * p.dys + c);
    if (GATE) z.load(static_cast<const T *>(p.z) + r * p.zs + c);
    place_grad<T, 1, GATE>(p, x, z, dy, w, b, __ldg(p.mean + at), __ldg(p.rstd + at), dxh, xh, sw, sb,
                           static_cast<T *>(nullptr));
  }
  dwp[(size_t)blockIdx.x * p.C + c] = sw.sum();
  dbp[(size_t)blockIdx.x * p.C + c] = sb.sum();
}

// ---------------------------------------------------------------- launches
template <int X> using Int = std::integral_constant<int, X>;
// f(W, NT, V) for the plan's team; PLACES: of a thread of a block that takes a group, 16 bytes at a time
template <int PLACES, class F>
void with_team(const GnPlan &pl, F f) {
  auto width = [&](auto w, auto places) {
    if (pl.places > 1) return pl.team == 32 ? f(w, Int<32>{}, Int<4>{}) : f(w, Int<256>{}, places);
    if (pl.team == 4) return f(w, Int<4>{}, Int<1>{});
    if (pl.team == 8) return f(w, Int<8>{}, Int<1>{});
    if (pl.team == 16) return f(w, Int<16>{}, Int<1>{});
    return f(w, Int<32>{}, Int<1>{});
  };
  if (pl.vec == 8) return width(Int<8>{}, Int<PLACES>{});
  return pl.vec == 2 ? width(Int<2>{}, Int<12>{}) : width(Int<1>{}, Int<12>{});
}
// f(W, V) for the plan's tiles
template <int PLACES, class F>
void with_tile(const GnPlan &pl, F f) {
  if (pl.vec == 8) return f(Int<8>{}, Int<PLACES>{});
  return pl.vec == 2 ? f(Int<2>{}, Int<12>{}) : f(Int<1>{}, Int<12>{});
}

// a launch with `bytes` of dynamic shared memory (with what a kernel has of its own they may pass the 48 KB of a plain
// launch)
template <class... P, class... A>
void launch_smem(void (*kernel)(P...), dim3 grid, int bytes, cudaStream_t s, A... args) {
  if (bytes > 32 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  kernel<<<grid, kThreads, bytes, s>>>(args...);
}

// a launch of clusters of pl.cluster blocks
template <class... P, class... A>
void launch_clusters(void (*kernel)(P...), unsigned grid, const GnPlan &pl, int bytes, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)pl.cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (bytes > 16 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) note_host_error();
}

template <typename T, bool GATE>
void forward(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s) {
  if (pl.tiles == 0) {
    with_team<kForwardPlaces>(pl, [&](auto w, auto nt, auto v) {
      const dim3 grid((p.G + pl.groups_per_block - 1) / pl.groups_per_block,
                      (p.n + pl.samples_per_block - 1) / pl.samples_per_block);
      constexpr int W = decltype(w)::value, NT = decltype(nt)::value, V = decltype(v)::value;
      constexpr int ring = V == 1 ? Ring<T, W, GATE ? 2 : 1>::kBytes : 0;
      SSD_LAUNCH("gn_forward", launch_smem(team_forward_kernel<T, W, NT, V, GATE>, grid, ring, s, p, pl));
    });
    return;
  }
  float *part = reinterpret_cast<float *>(ws + pl.part);
  const unsigned grid = (unsigned)p.n * (pl.cluster ? pl.cluster : pl.tiles) * p.G;
  with_tile<kForwardPlaces>(pl, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    if (pl.cluster) {
      SSD_LAUNCH("gn_forward", launch_clusters(cluster_forward_kernel<T, W, V, GATE>, grid, pl, 0, s, p, pl));
      return;
    }
    SSD_LAUNCH("gn_stats", (tile_stats_kernel<T, W, V><<<grid, kThreads, 0, s>>>(p, pl, part)));
    SSD_LAUNCH("gn_forward", (tile_forward_kernel<T, W, V, GATE><<<grid, kThreads, 0, s>>>(p, pl, part)));
  });
}

template <typename T, bool GATE>
void backward(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s) {
  const bool params = p.dw || p.db, own_columns = pl.own_columns;
  float *dwp = reinterpret_cast<float *>(ws + pl.dwp), *dbp = reinterpret_cast<float *>(ws + pl.dbp);
  float *kw = params && own_columns ? dwp : nullptr;  // partials written by the gradient kernel itself
  if (pl.tiles == 0) {
    with_team<kBackwardPlaces>(pl, [&](auto w, auto nt, auto v) {
      const dim3 grid((p.G + pl.groups_per_block - 1) / pl.groups_per_block,
                      (p.n + pl.samples_per_block - 1) / pl.samples_per_block);
      constexpr int W = decltype(w)::value, NT = decltype(nt)::value, V = decltype(v)::value;
      constexpr int ring = V == 1 ? Ring<T, W, GATE ? 3 : 2>::kBytes : 0, acc = 2 * kThreads * W * 4;
      SSD_LAUNCH("gn_backward", launch_smem(team_backward_kernel<T, W, NT, V, GATE>, grid, ring > acc ? ring : acc, s, p,
                                            pl, kw, dbp));
    });
  } else {
    float *part = reinterpret_cast<float *>(ws + pl.part);
    const unsigned grid = (unsigned)p.n * (pl.cluster ? pl.cluster : pl.tiles) * p.G;
    with_tile<kBackwardPlaces>(pl, [&](auto w, auto v) {
      constexpr int W = decltype(w)::value, V = decltype(v)::value;
      if (pl.cluster) {
        SSD_LAUNCH("gn_backward", launch_clusters(cluster_backward_kernel<T, W, V, GATE>, grid, pl,
                                                  Slots<T, W, (GATE ? 3 : 2) * V>::kBytes, s, p, pl, kw, dbp));
        return;
      }
      SSD_LAUNCH("gn_sums", (tile_sums_kernel<T, W, V, GATE><<<grid, kThreads, 0, s>>>(p, pl, part, kw, dbp)));
      SSD_LAUNCH("gn_backward", (tile_backward_kernel<T, W, V, GATE><<<grid, kThreads, 0, s>>>(p, pl, part)));
    });
  }
  if (!params) return;
  if (!own_columns) {
    const dim3 grid(pl.partials, (p.C + kThreads - 1) / kThreads);
    SSD_LAUNCH("gn_param", (param_kernel<T, GATE><<<grid, kThreads, 0, s>>>(p, dwp, dbp)));
  }
  SSD_LAUNCH("gn_param_sum", launch_gn_param_sum(p.C, pl.partials, dwp, dbp, p.dw, p.db, s));
}

}  // namespace gn
}  // namespace ssd
