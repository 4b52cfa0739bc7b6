// Group norm with an activation, channels last.  Per sample and group:
//     xhat = (x - mean) rstd,  u = xhat w + b,  y = u | u sigmoid(u) | u z sigmoid(z)
// and backwards, with du the gradient of u and M = rows * channels of the group:
//     dx = rstd (du w - sum(du w) / M - xhat sum(du w xhat) / M)
//     dw = sum du xhat,  db = sum du,  dz = dy u silu'(z)
// One block of 256 threads for each (sample, group); sums in a fixed order.
#include "group_norm.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kTileRows = 256;  // rows of a dweight / dbias partial

__device__ __forceinline__ float2 block_sum2(float a, float b, float *scratch) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    scratch[threadIdx.x >> 5] = a;
    scratch[8 + (threadIdx.x >> 5)] = b;
  }
  __syncthreads();
  a = b = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    a += scratch[w];
    b += scratch[8 + w];
  }
  return make_float2(a, b);
}

template <typename T>
struct Row {
  const T *p;
  long long s;
  __device__ float at(long long row, int c) const { return to_f<T>(p[row * s + c]); }
};

// du and the gate's gradient from dy
template <int ACT>
__device__ __forceinline__ float act_grad(float dy, float u, float z, float &dz) {
  if (ACT == SSD_ACT_NONE) return dy;
  const float a = ACT == SSD_ACT_SILU ? u : z, p = sigmoid_f(a), slope = p * (1.f + a * (1.f - p));
  if (ACT == SSD_ACT_SILU) return dy * slope;
  dz = dy * u * slope;
  return dy * z * p;
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads) gn_forward_kernel(GnProblem p) {
  __shared__ float red[16];
  const int n = blockIdx.x / p.G, g = blockIdx.x % p.G, c0 = g * p.cg;
  const long long row0 = (long long)n * p.m, M = (long long)p.m * p.cg;
  const Row<T> x{static_cast<const T *>(p.x) + c0, p.xs}, z{static_cast<const T *>(p.z) + c0, p.zs};
  float s = 0.f;
  for (long long e = threadIdx.x; e < M; e += kThreads) s += x.at(row0 + e / p.cg, e % p.cg);
  const float mean = block_sum2(s, 0.f, red).x / M;
  s = 0.f;
  for (long long e = threadIdx.x; e < M; e += kThreads) {
    const float d = x.at(row0 + e / p.cg, e % p.cg) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = 1.f / sqrtf(block_sum2(s, 0.f, red).x / M + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[blockIdx.x] = mean;
    if (p.rstd) p.rstd[blockIdx.x] = rstd;
  }
  T *y = static_cast<T *>(p.y) + c0;
  for (long long e = threadIdx.x; e < M; e += kThreads) {
    const long long row = row0 + e / p.cg;
    const int c = e % p.cg;
    float u = (x.at(row, c) - mean) * rstd;
    u = fmaf(u, p.w ? p.w[c0 + c] : 1.f, p.b ? p.b[c0 + c] : 0.f);
    if (ACT == SSD_ACT_SILU) u *= sigmoid_f(u);
    if (ACT == SSD_ACT_GATE) {
      const float zz = z.at(row, c);
      u *= zz * sigmoid_f(zz);
    }
    y[row * p.ys + c] = from_f<T>(u);
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads) gn_backward_kernel(GnProblem p) {
  __shared__ float red[16];
  const int n = blockIdx.x / p.G, g = blockIdx.x % p.G, c0 = g * p.cg;
  const long long row0 = (long long)n * p.m, M = (long long)p.m * p.cg;
  const Row<T> x{static_cast<const T *>(p.x) + c0, p.xs}, z{static_cast<const T *>(p.z) + c0, p.zs},
      dy{static_cast<const T *>(p.dy) + c0, p.dys};
  const float mean = p.mean[blockIdx.x], rstd = p.rstd[blockIdx.x];
  float sa = 0.f, sb = 0.f, a = 0.f, b = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (long long e = threadIdx.x; e < M; e += kThreads) {
      const long long row = row0 + e / p.cg;
      const int c = e % p.cg;
      const float w = p.w ? p.w[c0 + c] : 1.f, xh = (x.at(row, c) - mean) * rstd;
      const float u = fmaf(xh, w, p.b ? p.b[c0 + c] : 0.f);
      float dz = 0.f;
      const float du = act_grad<ACT>(dy.at(row, c), u, ACT == SSD_ACT_GATE ? z.at(row, c) : 0.f, dz) * w;
      if (pass == 0) {
        sa += du;
        sb = fmaf(du, xh, sb);
      } else {
        static_cast<T *>(p.dx)[row * p.dxs + c0 + c] = from_f<T>(rstd * (du - a - xh * b));
        if (ACT == SSD_ACT_GATE) static_cast<T *>(p.dz)[row * p.dzs + c0 + c] = from_f<T>(dz);
      }
    }
    if (pass == 0) {
      const float2 s = block_sum2(sa, sb, red);
      a = s.x / M;
      b = s.y / M;
    }
  }
}

// partial dweight and dbias of a tile of rows, a thread per channel
template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads) gn_param_kernel(GnProblem p, float *dwp, float *dbp) {
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= p.C) return;
  const long long rows = (long long)p.n * p.m, r0 = (long long)blockIdx.x * kTileRows;
  const Row<T> x{static_cast<const T *>(p.x), p.xs}, z{static_cast<const T *>(p.z), p.zs},
      dy{static_cast<const T *>(p.dy), p.dys};
  const float w = p.w ? p.w[c] : 1.f, b = p.b ? p.b[c] : 0.f;
  float sw = 0.f, sb = 0.f;
  for (long long r = r0; r < min(rows, r0 + kTileRows); ++r) {
    const long long at = r / p.m * p.G + c / p.cg;
    const float xh = (x.at(r, c) - p.mean[at]) * p.rstd[at];
    float dz;
    const float du = act_grad<ACT>(dy.at(r, c), fmaf(xh, w, b), ACT == SSD_ACT_GATE ? z.at(r, c) : 0.f, dz);
    sw = fmaf(du, xh, sw);
    sb += du;
  }
  dwp[(size_t)blockIdx.x * p.C + c] = sw;
  dbp[(size_t)blockIdx.x * p.C + c] = sb;
}

__global__ void __launch_bounds__(kThreads) gn_param_sum_kernel(int C, int tiles, const float *dwp, const float *dbp,
                                                                float *dw, float *db) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= C) return;
  float sw = 0.f, sb = 0.f;
  for (int t = 0; t < tiles; ++t) {
    sw += dwp[(size_t)t * C + c];
    sb += dbp[(size_t)t * C + c];
  }
  if (dw) dw[c] = sw;
  if (db) db[c] = sb;
}

template <typename T, int ACT>
void gn_backward(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s) {
  SSD_LAUNCH("gn_backward", (gn_backward_kernel<T, ACT><<<p.n * p.G, kThreads, 0, s>>>(p)));
  if (!p.dw && !p.db) return;
  float *dwp = reinterpret_cast<float *>(ws + pl.dwp), *dbp = reinterpret_cast<float *>(ws + pl.dbp);
  const dim3 grid(pl.tiles, (p.C + kThreads - 1) / kThreads);
  SSD_LAUNCH("gn_param", (gn_param_kernel<T, ACT><<<grid, kThreads, 0, s>>>(p, dwp, dbp)));
  SSD_LAUNCH("gn_param_sum",
             (gn_param_sum_kernel<<<(p.C + kThreads - 1) / kThreads, kThreads, 0, s>>>(p.C, pl.tiles, dwp, dbp, p.dw, p.db)));
}

}  // namespace

GnPlan gn_plan(const GnProblem &p, bool backward) {
  GnPlan pl{};
  pl.tiles = (int)(((long long)p.n * p.m + kTileRows - 1) / kTileRows);
  size_t off = 256;  // never empty
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  pl.dwp = take(backward ? (size_t)pl.tiles * p.C * 4 : 0);
  pl.dbp = take(backward ? (size_t)pl.tiles * p.C * 4 : 0);
  pl.total = off;
  return pl;
}

template <typename T>
void run_gn_forward(const GnProblem &p, const GnPlan &, char *, cudaStream_t s) {
  if (p.act == SSD_ACT_NONE)
    SSD_LAUNCH("gn_forward", (gn_forward_kernel<T, SSD_ACT_NONE><<<p.n * p.G, kThreads, 0, s>>>(p)));
  else if (p.act == SSD_ACT_SILU)
    SSD_LAUNCH("gn_forward", (gn_forward_kernel<T, SSD_ACT_SILU><<<p.n * p.G, kThreads, 0, s>>>(p)));
  else
    SSD_LAUNCH("gn_forward", (gn_forward_kernel<T, SSD_ACT_GATE><<<p.n * p.G, kThreads, 0, s>>>(p)));
}

template <typename T>
void run_gn_backward(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s) {
  if (p.act == SSD_ACT_NONE)
    gn_backward<T, SSD_ACT_NONE>(p, pl, ws, s);
  else if (p.act == SSD_ACT_SILU)
    gn_backward<T, SSD_ACT_SILU>(p, pl, ws, s);
  else
    gn_backward<T, SSD_ACT_GATE>(p, pl, ws, s);
}

template void run_gn_forward<float>(const GnProblem &, const GnPlan &, char *, cudaStream_t);
template void run_gn_forward<__nv_bfloat16>(const GnProblem &, const GnPlan &, char *, cudaStream_t);
template void run_gn_backward<float>(const GnProblem &, const GnPlan &, char *, cudaStream_t);
template void run_gn_backward<__nv_bfloat16>(const GnProblem &, const GnPlan &, char *, cudaStream_t);

}  // namespace ssd
