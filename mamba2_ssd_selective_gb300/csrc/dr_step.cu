// The gated delta rule, one token of each row against a cache of states:
//     S' = a S[slot],   d = beta (v - k S'),   S[slot] = S' + k^T d,   o = scale q S[slot]
// The state is read and written once, and that traffic is the bound.  Both sums over the state's rows (k S' and q S') are
// taken in one pass before the update, since q S[slot] = q S' + (q.k) d; the lengths of q and k and q.k ride along.
// Two kernels.  Many states of usual widths: a block on each SM goes through whole states, which bulk copies bring to
// shared memory and back, two on their way in while one is worked on.  Else a block takes 64 or 32 columns of one state, the
// layout of la_step.cu, all of a thread's elements in registers.  Between its loads and its stores stands a sum over the
// block, so that its memory is idle for a while: 256 rows, 32 heads of 128 x 128 took 235 us with it, and take 165 us
// (6.5 TB/s) with the first.
#include <type_traits>

#include "delta.h"
#include "tc_pipe.cuh"

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

constexpr int kStages = 3;
template <typename T> __host__ __device__ constexpr int vector_bytes(int dk, int dv) { return (2 * dk + dv) * (int)sizeof(T); }
template <typename T> __host__ __device__ constexpr int stage_bytes(int dk, int dv) {
  return (dk * dv * 4 + vector_bytes<T>(dk, dv) + 127) / 128 * 128;
}

// Whole states of dk (at most 128) x DV in a ring of stages: the state, then q, k and v.  A warp has rows of its own.
template <typename T, int DV>
__global__ void __launch_bounds__(kThreads, 1) dr_step_ring_kernel(DrProblem p, T *__restrict__ o, long long os,
                                                                   float *__restrict__ states, int nslots,
                                                                   const int *__restrict__ slot_idx) {
  constexpr int kLanes = DV / 4, kRows = kThreads / kLanes, kSweeps = 128 / kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kStages];
  __shared__ __align__(16) float part[2][kWarps][DV];
  __shared__ float dots[kWarps][4];
  const int tid = threadIdx.x, lc = tid % kLanes, a0 = tid / kLanes, c = 4 * lc;
  const int dk = p.dk, items = p.nseq * p.H, stage = stage_bytes<T>(dk, DV), sbytes = dk * DV * 4;
  auto slot_of = [&](int item) {
    const int r = item / p.H, s = slot_idx ? __ldg(slot_idx + r) : r;
    return s >= 0 && s < nslots ? s : -1;
  };
  auto fetch = [&](int item, int s) {  // thread 0
    const int r = item / p.H, h = item - r * p.H, slot = slot_of(item);
    uint8_t *to = smem + s * stage;
    sm100::mbar_expect_tx(&full[s], (slot >= 0 ? sbytes : 0) + vector_bytes<T>(dk, DV));
    if (slot >= 0) pipe::bulk_load(to, states + ((size_t)slot * p.H + h) * ((size_t)dk * DV), sbytes, &full[s]);
    to += sbytes;
    pipe::bulk_load(to, static_cast<const T *>(p.q) + r * p.qs + (size_t)(h / p.group) * dk, dk * sizeof(T), &full[s]);
    pipe::bulk_load(to + dk * sizeof(T), static_cast<const T *>(p.k) + r * p.ks + (size_t)(h / p.group) * dk, dk * sizeof(T), &full[s]);
    pipe::bulk_load(to + 2 * dk * sizeof(T), static_cast<const T *>(p.v) + r * p.vs + (size_t)h * DV, DV * sizeof(T), &full[s]);
  };
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) sm100::mbar_init(&full[s], 1);
    sm100::fence_mbar_init();
    for (int s = 0; s + 1 < kStages; ++s)
      if (blockIdx.x + s * gridDim.x < items) fetch(blockIdx.x + s * gridDim.x, s);
  }
  __syncthreads();
  int it = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x, ++it) {
    const int s = it % kStages, r = item / p.H, h = item - r * p.H;
    const bool live = slot_of(item) >= 0;
    const float g = load1(static_cast<const T *>(p.g) + r * p.gs + h), beta = load1(static_cast<const T *>(p.b) + r * p.bs + h);
    float4 *st = reinterpret_cast<float4 *>(smem + s * stage);
    const T *q = reinterpret_cast<const T *>(smem + s * stage + sbytes), *k = q + dk, *v = k + dk;
    sm100::mbar_wait_drain(&full[s], (it / kStages) & 1);
    T *out = o + r * os + (size_t)h * DV;
    float4 x[kSweeps];
    float kv[kSweeps], sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f}, kk = 0.f, qk = 0.f, qq = 0.f;
    if (live) {
#pragma unroll
      for (int i = 0; i < kSweeps; ++i) {
        const int a = a0 + kRows * i;
        x[i] = a < dk ? st[a * kLanes + lc] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kSweeps; ++i) {
        const int a = a0 + kRows * i;
        const float qv = a < dk ? load1(q + a) : 0.f;
        kv[i] = a < dk ? load1(k + a) : 0.f;
        kk = fmaf(kv[i], kv[i], kk);
        qk = fmaf(kv[i], qv, qk);
        qq = fmaf(qv, qv, qq);
        sk[0] = fmaf(kv[i], x[i].x, sk[0]), sk[1] = fmaf(kv[i], x[i].y, sk[1]);
        sk[2] = fmaf(kv[i], x[i].z, sk[2]), sk[3] = fmaf(kv[i], x[i].w, sk[3]);
        sq[0] = fmaf(qv, x[i].x, sq[0]), sq[1] = fmaf(qv, x[i].y, sq[1]);
        sq[2] = fmaf(qv, x[i].z, sq[2]), sq[3] = fmaf(qv, x[i].w, sq[3]);
      }
      if (kLanes < 32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sk[j] += __shfl_xor_sync(0xffffffffu, sk[j], 16);
          sq[j] += __shfl_xor_sync(0xffffffffu, sq[j], 16);
        }
        kk += __shfl_xor_sync(0xffffffffu, kk, 16);
        qk += __shfl_xor_sync(0xffffffffu, qk, 16);
        qq += __shfl_xor_sync(0xffffffffu, qq, 16);
      }
      if ((tid & 31) < kLanes) {
        *reinterpret_cast<float4 *>(&part[0][tid >> 5][c]) = make_float4(sk[0], sk[1], sk[2], sk[3]);
        *reinterpret_cast<float4 *>(&part[1][tid >> 5][c]) = make_float4(sq[0], sq[1], sq[2], sq[3]);
      }
      if ((tid & 31) == 0) {
        dots[tid >> 5][0] = kk;
        dots[tid >> 5][1] = qk;
        dots[tid >> 5][2] = qq;
      }
    }
    __syncthreads();
    if (live) {
      kk = qk = qq = 0.f;
      float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        kk += dots[w][0];
        qk += dots[w][1];
        qq += dots[w][2];
        const float4 y = *reinterpret_cast<const float4 *>(&part[0][w][c]);
        k4.x += y.x, k4.y += y.y, k4.z += y.z, k4.w += y.w;
      }
      const float rk = p.norm ? 1.f / sqrtf(kk + p.eps) : 1.f, rq = p.norm ? 1.f / sqrtf(qq + p.eps) : 1.f;
      const float2 lam = step_decay(g);
      auto low = [&](float y) { return fmaf(y, lam.x, y * lam.y); };
      const float d[4] = {beta * (load1(v + c) - rk * low(k4.x)), beta * (load1(v + c + 1) - rk * low(k4.y)),
                          beta * (load1(v + c + 2) - rk * low(k4.z)), beta * (load1(v + c + 3) - rk * low(k4.w))};
#pragma unroll
      for (int i = 0; i < kSweeps; ++i) {
        const int a = a0 + kRows * i;
        if (a < dk) {
          const float u = rk * kv[i];
          x[i].x = fmaf(x[i].x, lam.x, fmaf(x[i].x, lam.y, u * d[0]));
          x[i].y = fmaf(x[i].y, lam.x, fmaf(x[i].y, lam.y, u * d[1]));
          x[i].z = fmaf(x[i].z, lam.x, fmaf(x[i].z, lam.y, u * d[2]));
          x[i].w = fmaf(x[i].w, lam.x, fmaf(x[i].w, lam.y, u * d[3]));
          st[a * kLanes + lc] = x[i];
        }
      }
      if (tid < kLanes) {
        float4 q4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 y = *reinterpret_cast<const float4 *>(&part[1][w][c]);
          q4.x += y.x, q4.y += y.y, q4.z += y.z, q4.w += y.w;
        }
        const float f = rk * qk, sc = p.scale * rq;
        const float y[4] = {sc * (low(q4.x) + f * d[0]), sc * (low(q4.y) + f * d[1]), sc * (low(q4.z) + f * d[2]), sc * (low(q4.w) + f * d[3])};
#pragma unroll
        for (int e = 0; e < 4; ++e) out[c + e] = from_f<T>(y[e]);
      }
    } else if (tid < DV) {
      out[tid] = from_f<T>(0.f);
    }
    sm100::fence_async_smem();
    __syncthreads();
    if (tid == 0) {
      if (live) pipe::bulk_store(states + ((size_t)slot_of(item) * p.H + h) * ((size_t)dk * DV), sm100::smem_u32(st), sbytes);
      sm100::bulk_commit();
      // the stage of the state before this one: its store has read it
      asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      const long long next = (long long)item + (kStages - 1) * (long long)gridDim.x;
      if (next < items) fetch((int)next, (it + kStages - 1) % kStages);
    }
  }
  if (tid == 0) sm100::bulk_wait0();
}

template <typename T, int DV>
void run_ring(const DrProblem &p, void *o, long long os, float *states, int nslots, const int *slot_idx, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(dr_step_ring_kernel<T, DV>), kStages * stage_bytes<T>(128, DV), allowed);
  const int items = p.nseq * p.H, sms = device_sm_count();
  dr_step_ring_kernel<T, DV><<<items < sms ? items : sms, kThreads, kStages * stage_bytes<T>(p.dk, DV), s>>>(
      p, static_cast<T *>(o), os, states, nslots, slot_idx);
}

template <typename T, int COLS, int SWEEPS>
void run_step(const DrProblem &p, void *o, long long os, float *states, int nslots, const int *slot_idx, cudaStream_t s) {
  const dim3 grid((unsigned)p.nseq * ((p.dv + COLS - 1) / COLS), p.H);
  dr_step_kernel<T, COLS, SWEEPS><<<grid, kThreads, 0, s>>>(p, static_cast<T *>(o), os, states, nslots, slot_idx);
}

}  // namespace

template <typename T>
void launch_dr_step(const DrProblem &p, void *o, long long os, float *states, int nslots, const int *slot_idx, cudaStream_t s) {
  // the ring needs a few states for each SM
  if ((p.dv == 64 || p.dv == 128) && p.dk <= 128 && (long long)p.nseq * p.H >= 8 * 152) {
    p.dv == 64 ? run_ring<T, 64>(p, o, os, states, nslots, slot_idx, s) : run_ring<T, 128>(p, o, os, states, nslots, slot_idx, s);
    return;
  }
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
