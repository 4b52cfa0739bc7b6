// The gated delta rule on CUDA cores: fp32, or widths beyond the tensor-core kernels'.  The formulas are at
// delta.h.
//
// A state's columns do not meet: the chain of chunks takes 32 of them to a block, the state and the chunk's
// matrices in shared memory, every product as tiles of 4 x 2 a thread.  The gradients of q, k and the
// decays, which need whole rows, are a block for each chunk and head, side by side.
#include "delta.h"
#include "simt_gemm.cuh"

namespace ssd {

namespace {

constexpr int kThreads = 256, kCols = 32, kMatLd = kDrC + 4;

template <typename T> __device__ __forceinline__ float load1(const T *p) { return to_f<T>(*p); }

// four values of a row
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

// acc[i][c] += sum_(k < K) A[4 tm + i][k] B[k][2 tn + c], A's rows contiguous along k
__device__ __forceinline__ void mm_nt(float (&acc)[4][2], const float *A, int lda, const float *B, int K, int tm, int tn) {
  A += 4 * tm * lda;
  B += 2 * tn;
#pragma unroll 4
  for (int k = 0; k < K; k += 4) {
    float4 a[4];
    float2 b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(A + i * lda + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = *reinterpret_cast<const float2 *>(B + (k + e) * kCols);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i][0] = fmaf(a[i].x, b[0].x, fmaf(a[i].y, b[1].x, fmaf(a[i].z, b[2].x, fmaf(a[i].w, b[3].x, acc[i][0]))));
      acc[i][1] = fmaf(a[i].x, b[0].y, fmaf(a[i].y, b[1].y, fmaf(a[i].z, b[2].y, fmaf(a[i].w, b[3].y, acc[i][1]))));
    }
  }
}
// acc[i][c] += sum_(j >= j0) A[j][4 tm + i] B[j][2 tn + c] over the chunk's 64 rows; j0 a multiple of 8
__device__ __forceinline__ void mm_tn(float (&acc)[4][2], const float *A, int lda, const float *B, int tm, int tn, int j0 = 0) {
  A += 4 * tm;
  B += 2 * tn;
#pragma unroll 16
  for (int j = j0; j < kDrC; ++j) {
    const float4 a = *reinterpret_cast<const float4 *>(A + j * lda);
    const float2 b = *reinterpret_cast<const float2 *>(B + j * kCols);
    acc[0][0] = fmaf(a.x, b.x, acc[0][0]), acc[0][1] = fmaf(a.x, b.y, acc[0][1]);
    acc[1][0] = fmaf(a.y, b.x, acc[1][0]), acc[1][1] = fmaf(a.y, b.y, acc[1][1]);
    acc[2][0] = fmaf(a.z, b.x, acc[2][0]), acc[2][1] = fmaf(a.z, b.y, acc[2][1]);
    acc[3][0] = fmaf(a.w, b.x, acc[3][0]), acc[3][1] = fmaf(a.w, b.y, acc[3][1]);
  }
}
__device__ __forceinline__ void zero(float (&acc)[4][2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = 0.f;
}

// A chunk's tensors in shared memory: K, Q [64][dk + 4], N, P [64][68], the rows' factors, the state [dk][32],
// three tiles [64][32]
struct ChainShared {
  float *K, *Q, *N, *P, *S, *B1, *B2, *B3;
  DrRows *rows;
  int ld;
  __device__ ChainShared(uint8_t *raw, int dk) {
    rows = reinterpret_cast<DrRows *>(raw);
    float *f = reinterpret_cast<float *>(raw + sizeof(DrRows));
    ld = dk + 4;
    N = f;
    P = N + kDrC * kMatLd;
    S = P + kDrC * kMatLd;
    B1 = S + dk * kCols;
    B2 = B1 + kDrC * kCols;
    B3 = B2 + kDrC * kCols;
    K = B3 + kDrC * kCols;
    Q = K + kDrC * ld;
  }
  static int bytes(int dk) {
    return (int)sizeof(DrRows) + 4 * (2 * kDrC * kMatLd + dk * kCols + 3 * kDrC * kCols + 2 * kDrC * (dk + 4));
  }
};

// four threads to a row
template <typename T>
__device__ __forceinline__ void load_rows(float *dst, int ld, const void *src, long long stride, size_t t0, int n, int h, int dk) {
  const int r = threadIdx.x >> 2;
  const T *from = static_cast<const T *>(src) + (t0 + r) * stride + (size_t)h * dk;
#pragma unroll 4
  for (int c = 4 * (threadIdx.x & 3); c < dk; c += 16)
    *reinterpret_cast<float4 *>(dst + r * ld + c) = r < n ? load4(from + c) : make_float4(0.f, 0.f, 0.f, 0.f);
}
__device__ __forceinline__ void load_mat(float *dst, const float *src) {
#pragma unroll
  for (int e = threadIdx.x; e < kDrC * kDrC / 4; e += kThreads)
    *reinterpret_cast<float4 *>(dst + (e >> 4) * kMatLd + 4 * (e & 15)) = __ldg(reinterpret_cast<const float4 *>(src) + e);
}
__device__ __forceinline__ void load_factors(DrRows *dst, const DrRows *src) {
  for (int e = threadIdx.x; e < (int)(sizeof(DrRows) / 16); e += kThreads)
    reinterpret_cast<float4 *>(dst)[e] = __ldg(reinterpret_cast<const float4 *>(src) + e);
}
// The same in two steps, with the values in registers in between: a chunk's are on their way while the chunk before it
// is worked on (chains of rows of at most 64 channels: beyond, registers do not hold them).  7 sequences, 5003 tokens, 12 heads
// of 64: chains 218 and 413 us; 266 and 474 without, where of a chunk's 15000 cycles 5500 waited for its tensors.
struct RowsAhead {
  float4 x[4];
  template <typename T> __device__ __forceinline__ void load(const void *src, long long stride, size_t t0, int n, int h, int dk) {
    const int r = threadIdx.x >> 2;
    const T *from = static_cast<const T *>(src) + (t0 + r) * stride + (size_t)h * dk;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 4 * (threadIdx.x & 3) + 16 * i;
      x[i] = r < n && c < dk ? load4(from + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void put(float *dst, int ld, int dk) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 4 * (threadIdx.x & 3) + 16 * i;
      if (c < dk) *reinterpret_cast<float4 *>(dst + (threadIdx.x >> 2) * ld + c) = x[i];
    }
  }
};
struct MatAhead {
  float4 x[4];
  __device__ __forceinline__ void load(const float *src) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __ldg(reinterpret_cast<const float4 *>(src) + threadIdx.x + i * kThreads);
  }
  __device__ __forceinline__ void put(float *dst) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = threadIdx.x + i * kThreads;
      *reinterpret_cast<float4 *>(dst + (e >> 4) * kMatLd + 4 * (e & 15)) = x[i];
    }
  }
};
static_assert(4 * kThreads == kDrC * kDrC / 4 && kThreads == 4 * kDrC && sizeof(DrRows) / 16 <= kThreads, "what a thread takes of a chunk");
struct FactorsAhead {
  float4 x;
  __device__ __forceinline__ void load(const DrRows *src) {
    if (threadIdx.x < sizeof(DrRows) / 16) x = __ldg(reinterpret_cast<const float4 *>(src) + threadIdx.x);
  }
  __device__ __forceinline__ void put(DrRows *dst) const {
    if (threadIdx.x < sizeof(DrRows) / 16) reinterpret_cast<float4 *>(dst)[threadIdx.x] = x;
  }
};
// a thread's four rows and two columns of v or do
struct TileAhead {
  float x[4][2];
  template <typename T>
  __device__ __forceinline__ void load(const void *src, long long stride, size_t t0, int n, size_t at, bool live, int tm) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * tm + i;
      const T *from = static_cast<const T *>(src) + (t0 + r) * stride + at;
      x[i][0] = live && r < n ? load1(from) : 0.f;
      x[i][1] = live && r < n ? load1(from + 1) : 0.f;  // dv is even
    }
  }
};

// the block's columns of a state
__device__ __forceinline__ void load_state(float *S, const float *src, int dk, int dv, int c0) {
  for (int e = threadIdx.x; e < dk * kCols; e += kThreads) {
    const int r = e / kCols, c = c0 + e % kCols;
    S[e] = src && c < dv ? src[(size_t)r * dv + c] : 0.f;
  }
}
__device__ __forceinline__ void store_state(float *dst, const float *S, int dk, int dv, int c0) {
  for (int e = threadIdx.x; e < dk * kCols; e += kThreads) {
    const int r = e / kCols, c = c0 + e % kCols;
    if (c < dv) dst[(size_t)r * dv + c] = S[e];
  }
}
// S = e^Gall S + acc in the thread's elements of 64 rows from m0 on
__device__ __forceinline__ void carry(float *S, const float (&acc)[4][2], const DrRows &rows, int m0, int tm, int tn) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 &x = *reinterpret_cast<float2 *>(S + (m0 + 4 * tm + i) * kCols + 2 * tn);
    x.x = fmaf(x.x, rows.all_hi, fmaf(x.x, rows.all_lo, acc[i][0]));
    x.y = fmaf(x.y, rows.all_hi, fmaf(x.y, rows.all_lo, acc[i][1]));
  }
}

// OUT: outputs and the final state; else the states before the chunks and E, for the backward pass
template <typename T, bool OUT, bool AHEAD>
__global__ void __launch_bounds__(kThreads) dr_chain_kernel(DrProblem p, T *__restrict__ o, long long os, float *fin) {
  extern __shared__ __align__(16) uint8_t raw[];
  const ChainShared sm(raw, p.dk);
  const int seq = blockIdx.x / p.H, h = blockIdx.x - seq * p.H, c0 = blockIdx.y * kCols;
  const int tid = threadIdx.x, tm = tid >> 4, tn = tid & 15, col = c0 + 2 * tn;
  const size_t dd = (size_t)p.dk * p.dv;
  int a, len, slot0;
  dr_seq(p, seq, a, len, slot0);
  load_state(sm.S, p.init ? p.init + ((size_t)seq * p.H + h) * dd : nullptr, p.dk, p.dv, c0);
  const DrRows &rows = *sm.rows;
  const int upto = 8 * (tid >> 5) + 8;  // N and P are zero right of the diagonal: the columns of the warp's 8 rows
  RowsAhead ka, qa;
  MatAhead na, pa;
  FactorsAhead fa;
  TileAhead va;
  auto ahead = [&](int c) {
    const size_t t0 = (size_t)a + c * kDrC, at = (size_t)(slot0 + c) * p.H + h;
    const int n = min(kDrC, len - c * kDrC);
    ka.load<T>(p.k, p.ks, t0, n, h / p.group, p.dk);
    na.load(p.N + at * (kDrC * kDrC));
    fa.load(p.rows + at);
    va.load<T>(p.v, p.vs, t0, n, (size_t)h * p.dv + col, col < p.dv, tm);
    if (OUT) {
      qa.load<T>(p.q, p.qs, t0, n, h / p.group, p.dk);
      pa.load(p.P + at * (kDrC * kDrC));
    }
  };
  if (AHEAD && len > 0) ahead(0);
  for (int c = 0; c * kDrC < len; ++c) {
    const size_t t0 = (size_t)a + c * kDrC, at = (size_t)(slot0 + c) * p.H + h;
    const int n = min(kDrC, len - c * kDrC);
    __syncthreads();
    if (AHEAD) {
      ka.put(sm.K, sm.ld, p.dk);
      na.put(sm.N);
      fa.put(sm.rows);
      if (OUT) {
        qa.put(sm.Q, sm.ld, p.dk);
        pa.put(sm.P);
      }
    } else {
      load_rows<T>(sm.K, sm.ld, p.k, p.ks, t0, n, h / p.group, p.dk);
      load_mat(sm.N, p.N + at * (kDrC * kDrC));
      load_factors(sm.rows, p.rows + at);
      if (OUT) {
        load_rows<T>(sm.Q, sm.ld, p.q, p.qs, t0, n, h / p.group, p.dk);
        load_mat(sm.P, p.P + at * (kDrC * kDrC));
      }
      va.load<T>(p.v, p.vs, t0, n, (size_t)h * p.dv + col, col < p.dv, tm);
    }
    if (!OUT) store_state(p.S + at * dd, sm.S, p.dk, p.dv, c0);
    float y[4][2], acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i][0] = va.x[i][0], y[i][1] = va.x[i][1];
    __syncthreads();
    if (AHEAD && (c + 1) * kDrC < len) ahead(c + 1);
    zero(acc);
    mm_nt(acc, sm.K, sm.ld, sm.S, p.dk, tm, tn);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * tm + i;
      y[i][0] = fmaf(-rows.kin[r], acc[i][0], y[i][0]);
      y[i][1] = fmaf(-rows.kin[r], acc[i][1], y[i][1]);
      *reinterpret_cast<float2 *>(sm.B1 + r * kCols + 2 * tn) = make_float2(rows.beta[r] * y[i][0], rows.beta[r] * y[i][1]);
    }
    __syncthreads();
    zero(acc);
    mm_nt(acc, sm.N, kMatLd, sm.B1, upto, tm, tn);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * tm + i;
      const float e0 = y[i][0] - acc[i][0], e1 = y[i][1] - acc[i][1];
      const float2 d = make_float2(rows.beta[r] * e0, rows.beta[r] * e1);
      if (OUT) {
        *reinterpret_cast<float2 *>(sm.B2 + r * kCols + 2 * tn) = d;
      } else if (r < n && col < p.dv) {
        *reinterpret_cast<float2 *>(p.E + ((t0 + r) * p.H + h) * p.dv + col) = make_float2(e0, e1);
      }
      *reinterpret_cast<float2 *>(sm.B3 + r * kCols + 2 * tn) = make_float2(rows.kout[r] * d.x, rows.kout[r] * d.y);
    }
    if (OUT) {
      zero(acc);
      mm_nt(acc, sm.Q, sm.ld, sm.S, p.dk, tm, tn);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][0] *= rows.qin[4 * tm + i];
        acc[i][1] *= rows.qin[4 * tm + i];
      }
    }
    __syncthreads();
    if (OUT) {
      mm_nt(acc, sm.P, kMatLd, sm.B2, upto, tm, tn);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * tm + i;
        if (r < n && col < p.dv) {
          T *to = o + (t0 + r) * os + (size_t)h * p.dv + col;
          to[0] = from_f<T>(acc[i][0]);
          to[1] = from_f<T>(acc[i][1]);
        }
      }
    }
    for (int m0 = 0; m0 < p.dk; m0 += 64) {
      if (m0 + 4 * tm >= p.dk) continue;
      zero(acc);
      mm_tn(acc, sm.K + m0, sm.ld, sm.B3, tm, tn);
      carry(sm.S, acc, rows, m0, tm, tn);
    }
  }
  if (OUT && fin) {
    __syncthreads();
    store_state(fin + ((size_t)seq * p.H + h) * dd, sm.S, p.dk, p.dv, c0);
  }
}

// The chain backwards: Z, the gradients of the states behind the chunks and of the initial state
template <typename T, bool AHEAD>
__global__ void __launch_bounds__(kThreads) dr_reverse_kernel(DrProblem p, const T *__restrict__ dout, long long dos,
                                                              const float *dfin, float *dinit) {
  extern __shared__ __align__(16) uint8_t raw[];
  const ChainShared sm(raw, p.dk);
  const int seq = blockIdx.x / p.H, h = blockIdx.x - seq * p.H, c0 = blockIdx.y * kCols;
  const int tid = threadIdx.x, tm = tid >> 4, tn = tid & 15, col = c0 + 2 * tn;
  const size_t dd = (size_t)p.dk * p.dv;
  int a, len, slot0;
  dr_seq(p, seq, a, len, slot0);
  load_state(sm.S, dfin ? dfin + ((size_t)seq * p.H + h) * dd : nullptr, p.dk, p.dv, c0);
  const DrRows &rows = *sm.rows;
  const int from = 8 * (tid >> 5);  // N and P are zero above the diagonal: the rows of the warp's 8 columns
  RowsAhead ka, qa;
  MatAhead na, pa;
  FactorsAhead fa;
  TileAhead da;
  auto ahead = [&](int c) {
    const size_t t0 = (size_t)a + c * kDrC, at = (size_t)(slot0 + c) * p.H + h;
    const int n = min(kDrC, len - c * kDrC);
    ka.load<T>(p.k, p.ks, t0, n, h / p.group, p.dk);
    pa.load(p.P + at * (kDrC * kDrC));
    fa.load(p.rows + at);
    da.load<T>(dout, dos, t0, n, (size_t)h * p.dv + col, col < p.dv, tm);
    na.load(p.N + at * (kDrC * kDrC));
    qa.load<T>(p.q, p.qs, t0, n, h / p.group, p.dk);
  };
  if (AHEAD && len > 0) ahead((len - 1) / kDrC);
  for (int c = (len - 1) / kDrC; c * kDrC < len && c >= 0; --c) {
    const size_t t0 = (size_t)a + c * kDrC, at = (size_t)(slot0 + c) * p.H + h;
    const int n = min(kDrC, len - c * kDrC);
    __syncthreads();
    if (AHEAD) {
      ka.put(sm.K, sm.ld, p.dk);
      qa.put(sm.Q, sm.ld, p.dk);
      na.put(sm.N);
      pa.put(sm.P);
      fa.put(sm.rows);
    } else {
      load_rows<T>(sm.K, sm.ld, p.k, p.ks, t0, n, h / p.group, p.dk);
      load_rows<T>(sm.Q, sm.ld, p.q, p.qs, t0, n, h / p.group, p.dk);
      load_mat(sm.N, p.N + at * (kDrC * kDrC));
      load_mat(sm.P, p.P + at * (kDrC * kDrC));
      load_factors(sm.rows, p.rows + at);
      da.load<T>(dout, dos, t0, n, (size_t)h * p.dv + col, col < p.dv, tm);
    }
    store_state(p.dS + at * dd, sm.S, p.dk, p.dv, c0);
    float dob[4][2], d[4][2], acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * tm + i;
      dob[i][0] = da.x[i][0], dob[i][1] = da.x[i][1];
      *reinterpret_cast<float2 *>(sm.B3 + r * kCols + 2 * tn) = make_float2(dob[i][0], dob[i][1]);
    }
    __syncthreads();
    if (AHEAD && c > 0) ahead(c - 1);
    zero(d);
    mm_nt(d, sm.K, sm.ld, sm.S, p.dk, tm, tn);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i][0] *= rows.kout[4 * tm + i];
      d[i][1] *= rows.kout[4 * tm + i];
    }
    mm_tn(d, sm.P, kMatLd, sm.B3, tm, tn, from);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * tm + i;
      *reinterpret_cast<float2 *>(sm.B1 + r * kCols + 2 * tn) = make_float2(rows.beta[r] * d[i][0], rows.beta[r] * d[i][1]);
    }
    __syncthreads();
    zero(acc);
    mm_tn(acc, sm.N, kMatLd, sm.B1, tm, tn, from);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * tm + i;
      const float z0 = d[i][0] - acc[i][0], z1 = d[i][1] - acc[i][1], f = -rows.kin[r] * rows.beta[r];
      if (r < n && col < p.dv)
        *reinterpret_cast<float2 *>(p.Z + ((t0 + r) * p.H + h) * p.dv + col) = make_float2(z0, z1);
      *reinterpret_cast<float2 *>(sm.B2 + r * kCols + 2 * tn) = make_float2(f * z0, f * z1);
      *reinterpret_cast<float2 *>(sm.B3 + r * kCols + 2 * tn) = make_float2(rows.qin[r] * dob[i][0], rows.qin[r] * dob[i][1]);
    }
    __syncthreads();
    for (int m0 = 0; m0 < p.dk; m0 += 64) {
      if (m0 + 4 * tm >= p.dk) continue;
      zero(acc);
      mm_tn(acc, sm.Q + m0, sm.ld, sm.B3, tm, tn);
      mm_tn(acc, sm.K + m0, sm.ld, sm.B2, tm, tn);
      carry(sm.S, acc, rows, m0, tm, tn);
    }
  }
  if (dinit) {
    __syncthreads();
    store_state(dinit + ((size_t)seq * p.H + h) * dd, sm.S, p.dk, p.dv, c0);
  }
}

struct GradShared {
  float stage[kGemmSmemFloats];
  float dqk[kDrC][kDrC + 1], dkk[kDrC][kDrC + 1];  // of the products q.k and k.k, decayed
  float pass[kDrC], add[kDrC];                     // what passes to a row, and what a row adds to the state behind the chunk
  float scratch[8 * kDrC];
  DrRows rows;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) dr_grads_kernel(DrProblem p, const T *__restrict__ dout, long long dos, DrGrads g) {
  extern __shared__ __align__(16) uint8_t raw[];
  GradShared &sm = *reinterpret_cast<GradShared *>(raw);
  const int slot = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, tm = tid >> 4, tn = tid & 15;
  int t0, n;
  dr_chunk(p, slot, t0, n);
  if (n == 0) return;
  const int hk = h / p.group, dk = p.dk, dv = p.dv;
  const size_t at = (size_t)slot * p.H + h, dd = (size_t)dk * dv;
  load_factors(&sm.rows, p.rows + at);
  if (tid < kDrC) sm.pass[tid] = sm.add[tid] = 0.f;
  __syncthreads();
  const DrRows &rw = sm.rows;
  const T *q = static_cast<const T *>(p.q) + (size_t)t0 * p.qs + (size_t)hk * dk;
  const T *k = static_cast<const T *>(p.k) + (size_t)t0 * p.ks + (size_t)hk * dk;
  const T *dob_ = dout + (size_t)t0 * dos + (size_t)h * dv;
  const float *E = p.E + ((size_t)t0 * p.H + h) * dv, *Z = p.Z + ((size_t)t0 * p.H + h) * dv;
  const float *S = p.S + at * dd, *dS = p.dS + at * dd;
  const size_t es = (size_t)p.H * dv;
  auto do_r = [&](int i, int c) { return load1(dob_ + i * dos + c); };
  auto dv_r = [&](int i, int c) { return rw.beta[i] * Z[i * es + c]; };
  auto d_r = [&](int i, int c) { return rw.beta[i] * E[i * es + c]; };
  auto d_c = [&](int c, int j) { return rw.beta[j] * E[j * es + c]; };
  auto s_c = [&](int c, int m) { return S[(size_t)m * dv + c]; };
  auto ds_c = [&](int c, int m) { return dS[(size_t)m * dv + c]; };
  auto q_r = [&](int j, int c) { return rw.rq[j] * load1(q + j * p.qs + c); };
  auto k_r = [&](int j, int c) { return rw.rk[j] * load1(k + j * p.ks + c); };

  float acc[4][4];
  zero_acc(acc);
  gemm_tile<true, false>(acc, 0, n, 0, n, 0, dv, do_r, d_c, sm.stage);
  // M: what passes from token c to a later one r.  A comes from the tables (7 sequences, 5003 tokens, 12 heads of 64: 378 us;
  // made here again, by a product of k with k, 402)
  float l[4][4], pairs[4][4];
  auto add_pairs = [&](const float *table, float sign) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = tm * 4 + i, c = tn * 4;
      const float4 x = __ldg(reinterpret_cast<const float4 *>(table + at * (kDrC * kDrC) + r * kDrC + c));
      const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < r && r < n) pairs[i][j] = fmaf(sign * acc[i][j], f[j], pairs[i][j]);
    }
  };
  zero_acc(pairs);
  add_pairs(p.P, 1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = tm * 4 + i, c = tn * 4 + j;
      l[i][j] = c <= r ? expf((rw.ghi[r] - rw.ghi[c]) + (rw.glo[r] - rw.glo[c])) : 0.f;
      sm.dqk[r][c] = c <= r ? acc[i][j] * l[i][j] * p.scale : 0.f;
    }
  zero_acc(acc);
  gemm_tile<true, false>(acc, 0, n, 0, n, 0, dv, dv_r, d_c, sm.stage);
  add_pairs(p.A, -1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = tm * 4 + i, c = tn * 4 + j;
      sm.dkk[r][c] = c < r ? -acc[i][j] * l[i][j] : 0.f;
    }
  // row sums less column sums of the same values: pairs on one side of a token cancel, but for roundings of their own size
  tile_rowsum_add(pairs, sm.pass);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) pairs[i][j] = -pairs[i][j];
  tile_colsum_add(pairs, sm.pass, sm.scratch);
  // rows: dbeta, four threads to a row; dv itself
  {
    const int r = tid >> 2, part = tid & 3;
    float db = 0.f;
    if (r < n)
      for (int c = part; c < dv; c += 4) {
        const float z = Z[r * es + c];
        db = fmaf(E[r * es + c], z, db);
        static_cast<T *>(g.dv)[(size_t)(t0 + r) * g.dvs + (size_t)h * dv + c] = from_f<T>(rw.beta[r] * z);
      }
#pragma unroll
    for (int o = 2; o >= 1; o >>= 1) db += __shfl_xor_sync(0xffffffffu, db, o);
    if (part == 0 && r < n) static_cast<T *>(g.db)[(size_t)(t0 + r) * g.dbs + h] = from_f<T>(db);
  }
  float in_r[4], out_r[4], qin_r[4];  // e^G and e^(Gall - G) of the thread's rows, without lengths
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = tm * 4 + i;
    in_r[i] = r < n ? rw.kin[r] / rw.rk[r] : 0.f;
    out_r[i] = r < n ? rw.kout[r] / rw.rk[r] : 0.f;
    qin_r[i] = r < n ? rw.qin[r] / rw.rq[r] : 0.f;
  }
  auto dqk_r = [&](int i, int j) { return sm.dqk[i][j]; };
  auto dqk_t = [&](int i, int j) { return sm.dqk[j][i]; };
  auto dkk_b = [&](int i, int j) { return sm.dkk[i][j] + sm.dkk[j][i]; };
  __syncthreads();
  for (int n0 = 0; n0 < dk; n0 += kTile) {
    zero_acc(acc);
    gemm_tile<true, false>(acc, 0, n, n0, dk, 0, dv, do_r, s_c, sm.stage);
    float dots[4][4];  // what is read of the state before the chunk, less what is written over
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = tm * 4 + i, c = n0 + tn * 4 + j;
        acc[i][j] *= qin_r[i];
        dots[i][j] = r < n && c < dk ? acc[i][j] * q_r(r, c) : 0.f;
      }
    gemm_tile<true, true>(acc, 0, n, n0, dk, 0, n, dqk_r, k_r, sm.stage);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = tm * 4 + i, c = n0 + tn * 4 + j;
        if (r < n && c < dk) p.dqp[((size_t)(t0 + r) * p.H + h) * dk + c] = acc[i][j];
      }
    float upd[4][4];
    zero_acc(upd);
    gemm_tile<true, false>(upd, 0, n, n0, dk, 0, dv, d_r, ds_c, sm.stage);
    zero_acc(acc);
    gemm_tile<true, false>(acc, 0, n, n0, dk, 0, dv, dv_r, s_c, sm.stage);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = tm * 4 + i, c = n0 + tn * 4 + j;
        const float u = out_r[i] * upd[i][j], kv = r < n && c < dk ? k_r(r, c) : 0.f, over = in_r[i] * acc[i][j];
        upd[i][j] = u * kv;
        dots[i][j] = fmaf(-over, kv, dots[i][j]);
        acc[i][j] = u - over;
      }
    tile_rowsum_add(dots, sm.pass);
    tile_rowsum_add(upd, sm.add);
    gemm_tile<false, true>(acc, 0, n, n0, dk, 0, n, dqk_t, q_r, sm.stage);
    gemm_tile<true, true>(acc, 0, n, n0, dk, 0, n, dkk_b, k_r, sm.stage);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = tm * 4 + i, c = n0 + tn * 4 + j;
        if (r < n && c < dk) p.dkp[((size_t)(t0 + r) * p.H + h) * dk + c] = acc[i][j];
      }
  }
  float ss = 0.f;
  for (int e = tid; e < (int)dd; e += kThreads) ss = fmaf(S[e], dS[e], ss);
  ss = block_sum256(ss, sm.scratch) * (rw.all_hi + rw.all_lo);
  if (tid < n) {
    float to = 0.f, behind = 0.f;
    for (int i = n - 1; i >= tid; --i) to += sm.pass[i];
    for (int j = 0; j < tid; ++j) behind += sm.add[j];
    static_cast<T *>(g.dg)[(size_t)(t0 + tid) * g.dgs + h] = from_f<T>(to + behind + ss);
  }
}

// dq (y = 0) and dk (1): a warp to a row of one head of q and k
template <typename T> __global__ void __launch_bounds__(kThreads) dr_finish_kernel(DrProblem p, DrGrads g) {
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (long long)p.total * p.Hk) return;
  const long long t = w / p.Hk;
  const int hk = (int)(w - t * p.Hk);
  if (p.cu) {  // rows outside every sequence stay as they are
    int lo = 0, hi = p.nseq;  // the first bound behind t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) > t)
        hi = mid;
      else
        lo = mid + 1;
    }
    if (lo == 0 || lo > p.nseq || __ldg(p.cu + p.nseq) <= t) return;
  }
  const bool is_k = blockIdx.y != 0;
  const T *x = is_k ? static_cast<const T *>(p.k) + t * p.ks : static_cast<const T *>(p.q) + t * p.qs;
  T *to = is_k ? static_cast<T *>(g.dk) + t * g.dks : static_cast<T *>(g.dq) + t * g.dqs;
  const float *from = (is_k ? p.dkp : p.dqp) + ((size_t)t * p.H + (size_t)hk * p.group) * p.dk;
  x += (size_t)hk * p.dk;
  to += (size_t)hk * p.dk;
  constexpr int kPer = 8;  // 256 / 32
  float d[kPer], u[kPer], xx = 0.f, xd = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int c = lane + 32 * e;
    d[e] = u[e] = 0.f;
    if (c < p.dk) {
      for (int y = 0; y < p.group; ++y) d[e] += from[(size_t)y * p.dk + c];
      u[e] = load1(x + c);
    }
    xx = fmaf(u[e], u[e], xx);
    xd = fmaf(u[e], d[e], xd);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    xx += __shfl_xor_sync(0xffffffffu, xx, o);
    xd += __shfl_xor_sync(0xffffffffu, xd, o);
  }
  const float r = p.norm ? 1.f / sqrtf(xx + p.eps) : 1.f, f = p.norm ? xd * r * r : 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int c = lane + 32 * e;
    if (c < p.dk) to[c] = from_f<T>(r * (d[e] - u[e] * f));
  }
}

dim3 chain_grid(const DrProblem &p) { return dim3((unsigned)(p.nseq * p.H), (unsigned)((p.dv + kCols - 1) / kCols)); }

template <typename T, bool OUT, bool AHEAD> void run_chain(const DrProblem &p, T *o, long long os, float *fin, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(dr_chain_kernel<T, OUT, AHEAD>), ChainShared::bytes(256), allowed);
  dr_chain_kernel<T, OUT, AHEAD><<<chain_grid(p), kThreads, ChainShared::bytes(p.dk), s>>>(p, o, os, fin);
}
template <typename T, bool AHEAD>
void run_reverse(const DrProblem &p, const T *dout, long long dos, const float *dfin, float *dinit, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(dr_reverse_kernel<T, AHEAD>), ChainShared::bytes(256), allowed);
  dr_reverse_kernel<T, AHEAD><<<chain_grid(p), kThreads, ChainShared::bytes(p.dk), s>>>(p, dout, dos, dfin, dinit);
}
constexpr int kAheadWidth = 64;  // of RowsAhead

}  // namespace

template <typename T> void launch_dr_chain(const DrProblem &p, void *o, long long os, float *fin, cudaStream_t s) {
  T *to = static_cast<T *>(o);
  if (p.dk <= kAheadWidth)
    o ? run_chain<T, true, true>(p, to, os, fin, s) : run_chain<T, false, true>(p, nullptr, 0, nullptr, s);
  else
    o ? run_chain<T, true, false>(p, to, os, fin, s) : run_chain<T, false, false>(p, nullptr, 0, nullptr, s);
}

template <typename T>
void launch_dr_reverse(const DrProblem &p, const void *dout, long long dos, const float *dfin, float *dinit, cudaStream_t s) {
  const T *from = static_cast<const T *>(dout);
  p.dk <= kAheadWidth ? run_reverse<T, true>(p, from, dos, dfin, dinit, s) : run_reverse<T, false>(p, from, dos, dfin, dinit, s);
}

template <typename T>
void launch_dr_grads(const DrProblem &p, const void *dout, long long dos, const DrGrads &g, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(dr_grads_kernel<T>), sizeof(GradShared), allowed);
  dr_grads_kernel<T><<<dim3((unsigned)p.slots, (unsigned)p.H), kThreads, sizeof(GradShared), s>>>(p, static_cast<const T *>(dout), dos, g);
}

template <typename T> void launch_dr_finish(const DrProblem &p, const DrGrads &g, cudaStream_t s) {
  const long long warps = (long long)p.total * p.Hk;
  dr_finish_kernel<T><<<dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)), 2), kThreads, 0, s>>>(p, g);
}

#define SSD_DR_TYPES(T)                                                                                            \
  template void launch_dr_chain<T>(const DrProblem &, void *, long long, float *, cudaStream_t);                   \
  template void launch_dr_reverse<T>(const DrProblem &, const void *, long long, const float *, float *, cudaStream_t); \
  template void launch_dr_grads<T>(const DrProblem &, const void *, long long, const DrGrads &, cudaStream_t);     \
  template void launch_dr_finish<T>(const DrProblem &, const DrGrads &, cudaStream_t);
SSD_DR_TYPES(float)
SSD_DR_TYPES(__nv_bfloat16)

}  // namespace ssd
