// Linear attention with a decay for each head on the CUDA cores: fp32 tensors,
// and widths outside the tensor-core kernel's envelope.
//
// A block of 128 threads takes one segment of one sequence, one query head and
// 64 columns of v, and walks the segment in blocks of 32 tokens with the state's
// columns S (dk x 64) in shared memory:
//     A_ij = q_i . k_j lam^|i - j|          (j <= i; reverse: j >= i)
//     o_i  = lam^a(i) q_i S + sum_j A_ij v_j
//     S    = lam^nv S + sum_j lam^b(j) k_j^T v_j
// q and k are staged transposed, so that every product reads its operands as
// float4; sums are fp32 in a fixed order.
// Shared memory bounds it: a thread's tile of 4 x 4 (o) or 8 x 4 (S) reads two or three float4 for 16 or 32
// products, and a float4 takes its pipe four turns even where lanes read the same one.  Backward of 5003
// packed tokens, 12 heads of 64 with 4 key/value heads: 198 us for the three passes, the pipe busy 65% of the
// time, FMA 33%; 54 us for the segments' states.  Blocks of 64 tokens would halve the reads of o's and S's
// tiles, but double A's products, and leave two blocks of threads to an SM instead of four.
#include "retention.h"

namespace ssd {

namespace {

constexpr int kC = 32;        // tokens of a block
constexpr int kLdC = kC + 4;  // padded row of q, k, A (floats), float4 aligned
constexpr int kTV = 64;       // columns of v
constexpr int kLdV = kTV + 4;
constexpr int kThreads = 128;

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&v)[4]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2 *>(p) =
      make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Rows [0, nv) of (kC x d) tiles of two token-major tensors (SUMMARY: of the second only), transposed into
// dst[d][kLdC]; rows past nv are zero.  All of a turn's loads are issued before the first is used.
template <typename T, bool SUMMARY>
__device__ __forceinline__ void stage_transposed(float *qt, const T *q, long long qs, float *kt, const T *k, long long ks,
                                                 int nv, int d) {
  constexpr int kWarps = kThreads / 32;
  const int r = threadIdx.x & 31;
  for (int x0 = threadIdx.x >> 5; x0 < d / 8; x0 += 2 * kWarps) {
    float a[2][8] = {}, b[2][8] = {};
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int x = x0 + y * kWarps;
      if (r < nv && x < d / 8) {
        if (!SUMMARY) load8(q + (long long)r * qs + 8 * x, a[y]);
        load8(k + (long long)r * ks + 8 * x, b[y]);
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int x = x0 + y * kWarps;
      if (x < d / 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!SUMMARY) qt[(8 * x + i) * kLdC + r] = a[y][i];
          kt[(8 * x + i) * kLdC + r] = b[y][i];
        }
      }
    }
  }
}

template <typename T, bool SUMMARY>
__global__ void __launch_bounds__(kThreads, SUMMARY ? 5 : 4) la_simt_kernel(LaPlanDev pl, const __grid_constant__ LaBatch batch) {
  extern __shared__ __align__(16) float sm[];
  const int unit = blockIdx.x;
  if (unit >= la_units(pl)) return;
  const LaPass &p = batch.p[blockIdx.z % batch.n];
  const int tile = blockIdx.z / batch.n, c0 = tile * kTV;
  if (c0 >= p.dv) return;  // passes of a batch may differ in width
  const bool rev = p.reverse;
  const LaUnit u = la_unit(pl, unit, rev);
  if (SUMMARY && u.next < 0) return;  // nothing follows
  const int dkp = (p.dk + 63) & ~63;
  float *Qt = sm, *Kt = SUMMARY ? sm : Qt + dkp * kLdC, *S = Kt + dkp * kLdC, *V = S + dkp * kLdV, *At = V + kC * kLdV,
        *pw = SUMMARY ? At : At + kC * kLdC;  // pw[0..kC]: lam^n
  const float p_scale = p.o_scale * p.p_scale;
  const int h = blockIdx.y, tid = threadIdx.x, ncol = min(kTV, p.dv - c0);
  const float g = __ldg(p.g + h);
  const T *q = static_cast<const T *>(p.q) + u.t0 * p.qs + (h / p.gq) * p.dk;
  const T *k = static_cast<const T *>(p.k) + u.t0 * p.ks + (h / p.gk) * p.dk;
  const T *v = static_cast<const T *>(p.v) + u.t0 * p.vs + (h / p.gv) * p.dv + c0;

  if (tid <= kC) pw[tid] = la_pow(g, tid);
  const float2 carry_full = la_pow2(g, kC);
  // q and k rows past dk (up to the padded width) stay zero
  for (int e = p.dk * kLdC + tid; e < dkp * kLdC; e += kThreads) {
    if (!SUMMARY) Qt[e] = 0.f;
    Kt[e] = 0.f;
  }
  {
    int sa, sb;
    const float *in = SUMMARY ? nullptr : la_state_in(p, u.level, u.next, u.seq, unit, h, sa, sb);
    for (int e = tid; e < dkp * kTV; e += kThreads) {
      const int a = e / kTV, b = e % kTV;
      S[a * kLdV + b] = in && a < p.dk && b < ncol ? in[(size_t)a * sa + (size_t)(c0 + b) * sb] : 0.f;
    }
  }
  const int nb = (u.len + kC - 1) / kC;
  for (int ib = 0; ib < nb; ++ib) {
    const int blk = rev ? nb - 1 - ib : ib, r0 = blk * kC, nv = min(kC, u.len - r0);
    __syncthreads();  // the previous block's operands have been read
    stage_transposed<T, SUMMARY>(Qt, q + (long long)r0 * p.qs, p.qs, Kt, k + (long long)r0 * p.ks, p.ks, nv, p.dk);
    {
      constexpr int kTurns = kC * (kTV / 8) / kThreads, kRowsATurn = kThreads / (kTV / 8);
      const int r = tid / (kTV / 8), x = tid % (kTV / 8);
      float w[kTurns][8] = {};
#pragma unroll
      for (int y = 0; y < kTurns; ++y)
        if (r + y * kRowsATurn < nv && 8 * x < ncol) load8(v + (long long)(r0 + r + y * kRowsATurn) * p.vs + 8 * x, w[y]);
#pragma unroll
      for (int y = 0; y < kTurns; ++y)
#pragma unroll
        for (int i = 0; i < 8; i += 4)
          *reinterpret_cast<float4 *>(V + (r + y * kRowsATurn) * kLdV + 8 * x + i) =
              make_float4(w[y][i], w[y][i + 1], w[y][i + 2], w[y][i + 3]);
    }
    __syncthreads();
    if (!SUMMARY) {
      {  // A: 2 rows x 4 columns a thread, stored transposed
        const int i0 = 2 * (tid >> 3), j0 = 4 * (tid & 7);
        float acc[2][4] = {};
#pragma unroll 4
        for (int x = 0; x < p.dk; ++x) {
          const float2 a = *reinterpret_cast<const float2 *>(Qt + x * kLdC + i0);
          const float4 b = *reinterpret_cast<const float4 *>(Kt + x * kLdC + j0);
          const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[0][j] = fmaf(a.x, bv[j], acc[0][j]);
            acc[1][j] = fmaf(a.y, bv[j], acc[1][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 out;
          const int d0 = rev ? j0 + j - i0 : i0 - j0 - j, d1 = rev ? d0 - 1 : d0 + 1;
          out.x = d0 >= 0 ? acc[0][j] * (pw[d0] * p_scale) : 0.f;
          out.y = d1 >= 0 ? acc[1][j] * (pw[d1] * p_scale) : 0.f;
          *reinterpret_cast<float2 *>(At + (j0 + j) * kLdC + i0) = out;
        }
      }
      __syncthreads();
      // o: 4 rows x 4 columns a thread
      const int i0 = 4 * (tid >> 4), n0 = 4 * (tid & 15);
      float acc[4][4] = {};
#pragma unroll 4
      for (int x = 0; x < p.dk; ++x) {
        const float4 a = *reinterpret_cast<const float4 *>(Qt + x * kLdC + i0);
        const float4 b = *reinterpret_cast<const float4 *>(S + x * kLdV + n0);
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = p.o_scale * pw[rev ? max(nv - 1 - i0 - i, 0) : i0 + i + 1];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] *= w;
      }
#pragma unroll 4
      for (int x = 0; x < kC; ++x) {
        const float4 a = *reinterpret_cast<const float4 *>(At + x * kLdC + i0);
        const float4 b = *reinterpret_cast<const float4 *>(V + x * kLdV + n0);
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
      if (n0 < ncol) {  // widths are multiples of 8
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i0 + i >= nv) break;
          const long long at = (long long)(u.t0 + r0 + i0 + i) * p.os + (long long)h * p.dv + c0 + n0;
          if (p.o_f32)
            store4(static_cast<float *>(p.o) + at, acc[i]);
          else
            store4(static_cast<T *>(p.o) + at, acc[i]);
        }
      }
      __syncthreads();  // S has been read
    }
    // S: 8 rows x 4 columns a thread, 64 rows at a time
    const float2 carry = nv == kC ? carry_full : la_pow2(g, nv);
    const int n0 = 4 * (tid & 15);
    for (int a0 = 8 * (tid >> 4); a0 < dkp; a0 += 64) {
      float acc[8][4] = {};
#pragma unroll 2
      for (int j0 = 0; j0 < kC; j0 += 4) {
        float vv[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 b = *reinterpret_cast<const float4 *>(V + (j0 + j) * kLdV + n0);
          const int r = j0 + j;
          const float w = r < nv ? p.st_scale * pw[rev ? r + 1 : nv - 1 - r] : 0.f;
          vv[j][0] = b.x * w; vv[j][1] = b.y * w; vv[j][2] = b.z * w; vv[j][3] = b.w * w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 a = *reinterpret_cast<const float4 *>(Kt + (a0 + i) * kLdC + j0);
          const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = fmaf(av[j], vv[j][c], acc[i][c]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float4 *sp = reinterpret_cast<float4 *>(S + (a0 + i) * kLdV + n0);
        float4 t = *sp;
        t.x = fmaf(t.x, carry.x, fmaf(t.x, carry.y, acc[i][0]));
        t.y = fmaf(t.y, carry.x, fmaf(t.y, carry.y, acc[i][1]));
        t.z = fmaf(t.z, carry.x, fmaf(t.z, carry.y, acc[i][2]));
        t.w = fmaf(t.w, carry.x, fmaf(t.w, carry.y, acc[i][3]));
        *sp = t;
      }
    }
  }
  __syncthreads();
  int sa, sb;
  float *out = la_state_out(p, u.next, u.seq, h, SUMMARY, sa, sb);
  if (out)
    for (int e = tid; e < p.dk * kTV; e += kThreads) {
      const int a = e / kTV, b = e % kTV;
      if (b < ncol) out[(size_t)a * sa + (size_t)(c0 + b) * sb] = S[a * kLdV + b];
    }
}

// The states between segments of a cut sequence: per head, in processing order,
//     next = lam^len S + W_seg,   W_seg (from a zero state, where S belongs) replaced by S.
// The last segment has no W_seg: the pass that starts from its S writes the final state.
constexpr int kScanThreads = 256, kScanMax = 512;
__global__ void __launch_bounds__(kScanThreads) la_scan_kernel(LaPlanDev pl, const __grid_constant__ LaBatch batch) {
  __shared__ int units[kScanMax];
  const LaPass &p = batch.p[blockIdx.z];
  const int dd = p.dk * p.dv, nblk = (batch.p[0].dk * batch.p[0].dv + kScanThreads - 1) / kScanThreads;
  const int s = blockIdx.x / nblk, h = blockIdx.y;
  int a, len;
  la_seq_bounds(pl, s, a, len);
  // (unit s of a table is the first segment of sequence s)
  const int n = pl.table ? pl.table[s].nseg : la_segments(len, pl.seg_len);
  if (n == 1) return;
  const int e = blockIdx.x % nblk * kScanThreads + threadIdx.x;
  const bool live = e < dd;
  const size_t user = ((size_t)s * p.H + h) * dd + (size_t)(e / p.dv) * p.sa + (size_t)(e % p.dv) * p.sb;
  const float g = __ldg(p.g + h);
  const float2 full = la_pow2(g, pl.seg_len), tail = la_pow2(g, len - (n - 1) * pl.seg_len);
  float st = live && p.init ? p.init[user] : 0.f;
  float *base = p.seg_state + (size_t)h * dd + e;
  const size_t step = (size_t)p.H * dd;
  if (live && p.init_kept) base[s * step] = st;  // (unit s is the first of sequence s)
  constexpr int kAhead = 8;
  // level i + 1 holds what level i's segment gives, then the state after it
  for (int l0 = 1; l0 < n; l0 += kScanMax) {
    const int m = min(kScanMax, n - l0);
    __syncthreads();
    for (int i = threadIdx.x; i < m; i += kScanThreads) {
      const int level = l0 + i;
      int at = 0;
      if (!pl.table) {
        at = level * pl.nseq + s;
      } else {
        for (int x = 0; x < pl.nseq; ++x) {
          int xa, xl;
          la_seq_bounds(pl, x, xa, xl);
          const int xn = la_segments(xl, pl.seg_len);
          at += min(xn, level) + (x < s && xn > level);
        }
      }
      units[i] = at;
    }
    __syncthreads();
    if (!live) continue;
    for (int i0 = 0; i0 < m; i0 += kAhead) {
      float w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i0 + i < m) w[i] = base[units[i0 + i] * step];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i0 + i < m) {
          // the segment before this level: the sequence's tail comes first in reverse
          const float2 c = p.reverse && l0 + i0 + i == 1 ? tail : full;
          st = fmaf(st, c.x, fmaf(st, c.y, w[i]));
          base[units[i0 + i] * step] = st;
        }
    }
  }
}

// out(row, kv, c) = sum of in(row, kv * group + i, c) over i, in order; blockIdx.y: which of two tensors
template <typename T>
__global__ void __launch_bounds__(256) la_sum_heads_kernel(const LaHeadSum x, const LaHeadSum y, long long rows, int Hkv,
                                                           int group) {
  const LaHeadSum &p = blockIdx.y ? y : x;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  const int d4 = p.d / 4, c = (int)(e % d4);
  const long long rk = e / d4, row = rk / Hkv;
  if (row >= rows) return;
  const int kv = (int)(rk % Hkv);
  const float4 *src = reinterpret_cast<const float4 *>(p.in) + (row * Hkv + kv) * (long long)group * d4 + c;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < group; ++i) {
    const float4 t = __ldg(src + (long long)i * d4);
    acc[0] += t.x; acc[1] += t.y; acc[2] += t.z; acc[3] += t.w;
  }
  store4(static_cast<T *>(p.out) + row * p.os + (long long)kv * p.d + 4 * c, acc);
}

constexpr int smem_bytes(int dk, bool summary) {
  const int dkp = (dk + 63) & ~63;
  return 4 * ((summary ? 1 : 2) * dkp * kLdC + dkp * kLdV + kC * kLdV + (summary ? 0 : kC * kLdC) + kC + 4);
}

template <typename T, bool SUMMARY>
void run_simt(const LaPlanDev &pl, const LaBatch &b, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(la_simt_kernel<T, SUMMARY>), smem_bytes(256, SUMMARY), allowed);
  int dk = 0, dv = 0;
  for (int i = 0; i < b.n; ++i) {
    dk = b.p[i].dk > dk ? b.p[i].dk : dk;
    dv = b.p[i].dv > dv ? b.p[i].dv : dv;
  }
  const dim3 grid(pl.units, pl.H, (dv + kTV - 1) / kTV * b.n);
  la_simt_kernel<T, SUMMARY><<<grid, kThreads, smem_bytes(dk, SUMMARY), s>>>(pl, b);
}

}  // namespace

template <typename T>
void launch_la_simt(const LaPlanDev &pl, const LaBatch &b, bool summary, cudaStream_t s) {
  summary ? run_simt<T, true>(pl, b, s) : run_simt<T, false>(pl, b, s);
}

void launch_la_scan(const LaPlanDev &pl, const LaBatch &b, cudaStream_t s) {
  const int nblk = (b.p[0].dk * b.p[0].dv + kScanThreads - 1) / kScanThreads;  // the same for every pass
  la_scan_kernel<<<dim3(nblk * pl.nseq, pl.H, b.n), kScanThreads, 0, s>>>(pl, b);
}

template <typename T>
void launch_la_sum_heads(const LaHeadSum &x, const LaHeadSum &y, long long rows, int Hkv, int group, cudaStream_t s) {
  const long long n4 = rows * Hkv * ((x.d > y.d ? x.d : y.d) / 4);
  la_sum_heads_kernel<T><<<dim3((unsigned)((n4 + 255) / 256), 2), 256, 0, s>>>(x, y, rows, Hkv, group);
}

template void launch_la_simt<float>(const LaPlanDev &, const LaBatch &, bool, cudaStream_t);
template void launch_la_simt<__nv_bfloat16>(const LaPlanDev &, const LaBatch &, bool, cudaStream_t);
template void launch_la_sum_heads<float>(const LaHeadSum &, const LaHeadSum &, long long, int, int, cudaStream_t);
template void launch_la_sum_heads<__nv_bfloat16>(const LaHeadSum &, const LaHeadSum &, long long, int, int, cudaStream_t);

}  // namespace ssd
