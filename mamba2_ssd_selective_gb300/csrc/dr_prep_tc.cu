// What the tensor-core chains of the gated delta rule need of every chunk before the state is known: the rows' factors, and
// N and P as tiles of two bf16 terms (delta.h has the formulas).
//
// A block of four warps takes a chunk and a head of q and k: K K^T and Q K^T by matrix instructions, a warp's 16 rows of both
// in its registers, for all states that share the head; A and P share their exponentials.  A warp has 8 rows of the upper
// and 8 of the lower half, so that all warps have as much below the diagonal.
// N = (I + A diag(b))^-1 A in blocks, without a division by b: diagonal blocks of 16 column by column, a thread to a
// column, then twice the block below two that are done (b1, b2: theirs),
//     N21 = M - N22 (b2 M),   M = A21 - A21 (b1 N11),
// in place, since A's blocks are not read again.  Sums of log decays are whole numbers of 2^-32 (dr_rows.cuh).
#include "delta.h"
#include "dr_rows.cuh"
#include "tc_pipe.cuh"
#include "tc_util.cuh"

namespace ssd {

namespace {

using bf16 = __nv_bfloat16;
using namespace sm100;

constexpr int kThreads = 128, kLd = kDrC + 4;
constexpr uint32_t kBox = 8192;

constexpr int kHeads = 2;  // whose rows' factors are made at once, by a warp each
// The boxes of K and Q, and in their place, once their products are made, N's and P's tiles on their way out.
constexpr uint32_t kTilesN = 0, kTilesP = 2 * kBox;
struct Work {
  float m[kDrC][kLd];  // A, then N
  float rk[kDrC], rq[kDrC];
  DrRows rows[kHeads];
  int first_nan[kHeads];
  uint64_t full;
};
constexpr int kSmemBytes = 4 * (int)kBox + (int)sizeof(Work) + 1024;

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x[r][c] -= sum_k A[r][k] b[k] B[k][c], k from k0 to k1: ROWS rows STEP apart x 2 values a thread
template <int ROWS, int STEP>
__device__ __forceinline__ void minus_product(float (&x)[ROWS][2], const float *A, const float *b, const float *B, int k0, int k1) {
#pragma unroll 4
  for (int k = k0; k < k1; k += 4) {
    const float4 bb = *reinterpret_cast<const float4 *>(b + k);
    float2 y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = *reinterpret_cast<const float2 *>(B + (k + e) * kLd);
    y[0].x *= -bb.x, y[0].y *= -bb.x, y[1].x *= -bb.y, y[1].y *= -bb.y;
    y[2].x *= -bb.z, y[2].y *= -bb.z, y[3].x *= -bb.w, y[3].y *= -bb.w;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float4 a = *reinterpret_cast<const float4 *>(A + r * STEP * kLd + k);
      x[r][0] = fmaf(a.x, y[0].x, fmaf(a.y, y[1].x, fmaf(a.z, y[2].x, fmaf(a.w, y[3].x, x[r][0]))));
      x[r][1] = fmaf(a.x, y[0].y, fmaf(a.y, y[1].y, fmaf(a.z, y[2].y, fmaf(a.w, y[3].y, x[r][1]))));
    }
  }
}
template <int ROWS, int STEP> __device__ __forceinline__ void get(float (&x)[ROWS][2], const float *m) {
#pragma unroll
  for (int e = 0; e < ROWS; ++e) {
    const float2 t = *reinterpret_cast<const float2 *>(m + e * STEP * kLd);
    x[e][0] = t.x, x[e][1] = t.y;
  }
}
template <int ROWS, int STEP> __device__ __forceinline__ void put(const float (&x)[ROWS][2], float *m) {
#pragma unroll
  for (int e = 0; e < ROWS; ++e) *reinterpret_cast<float2 *>(m + e * STEP * kLd) = make_float2(x[e][0], x[e][1]);
}

__device__ __forceinline__ void sts(uint32_t at, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); }

// PT: terms of P that are wanted
template <int KB, int PT>
__global__ void __launch_bounds__(kThreads, 4) dr_prep_tc_kernel(const __grid_constant__ CUtensorMap tq,
                                                                 const __grid_constant__ CUtensorMap tk, const DrProblem p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = tc::aligned_smem(smem_raw);
  Work &w = *reinterpret_cast<Work *>(sm + 4 * kBox);
  float(*m)[kLd] = w.m;
  const int slot = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (slot == 0 && hk == 0 && tid == 0) *p.status = 0;
  int t0, n;
  dr_chunk(p, slot, t0, n);
  if (n == 0) return;
  const uint32_t s0 = smem_u32(sm);
  if (tid == 0) {
    mbar_init(&w.full, 1);
    fence_mbar_init();
    mbar_expect_tx(&w.full, 2 * KB * kBox);
    for (int b = 0; b < KB; ++b) {
      tma_load_3d(sm + b * kBox, &tk, &w.full, 64 * b, hk, t0);
      tma_load_3d(sm + (KB + b) * kBox, &tq, &w.full, 64 * b, hk, t0);
    }
  }
  DrSums sums;
  if (warp < kHeads && warp < p.group) sums = dr_sums(dr_load_gates<bf16>(p, hk * p.group + warp, t0, n, lane), lane);
  __syncthreads();
  mbar_wait_drain(&w.full, 0);
  // rows i0 on and i1 on of both products: columns 8 y + 2 (lane % 4) and the next, rows lane / 4.  The lengths of q are
  // the diagonals of Q Q^T's blocks of 8 x 8, those of k of K K^T's
  const int i0 = 8 * warp, i1 = 56 - 8 * warp;
  const int ir = (lane & 8 ? i1 : i0) + (lane & 7);
  float kk[8][4], qk[8][4], qq[2][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int y = 0; y < 8; ++y) kk[y][e] = qk[y][e] = 0.f;
    qq[0][e] = qq[1][e] = 0.f;
  }
#pragma unroll
  for (int b = 0; b < KB; ++b) {
    const uint32_t tb = s0 + b * kBox, ta = s0 + (KB + b) * kBox;
#pragma unroll
    for (int c = 0; c < 64; c += 16) {
      uint32_t fk[4], fq[4];
      ldmatrix4(tb + sw128_offset(ir, c + 8 * (lane >> 4)), fk);
      ldmatrix4(ta + sw128_offset(ir, c + 8 * (lane >> 4)), fq);
      mma16816(qq[0], fq, fq[0], fq[2]);  // rows of the second operand are those of the first's fragments
      mma16816(qq[1], fq, fq[1], fq[3]);
#pragma unroll
      for (int y = 0; y < 8; y += 2) {
        if (8 * y > i1) continue;  // above the diagonal
        uint32_t fb[4];
        ldmatrix4(tb + sw128_offset(8 * y + (lane & 7) + 8 * (lane >> 4), c + 8 * ((lane >> 3) & 1)), fb);
        mma16816(kk[y], fk, fb[0], fb[1]);
        mma16816(kk[y + 1], fk, fb[2], fb[3]);
        mma16816(qk[y], fq, fb[0], fb[1]);
        mma16816(qk[y + 1], fq, fb[2], fb[3]);
      }
    }
  }
  const int r0 = lane >> 2, c0 = 2 * (lane & 3);
#pragma unroll
  for (int e = 0; e < 2; ++e) {  // a row's diagonal value is column lane / 4 of its block
    const int i = (e ? i1 : i0) + r0;
    float k2 = 0.f;
#pragma unroll
    for (int y = 0; y < 8; ++y)
      if (8 * y == (e ? i1 : i0)) k2 = lane >> 2 & 1 ? kk[y][2 * e + 1] : kk[y][2 * e];
    const float q2 = lane >> 2 & 1 ? qq[e][2 * e + 1] : qq[e][2 * e];
    if ((lane & 3) == lane >> 3) {
      w.rk[i] = p.norm ? 1.f / sqrtf(k2 + p.eps) : 1.f;
      w.rq[i] = p.norm ? 1.f / sqrtf(q2 + p.eps) : 1.f;
    }
  }
#pragma unroll 1
  for (int g = 0; g < p.group; ++g) {
    const int h = hk * p.group + g;
    const size_t at = (size_t)slot * p.H + h;
    if (g % kHeads == 0) {  // the factors of the next heads
      if (g > 0 && warp < kHeads && g + warp < p.group)
        sums = dr_sums(dr_load_gates<bf16>(p, h + warp, t0, n, lane), lane);
      __syncthreads();  // the lengths are there, the boxes and the last factors read
      if (warp < kHeads && g + warp < p.group) {
        dr_put_rows(w.rows[warp], sums, w.rk, w.rq, p.scale, n, lane);
        if (lane == 0) w.first_nan[warp] = sums.first_nan;
      }
    }
    if (g > 0 && tid == kThreads - 1) bulk_wait_read0();  // the last head's P has left
    __syncthreads();
    const DrRows &rows = w.rows[g % kHeads];
    const int nan_at = w.first_nan[g % kHeads];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int first = e ? i1 : i0, i = first + r0;
      const float hi = rows.ghi[i], lo = rows.glo[i], rk = rows.rk[i], rq = rows.rq[i] * p.scale;
      const uint32_t row = s0 + kTilesP + i * 128 + 2 * c0;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const int j = 8 * y + c0;
        float a[2] = {0.f, 0.f}, q[2] = {0.f, 0.f};
        if (8 * y <= first && i < n) {
          const float2 gh = *reinterpret_cast<const float2 *>(rows.ghi + j), gl = *reinterpret_cast<const float2 *>(rows.glo + j),
                       rj = *reinterpret_cast<const float2 *>(rows.rk + j);
          float l[2] = {__expf((hi - gh.x) + (lo - gl.x)) * rj.x, __expf((hi - gh.y) + (lo - gl.y)) * rj.y};
          if (nan_at < kDrC && i >= nan_at) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (j + x < nan_at) l[x] = __int_as_float(0x7fffffff);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            a[x] = kk[y][2 * e + x] * (l[x] * rk);
            q[x] = qk[y][2 * e + x] * (l[x] * rq);
          }
          if (8 * y == first) {  // the diagonal's block
            a[0] = j < i ? a[0] : 0.f, a[1] = j + 1 < i ? a[1] : 0.f;
            q[0] = j <= i ? q[0] : 0.f, q[1] = j + 1 <= i ? q[1] : 0.f;
          }
        }
        *reinterpret_cast<float2 *>(&m[i][j]) = make_float2(a[0], a[1]);
        uint32_t qh, ql;
        tc::split2(q[0], q[1], qh, ql);
        sts(row + ((y ^ (lane >> 2)) << 4), qh);  // the 128-byte swizzle: the row is lane / 4 modulo 8
        if (PT == 2) sts(row + kBox + ((y ^ (lane >> 2)) << 4), ql);
      }
    }
    {
      const float4 *from = reinterpret_cast<const float4 *>(&rows);
      float4 *to = reinterpret_cast<float4 *>(p.rows + at);
      for (int e = tid; e < (int)(sizeof(DrRows) / 16); e += kThreads) to[e] = from[e];
    }
    fence_async_smem();
    __syncthreads();
    if (tid == kThreads - 1) {
      pipe::bulk_store(reinterpret_cast<uint8_t *>(p.N) + at * (4 * kDrTile) + 2 * kDrTile, s0 + kTilesP, PT * kBox);
      bulk_commit();
    }
    if (tid < kDrC) {
      float x[16];
      const int d0 = tid & 48, c = tid & 15;  // column c of the diagonal block from d0
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = m[d0 + i][d0 + c];  // zeros up to the diagonal
#pragma unroll
      for (int k = 1; k < 15; ++k) {
        const float f = -rows.beta[d0 + k] * x[k];
#pragma unroll
        for (int i = k + 1; i < 16; ++i) x[i] = fmaf(f, m[d0 + i][d0 + k], x[i]);
      }
      __syncwarp();  // a block is one half-warp's
#pragma unroll
      for (int i = 1; i < 16; ++i) m[d0 + i][d0 + c] = x[i];
    }
    __syncthreads();
    {  // two blocks of 16 x 16, a half of the threads each: 2 x 2 values a thread
      const int d0 = tid >> 6 ? 32 : 0, r = 2 * ((tid & 63) >> 3), c = 2 * (tid & 7);
      float x[2][2], *mine = &m[d0 + 16 + r][d0 + c];
      get<2, 1>(x, mine);
      minus_product<2, 1>(x, &m[d0 + 16 + r][d0], rows.beta + d0, &m[d0][d0 + c], 0, 16);
      __syncthreads();
      put<2, 1>(x, mine);
      __syncthreads();
      minus_product<2, 1>(x, &m[d0 + 16 + r][d0 + 16], rows.beta + d0 + 16, &m[d0 + 16][d0 + c], 0, 16);
      __syncthreads();
      put<2, 1>(x, mine);
    }
    __syncthreads();
    {  // 32 x 32: 8 values a thread.  N11 has zeros up to its diagonal, so a warp's 8 columns leave the sum's first terms out
      const int r = lane & 7, c = 8 * warp + 2 * (lane >> 3);
      float x[4][2];
      get<4, 8>(x, &m[32 + r][c]);
      minus_product<4, 8>(x, &m[32 + r][0], rows.beta, &m[0][c], 8 * warp, 32);
      __syncthreads();
      put<4, 8>(x, &m[32 + r][c]);
    }
    __syncthreads();
    {  // and N22 from it, so that a warp's 8 rows leave out the last
      const int r = 8 * warp + 4 * (lane >> 4), c = 2 * (lane & 15);
      float x[4][2];
      get<4, 1>(x, &m[32 + r][c]);
      minus_product<4, 1>(x, &m[32 + r][32], rows.beta + 32, &m[32][c], 0, 8 * warp + 8);
      if (tid == 0) bulk_wait_read0();  // the last head's N has left
      __syncthreads();
      put<4, 1>(x, &m[32 + r][c]);
    }
    __syncthreads();
#pragma unroll
    for (int e = tid; e < kDrC * 8; e += kThreads) {  // N's terms, 8 columns at a time
      const int i = e >> 3, y = e & 7;
      const float4 x0 = *reinterpret_cast<const float4 *>(&m[i][8 * y]), x1 = *reinterpret_cast<const float4 *>(&m[i][8 * y + 4]);
      uint4 hi, lo;
      tc::split2(x0.x, x0.y, hi.x, lo.x);
      tc::split2(x0.z, x0.w, hi.y, lo.y);
      tc::split2(x1.x, x1.y, hi.z, lo.z);
      tc::split2(x1.z, x1.w, hi.w, lo.w);
      const uint32_t to = s0 + kTilesN + i * 128 + ((y ^ (i & 7)) << 4);
      pipe::sts_u4(to, hi);
      pipe::sts_u4(to + kBox, lo);
    }
    fence_async_smem();
    __syncthreads();
    if (tid == 0) {
      pipe::bulk_store(reinterpret_cast<uint8_t *>(p.N) + at * (4 * kDrTile), s0 + kTilesN, 2 * kBox);
      bulk_commit();
    }
  }
  if (tid == 0 || tid == kThreads - 1) bulk_wait_read0();
}

template <int KB, int PT> void run(const DrProblem &p, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  constexpr int bytes = kSmemBytes;
  allow_smem(reinterpret_cast<const void *>(dr_prep_tc_kernel<KB, PT>), bytes, allowed);
  CUtensorMap tq, tk;
  if (!encode_tmap_bf16_heads(&tq, p.q, p.dk, p.Hk, p.total, p.qs * 2, kDrC) ||
      !encode_tmap_bf16_heads(&tk, p.k, p.dk, p.Hk, p.total, p.ks * 2, kDrC)) {
    note_host_error();
    return;
  }
  dr_prep_tc_kernel<KB, PT><<<dim3((unsigned)p.slots, (unsigned)p.Hk), kThreads, bytes, s>>>(tq, tk, p);
}

}  // namespace

void launch_dr_prep_tc(const DrProblem &p, bool backward, cudaStream_t s) {
  if (la_tc_boxes(p.dk) == 1)
    backward ? run<1, 2>(p, s) : run<1, 1>(p, s);
  else
    backward ? run<2, 2>(p, s) : run<2, 1>(p, s);
}

}  // namespace ssd
