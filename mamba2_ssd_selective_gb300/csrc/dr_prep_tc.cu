// What the tensor-core chains of the gated delta rule need of every chunk before the state is known: the rows' factors, and
// N and P as tiles of two bf16 terms (delta.h has the formulas).
//
// A block of four warps takes a chunk and a head of q and k: K K^T and Q K^T by matrix instructions, a warp's 16 rows of both
// in its registers, for all states that share the head; A and P share their exponentials.  A warp has 8 rows of the upper
// and 8 of the lower half, so that all warps have as much below the diagonal.
// N = (I + A diag(b))^-1 A in blocks of 16, without a division by b.  The diagonal's blocks column by column, a thread to a
// column; then a warp has a column J of blocks, from the diagonal down,
//     N_IJ = M - N_II (b_I M),    M = A_IJ - sum_(J <= K < I) A_IK (b_K N_KJ),
// transposed, so that what a step makes is the next one's first operand as it stands in the registers.  Both operands are
// sums of two bf16 terms, which is how N goes out too.
// 4 x 8192 tokens, 16 heads of q and k for 32 states take 205 us, their bytes 124 us at 6.8 TB/s (with one term of P 195 us;
// with products of 16 and 32 rows in fp32 on the CUDA cores 239 us).  What bounds it is latency: a block's steps follow one another, and registers and
// shared memory let four blocks onto an SM (a third of the instructions that it could issue).
#include "delta.h"
#include "dr_rows.cuh"
#include "tc_pipe.cuh"
#include "tc_util.cuh"

namespace ssd {

namespace {

using bf16 = __nv_bfloat16;
using namespace sm100;

constexpr int kThreads = 128;
constexpr uint32_t kBox = 8192;
constexpr int kHeads = 2;  // whose rows' factors are made at once, by a warp each
// The boxes of K and Q, and in their place, once their products are made, N's and P's tiles on their way out; behind them
// A's two terms, whose diagonal blocks of 16 hold A itself instead (diag_at).
constexpr uint32_t kTilesN = 0, kTilesP = 2 * kBox, kTilesA = 4 * kBox;
struct Work {
  float rk[kDrC], rq[kDrC];
  DrRows rows[kHeads];
  int first_nan[kHeads];
  uint64_t full;
};
constexpr int kSmemBytes = 6 * (int)kBox + (int)sizeof(Work) + 1024;

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
// Element (r, c) of the diagonal block from row 16 I on, in fp32: columns 0-7 in the first tile's place of the block, 8-15 in
// the second's
__device__ __forceinline__ uint32_t diag_at(uint32_t tiles, int I, int r, int c) {
  const int row = 16 * I + r;
  return tiles + (c & 8 ? kBox : 0) + row * 128 + (((2 * I + ((c & 7) >> 2)) ^ (row & 7)) << 4) + (c & 3) * 4;
}
// A 16 x 16 block as a result or a first operand of the matrix instruction: rows lane / 4 and 8 more, columns
// 2 (lane % 4) and the next, [.][2..3] in the second rows, [1] 8 columns on.
using Block = float[2][4];
// the transpose of the block of a tile's two terms from row r0, column c0 on
__device__ __forceinline__ void load_transposed(Block &x, uint32_t tile, int r0, int c0, int lane) {
  const uint32_t at = tile + sw128_offset(r0 + (lane & 7) + 8 * (lane >> 4), c0 + 8 * ((lane >> 3) & 1));
  uint32_t h[4], l[4];
  ldmatrix4_trans(at, h[0], h[1], h[2], h[3]);
  ldmatrix4_trans(at + kBox, l[0], l[1], l[2], l[3]);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e >> 1][2 * (e & 1)] = __uint_as_float(h[e] << 16) + __uint_as_float(l[e] << 16);
    x[e >> 1][2 * (e & 1) + 1] = __uint_as_float(h[e] & 0xffff0000u) + __uint_as_float(l[e] & 0xffff0000u);
  }
}
struct Terms {
  uint32_t hi[4], lo[4];
};
// a block's columns times -b, as a first operand of two terms
__device__ __forceinline__ void make_terms(Terms &t, const Block &x, const float *b, int lane) {
  const float2 b0 = *reinterpret_cast<const float2 *>(b + 2 * (lane & 3)), b1 = *reinterpret_cast<const float2 *>(b + 8 + 2 * (lane & 3));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = e >> 1 ? b1 : b0;
    tc::split2(-f.x * x[e >> 1][2 * (e & 1)], -f.y * x[e >> 1][2 * (e & 1) + 1], t.hi[e], t.lo[e]);
  }
}
// x += t B^T, B the block of a tile's two terms from row r0, column c0 on (what two low terms make is left out)
__device__ __forceinline__ void add_product(Block &x, const Terms &t, uint32_t tile, int r0, int c0, int lane) {
  const uint32_t at = tile + sw128_offset(r0 + (lane & 7) + 8 * (lane >> 4), c0 + 8 * ((lane >> 3) & 1));
  uint32_t h[4], l[4];
  ldmatrix4(at, h);
  ldmatrix4(at + kBox, l);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    mma16816(x[n], t.lo, h[2 * n], h[2 * n + 1]);
    mma16816(x[n], t.hi, l[2 * n], l[2 * n + 1]);
    mma16816(x[n], t.hi, h[2 * n], h[2 * n + 1]);
  }
}
// the block's transpose as a tile's two terms, from row r0, column c0 on
__device__ __forceinline__ void store_transposed(const Block &x, uint32_t tile, int r0, int c0, int lane) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) tc::split2(x[e >> 1][2 * (e & 1)], x[e >> 1][2 * (e & 1) + 1], h[e], l[e]);
  const uint32_t at = tile + sw128_offset(r0 + (lane & 7) + 8 * (lane >> 4), c0 + 8 * ((lane >> 3) & 1));
  stmatrix4_trans(at, h[0], h[1], h[2], h[3]);
  stmatrix4_trans(at + kBox, l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ float lds(uint32_t at) { return pipe::lds_f(at); }

__device__ __forceinline__ void sts(uint32_t at, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); }

template <int KB>
__global__ void __launch_bounds__(kThreads, 4) dr_prep_tc_kernel(const __grid_constant__ CUtensorMap tq,
                                                                 const __grid_constant__ CUtensorMap tk, const DrProblem p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = tc::aligned_smem(smem_raw);
  Work &w = *reinterpret_cast<Work *>(sm + 6 * kBox);
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
    if (g > 0 && tid == kThreads - 1) bulk_wait_read0();  // the last head's factors and P have left
    if (g % kHeads == 0) {  // the factors of the next heads
      if (g > 0 && warp < kHeads && g + warp < p.group)
        sums = dr_sums(dr_load_gates<bf16>(p, h + warp, t0, n, lane), lane);
      __syncthreads();  // the lengths are there, the boxes and the last factors read
      if (warp < kHeads && g + warp < p.group) {
        dr_put_rows(w.rows[warp], sums, w.rk, w.rq, p.scale, n, lane);
        if (lane == 0) w.first_nan[warp] = sums.first_nan;
      }
    }
    __syncthreads();
    const DrRows &rows = w.rows[g % kHeads];
    const int nan_at = w.first_nan[g % kHeads];
    float hi[2], lo[2], rk[2], rq[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = (e ? i1 : i0) + r0;
      hi[e] = rows.ghi[i], lo[e] = rows.glo[i], rk[e] = rows.rk[i], rq[e] = rows.rq[i] * p.scale;
    }
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      const int j = 8 * y + c0;
      float2 gh = make_float2(0.f, 0.f), gl = gh, rj = gh;
      if (8 * y <= i1) {
        gh = *reinterpret_cast<const float2 *>(rows.ghi + j), gl = *reinterpret_cast<const float2 *>(rows.glo + j);
        rj = *reinterpret_cast<const float2 *>(rows.rk + j);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int first = e ? i1 : i0, i = first + r0;
        const bool below = 8 * y <= first, diagonal = 8 * (y & ~1) == (first & ~15);  // a block of the diagonal's 16 x 16
        if (!below && g > 0) continue;  // zeros above the diagonal stay
        const uint32_t at_j = i * 128 + 2 * c0 + ((y ^ (lane >> 2)) << 4);  // the 128-byte swizzle: the row is lane / 4 modulo 8
        float a[2] = {0.f, 0.f}, q[2] = {0.f, 0.f};
        if (below && i < n) {
          float l[2] = {__expf((hi[e] - gh.x) + (lo[e] - gl.x)) * rj.x, __expf((hi[e] - gh.y) + (lo[e] - gl.y)) * rj.y};
          if (nan_at < kDrC && i >= nan_at) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (j + x < nan_at) l[x] = __int_as_float(0x7fffffff);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            a[x] = kk[y][2 * e + x] * (l[x] * rk[e]);
            q[x] = qk[y][2 * e + x] * (l[x] * rq[e]);
          }
          if (8 * y == first) {  // the diagonal's block
            a[0] = j < i ? a[0] : 0.f, a[1] = j + 1 < i ? a[1] : 0.f;
            q[0] = j <= i ? q[0] : 0.f, q[1] = j + 1 <= i ? q[1] : 0.f;
          }
        }
        if (diagonal) {
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(diag_at(s0 + kTilesA, first >> 4, i & 15, j & 15)), "f"(a[0]), "f"(a[1]) : "memory");
        } else if (below) {
          uint32_t ah, al;
          tc::split2(a[0], a[1], ah, al);
          sts(s0 + kTilesA + at_j, ah);
          sts(s0 + kTilesA + at_j + kBox, al);
        }
        if (!below) {
          sts(s0 + kTilesN + at_j, 0);
          sts(s0 + kTilesN + at_j + kBox, 0);
        }
        uint32_t qh, ql;
        tc::split2(q[0], q[1], qh, ql);
        sts(s0 + kTilesP + at_j, qh);
        sts(s0 + kTilesP + at_j + kBox, ql);
      }
    }
    fence_async_smem();
    if (g > 0 && tid == 0) bulk_wait_read0();  // the last head's N has left
    __syncthreads();
    if (tid == kThreads - 1) {
      pipe::bulk_store(p.rows + at, smem_u32(&rows), sizeof(DrRows));
      pipe::bulk_store(reinterpret_cast<uint8_t *>(p.N) + at * (4 * kDrTile) + 2 * kDrTile, s0 + kTilesP, 2 * kBox);
      bulk_commit();
    }
    if (tid >= kDrC) {
      float x[16];
      const int I = (tid >> 4) & 3, c = tid & 15;  // column c of the diagonal's block I
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = lds(diag_at(s0 + kTilesA, I, i, c));  // zeros up to the diagonal
#pragma unroll
      for (int k = 1; k < 15; ++k) {
        const float f = -rows.beta[16 * I + k] * x[k];
#pragma unroll
        for (int i = k + 1; i < 16; ++i) x[i] = fmaf(f, lds(diag_at(s0 + kTilesA, I, i, k)), x[i]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]), lo = __float2bfloat16_rn(x[i] - __bfloat162float(hi));
        uint8_t *to = sm + kTilesN + sw128_offset(16 * I + i, 16 * I + c);
        *reinterpret_cast<__nv_bfloat16 *>(to) = hi;
        *reinterpret_cast<__nv_bfloat16 *>(to + kBox) = lo;
      }
    }
    __syncthreads();
    {
      const int J = warp;
      Terms done[3];  // of -b N_KJ, transposed
      Block x;
      if (J < 3) {
        load_transposed(x, s0 + kTilesN, 16 * J, 16 * J, lane);
        make_terms(done[0], x, rows.beta + 16 * J, lane);
      }
#pragma unroll
      for (int d = 1; d < 4; ++d) {
        const int I = J + d;
        if (I < 4) {
          load_transposed(x, s0 + kTilesA, 16 * I, 16 * J, lane);
#pragma unroll
          for (int e = 0; e < d; ++e) add_product(x, done[e], s0 + kTilesA, 16 * I, 16 * (J + e), lane);
          Terms t;
          make_terms(t, x, rows.beta + 16 * I, lane);
          add_product(x, t, s0 + kTilesN, 16 * I, 16 * I, lane);
          store_transposed(x, s0 + kTilesN, 16 * I, 16 * J, lane);
          if (d < 3) make_terms(done[d], x, rows.beta + 16 * I, lane);
        }
      }
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

template <int KB> void run(const DrProblem &p, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  constexpr int bytes = kSmemBytes;
  allow_smem(reinterpret_cast<const void *>(dr_prep_tc_kernel<KB>), bytes, allowed);
  CUtensorMap tq, tk;
  if (!encode_tmap_bf16_heads(&tq, p.q, p.dk, p.Hk, p.total, p.qs * 2, kDrC) ||
      !encode_tmap_bf16_heads(&tk, p.k, p.dk, p.Hk, p.total, p.ks * 2, kDrC)) {
    note_host_error();
    return;
  }
  dr_prep_tc_kernel<KB><<<dim3((unsigned)p.slots, (unsigned)p.Hk), kThreads, bytes, s>>>(tq, tk, p);
}

}  // namespace

void launch_dr_prep_tc(const DrProblem &p, cudaStream_t s) { la_tc_boxes(p.dk) == 1 ? run<1>(p, s) : run<2>(p, s); }

}  // namespace ssd
