// Linear attention with a decay for each head on the 5th-generation tensor cores
// (tcgen05, accumulators and the state operand in TMEM): bf16 tensors, widths up to 128.
//
// One CTA takes one segment of one sequence and one query head, and walks it in
// blocks of 64 tokens.  With P_ij = scale q_i . k_j lam^|i - j| inside the block
// (j <= i; reverse: j >= i) and the incoming state S (dk x dv):
//     O^T  = V^T P^T              Oi^T = S^T Q^T
//     o_i  = O_i + lam^a(i) Oi_i
//     S    = lam^nv S + (diag(lam^b) K)^T V
// The outputs are formed transposed, so that dv (up to 128) fills the lanes of
// the accumulators and the state, which its warps hold in registers as S^T (lane =
// dv), goes into TMEM as the A operand of Oi without a detour through shared
// memory.  P and S are rounded to bf16 as operands (the outputs are bf16 too);
// what goes into the state is not: diag(lam^b) K is split into three bf16 terms
// (24 bits), so that states keep fp32 precision over any length.
//
// Warps:
//   0, 1    P: scores out of TMEM (lane = row i of the block), decay and mask, P into shared memory
//   2       TMA producer: Q, K, V blocks [64 x 64 columns each], a ring of stages
//   3       TMEM owner and MMA issuer
//   4-7     outputs: O^T and Oi^T out of TMEM, combined, transposed through shared memory
//   8-15    state: the three terms of diag(lam^b) K, then S = lam^nv S + W and S^T into TMEM
// A block's scores are issued one block ahead, so that P is ready when the
// tensor core gets to it.  The last block of a sequence is masked: rows past its
// end belong to another sequence, so K's rows there are not used, V's are zeroed
// (0 * NaN would be NaN), and nothing is stored there.
#include "retention.h"
#include "tc_pipe.cuh"
#include "tc_util.cuh"

namespace ssd {

namespace {

using bf16 = __nv_bfloat16;
using namespace sm100;
using pipe::parity;

constexpr int kC = 64;  // tokens of a block
constexpr int kThreads = 512;
constexpr int kStateWarp0 = 8, kStateWarps = 8, kOutWarp0 = 4;
constexpr uint32_t kBox = 8192;  // [64 tokens x 64 columns] bf16

// TMEM columns
constexpr uint32_t kTmQK = 0, kTmO = 64, kTmOi = 192, kTmW = 320, kTmS = 448, kTmCols = 512;

template <int KB, int VB, bool SUMMARY>
struct Layout {
  static constexpr int kStages = KB + VB == 2 ? 4 : 3;
  // a stage: Q, later the block's outputs; K, later the first term of the weighted K; V
  static constexpr int kQBoxes = SUMMARY ? 0 : KB > VB ? KB : VB;
  static constexpr uint32_t kQ = 0, kK = kQBoxes * kBox, kV = kK + KB * kBox, kStage = kV + VB * kBox;
  static constexpr uint32_t kLoad = ((SUMMARY ? 1 : 2) * KB + VB) * kBox;  // bytes loaded into a stage
  static constexpr uint32_t kKt = kStages * kStage;                // two buffers of the other two terms
  static constexpr uint32_t kP = kKt + 4 * KB * kBox;              // two P buffers
  static constexpr uint32_t kTab = kP + (SUMMARY ? 0 : 2 * kBox);  // lam^n times each scale, n = 0..64
  static constexpr uint32_t kBar = kTab + 3 * 272 + 16;
  static constexpr int kNumBars = 2 * kStages + 2 + 1 + 1 + 2 + 2 + 1 + 2 + 1 + 2 + 2 + 1;
  static constexpr uint32_t kEnd = kBar + kNumBars * 8 + 16;
  static constexpr int kBytes = (int)kEnd + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};

// The m-th use of a barrier that alternates between two is completion m / 2 of
// barrier m & 1.  Alternation is needed wherever the arriving side may be a block
// ahead of a waiter (k_done, kt_ready).
template <int ST>
struct Bars {
  uint64_t *full, *free;        // [ST] stage loaded / its operands and outputs read
  uint64_t *k_done;             // [2] scores formed (for the state warps, which then overwrite K)
  uint64_t *qk_full, *qk_free;  // scores (for the P warps)
  uint64_t *p_ready, *p_free;   // [2]
  uint64_t *s_ready;            // S^T of the block in TMEM, and the previous W read
  uint64_t *kt_ready;           // [2] weighted K in shared memory (and V's tail zeroed)
  uint64_t *w_full;             // W formed, weighted K and S^T read
  uint64_t *o_full, *o_free;    // [2]
  uint64_t *drain;
  __device__ explicit Bars(uint64_t *b) {
    full = b;
    free = full + ST;
    k_done = free + ST;
    qk_full = k_done + 2;
    qk_free = qk_full + 1;
    p_ready = qk_free + 1;
    p_free = p_ready + 2;
    s_ready = p_free + 2;
    kt_ready = s_ready + 1;
    w_full = kt_ready + 2;
    o_full = w_full + 1;
    o_free = o_full + 2;
    drain = o_free + 2;
  }
};

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two values x as three bf16 pairs that add up to them: each term is the rest's
// leading 8 bits (cut off, so that the rest is exact and packing is a byte
// permute), the last one rounded.
__device__ __forceinline__ void split3(uint64_t x, uint32_t &a, uint32_t &b, uint32_t &c) {
  float f0, f1;
  upk2(x, f0, f1);
  uint32_t u0 = __float_as_uint(f0), u1 = __float_as_uint(f1);
  a = __byte_perm(u0, u1, 0x7632);
  x = add2(x, pk2(__uint_as_float((u0 & 0xffff0000u) ^ 0x80000000u), __uint_as_float((u1 & 0xffff0000u) ^ 0x80000000u)));
  upk2(x, f0, f1);
  u0 = __float_as_uint(f0), u1 = __float_as_uint(f1);
  b = __byte_perm(u0, u1, 0x7632);
  c = tc::pack_bf16x2(f0 - __uint_as_float(u0 & 0xffff0000u), f1 - __uint_as_float(u1 & 0xffff0000u));
}

// KB, VB: 64-column boxes of the q/k roles and of the v/o roles
template <int KB, int VB, bool REV, bool SUMMARY>
__global__ void __launch_bounds__(kThreads, 1)
    la_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, LaPass p) {
  using L = Layout<KB, VB, SUMMARY>;
  constexpr int ST = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  LaUnit u;
  const int unit = blockIdx.x / p.H, h = blockIdx.x - unit * p.H;
  if (!la_find_unit(p, unit, u)) return;  // every warp finds the same
  uint8_t *sm = tc::aligned_smem(smem_raw);
  const WaitCtl wait{p.status, p.wait_ns};
  const Bars<ST> bar(reinterpret_cast<uint64_t *>(sm + L::kBar));
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::kBar + L::kNumBars * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nb = (u.len + kC - 1) / kC;
  const float g = __ldg(p.g + h);
  // tables: lam^n, n = 0..64, times the scale of the products, the incoming state, the outgoing state
  float *tab_p = reinterpret_cast<float *>(sm + L::kTab), *tab_in = tab_p + 68, *tab_st = tab_in + 68;

  if (threadIdx.x == 64) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.free[i], SUMMARY ? 1 : 2);
    }
    mbar_init(bar.qk_full, 1);
    mbar_init(bar.qk_free, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.p_ready[i], 2);
      mbar_init(&bar.p_free[i], 1);
      mbar_init(&bar.o_full[i], 1);
      mbar_init(&bar.o_free[i], 2 * VB);
      mbar_init(&bar.k_done[i], 1);
      mbar_init(&bar.kt_ready[i], kStateWarps);
    }
    mbar_init(bar.s_ready, kStateWarps);
    mbar_init(bar.w_full, 1);
    mbar_init(bar.drain, 1);
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc(tslot, kTmCols);
    tmem_relinquish();
  }
  if (threadIdx.x <= kC) {
    const float w = la_pow(g, threadIdx.x);
    tab_p[threadIdx.x] = p.p_scale * w;
    tab_in[threadIdx.x] = p.in_scale * w;
    tab_st[threadIdx.x] = p.st_scale * w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  // processing order: block i is rows [64 blk, 64 blk + nv) of the segment
  auto block_of = [&](int i) { return REV ? nb - 1 - i : i; };
  auto rows_of = [&](int blk) { return min(kC, u.len - blk * kC); };

  if (warp == 2) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && nb > 0) {
      if (!SUMMARY) prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
      int i = 0;
      for (; i < nb; ++i) {
        const int st = i % ST, row = u.t0 + block_of(i) * kC;
        if (i >= ST && !mbar_wait(&bar.free[st], parity(i / ST - 1), wait)) break;
        uint8_t *base = sm + st * L::kStage;
        mbar_expect_tx(&bar.full[st], L::kLoad);
        for (int b = 0; b < KB; ++b) {
          if (!SUMMARY) tma_load_3d(base + L::kQ + b * kBox, &tm_q, &bar.full[st], 64 * b, h / p.gq, row);
          tma_load_3d(base + L::kK + b * kBox, &tm_k, &bar.full[st], 64 * b, h / p.gk, row);
        }
        for (int b = 0; b < VB; ++b)
          tma_load_3d(base + L::kV + b * kBox, &tm_v, &bar.full[st], 64 * b, h / p.gv, row);
      }
      // every load issued has landed before the CTA releases its shared memory
      for (int m = i > ST ? i - ST : 0; m < i; ++m) mbar_wait_drain(&bar.full[m % ST], parity(m / ST));
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t s0 = smem_u32(sm);
      // K-major operands: Q (A and B), K, P; MN-major: V (A), weighted K (B).  A's 128
      // rows run past Q's 64 into the shared memory behind it; those rows of the
      // result (and the lanes past 64 when VB = 1) are not read.
      const uint64_t dQ = desc_sw128(s0 + L::kQ, 16, 1024), dK = desc_sw128(s0 + L::kK, 16, 1024),
                     dV = desc_sw128(s0 + L::kV, kBox, 1024), dK1 = desc_sw128(s0 + L::kK, kBox, 1024),
                     dKt = desc_sw128(s0 + L::kKt, kBox, 1024),
                     dP = desc_sw128(s0 + L::kP, 16, 1024);
      constexpr uint32_t iQK = idesc_bf16(128, 64, false, false), iPV = idesc_bf16(128, 64, true, false),
                         iQS = idesc_bf16(128, 64, false, false), iW = idesc_bf16(128, 64 * KB, true, true);
      auto stage = [&](int i) { return (uint64_t)((i % ST) * (L::kStage / 16)); };
      auto scores = [&](int i) {
        mbar_wait(&bar.full[i % ST], parity(i / ST), wait);
        if (i > 0) mbar_wait(bar.qk_free, parity(i - 1), wait);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < KB; ++b)
          pipe::umma_k<4>(tmem + kTmQK, dQ + stage(i) + b * (kBox / 16), dK + stage(i) + b * (kBox / 16), pipe::kStepK,
                          pipe::kStepK, iQK, b > 0);
        umma_commit(bar.qk_full);
        umma_commit(&bar.k_done[i & 1]);
      };
      if (!SUMMARY && nb > 0) scores(0);
      for (int i = 0; i < nb; ++i) {
        const int ob = i & 1;
        if (!SUMMARY) {
          if (i + 1 < nb) scores(i + 1);
          if (i >= 2) mbar_wait(&bar.o_free[ob], parity(i / 2 - 1), wait);
          if (rows_of(block_of(i)) < kC) mbar_wait(&bar.kt_ready[ob], parity(i / 2), wait);  // V's tail
          mbar_wait(&bar.p_ready[ob], parity(i / 2), wait);
          tc_fence_after();
          pipe::umma_k<4>(tmem + kTmO + 64 * ob, dV + stage(i), dP + ob * (kBox / 16), pipe::kStepMN, pipe::kStepK, iPV,
                          false);
          umma_commit(&bar.p_free[ob]);
          mbar_wait(bar.s_ready, parity(i), wait);
          tc_fence_after();
#pragma unroll
          for (int b = 0; b < KB; ++b)
            pipe::umma_ts_k<4>(tmem + kTmOi + 64 * ob, tmem + kTmS + 32 * b, dQ + stage(i) + b * (kBox / 16), 8,
                               pipe::kStepK, iQS, b > 0);
          umma_commit(&bar.o_full[ob]);
        } else {
          mbar_wait(&bar.full[i % ST], parity(i / ST), wait);
          mbar_wait(bar.s_ready, parity(i), wait);
        }
        mbar_wait(&bar.kt_ready[ob], parity(i / 2), wait);
        tc_fence_after();
        const uint64_t v = dV + stage(i), kt = dKt + (uint64_t)(ob * 2 * KB * (kBox / 16));
        pipe::umma_k<4>(tmem + kTmW, v, dK1 + stage(i), pipe::kStepMN, pipe::kStepMN, iW, false);
        pipe::umma_k<4>(tmem + kTmW, v, kt, pipe::kStepMN, pipe::kStepMN, iW, true);
        pipe::umma_k<4>(tmem + kTmW, v, kt + KB * (kBox / 16), pipe::kStepMN, pipe::kStepMN, iW, true);
        umma_commit(bar.w_full);
        umma_commit(&bar.free[i % ST]);
      }
      // every MMA and every arrival of a commit has landed before the CTA ends
      umma_commit(bar.drain);
      mbar_wait_drain(bar.drain, 0);
      for (int m = nb > ST ? nb - ST : 0; m < nb; ++m) mbar_wait_drain(&bar.free[m % ST], parity(m / ST));
      if (nb > 0) mbar_wait_drain(bar.w_full, parity(nb - 1));
      if (!SUMMARY && nb > 0) {
        mbar_wait_drain(bar.qk_full, parity(nb - 1));
        for (int m = nb > 2 ? nb - 2 : 0; m < nb; ++m) {
          mbar_wait_drain(&bar.p_free[m & 1], parity(m / 2));
          mbar_wait_drain(&bar.o_full[m & 1], parity(m / 2));
          mbar_wait_drain(&bar.k_done[m & 1], parity(m / 2));
        }
      }
    }
  } else if (warp < 2) {
    // ------------------------------------------------------------ P
    if (!SUMMARY) {
      const int r = threadIdx.x;  // row of the block
      for (int i = 0; i < nb; ++i) {
        const int nv = rows_of(block_of(i));
        mbar_wait(bar.qk_full, parity(i), wait);
        tc_fence_after();
        float s[64];
        tmem_ld32(pipe::tmem_quad(tmem + kTmQK, 0), *reinterpret_cast<float(*)[32]>(s));
        tmem_ld32(pipe::tmem_quad(tmem + kTmQK, 32), *reinterpret_cast<float(*)[32]>(s + 32));
        tc_fence_before();
        pipe::warp_arrive(bar.qk_free);
        if (i >= 2) mbar_wait(&bar.p_free[i & 1], parity(i / 2 - 1), wait);
        const uint32_t dst = smem_u32(sm + L::kP + (i & 1) * kBox);
        // columns past the end: in order, only rows past it see them
        const int jmax = REV ? nv : kC;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int j = 8 * x + e, d = REV ? j - r : r - j;
            // a select, not a factor of zero: masked scores may be NaN
            v[e] = d >= 0 && j < jmax ? s[j] * tab_p[d] : 0.f;
          }
          pipe::sts_u4(dst + sw128_offset(r, 8 * x), tc::pack8(v));
        }
        fence_async_smem();
        pipe::warp_arrive(&bar.p_ready[i & 1]);
      }
    }
  } else if (warp < kStateWarp0) {
    // ------------------------------------------------------------ outputs
    if (!SUMMARY && warp < kOutWarp0 + 2 * VB) {
      constexpr int kOutThreads = 64 * VB;
      const int tt = threadIdx.x - 32 * kOutWarp0, quad = warp & 3;
      // the address this lane gives to a group of four fragments: row i, columns of v
      const int fi = 8 * (lane >> 4) + (lane & 7), fc = 32 * quad + 8 * ((lane >> 3) & 1);
      for (int i = 0; i < nb; ++i) {
        const int ob = i & 1, st = i % ST, blk = block_of(i), nv = rows_of(blk);
        const long long row0 = u.t0 + (long long)blk * kC;
        const uint32_t so = smem_u32(sm + st * L::kStage + L::kQ);
        float w[16];  // what the incoming state's part of this lane's columns i weighs
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * m + 2 * (lane & 3) + e;
            w[2 * m + e] = tab_in[REV ? max(nv - 1 - r, 0) : r + 1];
          }
        mbar_wait(&bar.o_full[ob], parity(i / 2), wait);
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // 16 lanes (columns of v) at a time
          uint32_t a[32], b[32];
          const uint32_t lanes = (uint32_t)(16 * half) << 16;
          tmem_ld_16x256_async(pipe::tmem_quad(tmem + kTmO + 64 * ob, 0) + lanes, a);
          tmem_ld_16x256_async(pipe::tmem_quad(tmem + kTmOi + 64 * ob, 0) + lanes, b);
          tmem_wait_ld32(a);
          tmem_wait_ld32(b);
          if (half == 1) {
            tc_fence_before();
            pipe::warp_arrive(&bar.o_free[ob]);
          }
          float o[32];
#pragma unroll
          for (int x = 0; x < 32; ++x)
            o[x] = fmaf(w[2 * (x >> 2) + (x & 1)], __uint_as_float(b[x]), __uint_as_float(a[x]));
          if (p.o_f32) {
            float *dst = static_cast<float *>(p.o) + row0 * p.os + (long long)h * p.dv;
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const int r = 8 * (x >> 2) + 2 * (lane & 3) + (x & 1), c = 32 * quad + 16 * half + (lane >> 2) + 4 * (x & 2);
              if (r < nv && c < p.dv) dst[r * p.os + c] = o[x];
            }
          } else {
#pragma unroll
            for (int m = 0; m < 8; m += 2) {
              const int r = 8 * m + fi, c = fc + 16 * half;
              stmatrix4_trans(so + (uint32_t)(c >> 6) * kBox + sw128_offset(r, c & 63),
                              tc::pack_bf16x2(o[4 * m], o[4 * m + 1]), tc::pack_bf16x2(o[4 * m + 2], o[4 * m + 3]),
                              tc::pack_bf16x2(o[4 * m + 4], o[4 * m + 5]), tc::pack_bf16x2(o[4 * m + 6], o[4 * m + 7]));
            }
          }
        }
        if (!p.o_f32) {
          fence_async_smem();
          asm volatile("bar.sync 2, %0;" ::"n"(kOutThreads) : "memory");
          if (nv < kC) {  // rows past the end belong to another sequence: row by row
            bf16 *out = static_cast<bf16 *>(p.o) + row0 * p.os + (long long)h * p.dv;
            for (int e = tt; e < nv * 8 * VB; e += kOutThreads) {
              const int r = e / (8 * VB), c = 8 * (e % (8 * VB));
              if (c < p.dv) {
                uint4 v;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                             : "r"(so + (uint32_t)(c >> 6) * kBox + sw128_offset(r, c & 63)));
                *reinterpret_cast<uint4 *>(out + r * p.os + c) = v;
              }
            }
            asm volatile("bar.sync 2, %0;" ::"n"(kOutThreads) : "memory");
          } else if (tt == 0) {
            for (int b = 0; b < VB; ++b)
              if (64 * b < p.dv) tma_store_3d(&tm_o, so + b * kBox, 64 * b, h, (int)row0);
            bulk_commit();
            bulk_wait_read0();
          }
        }
        if (tt == 0) mbar_arrive(&bar.free[st]);
      }
      if (tt == 0) bulk_wait0();
    }
  } else {
    // ------------------------------------------------------------ state
    constexpr int kCols = 32 * KB;  // state rows (dk) of a thread
    const int tt = threadIdx.x - 32 * kStateWarp0, quad = warp & 3, half = (warp - kStateWarp0) >> 2;
    const int c = 32 * quad + lane, a0 = half * kCols;
    const bool holds = quad < 2 * VB;  // this warp's lanes are columns of the state (warp-uniform)
    const size_t dd = (size_t)p.dk * p.dv;
    uint64_t S[kCols / 2];  // pairs along dk
    {
      const float *in = nullptr;
      int sa = p.sa, sb = p.sb;
      if (!SUMMARY && p.split) {
        in = p.seg_state + ((size_t)unit * p.H + h) * dd;
        sa = p.dv;
        sb = 1;
      } else if (!SUMMARY && p.init) {
        in = p.init + ((size_t)u.seq * p.H + h) * dd;
      }
      const bool live = in && holds && c < p.dv;
#pragma unroll
      for (int a = 0; a < kCols; a += 2) {  // dk is even
        float x = 0.f, y = 0.f;
        if (live && a0 + a < p.dk) {
          x = in[(size_t)(a0 + a) * sa + (size_t)c * sb];
          y = in[(size_t)(a0 + a + 1) * sa + (size_t)c * sb];
        }
        S[a / 2] = pk2(x, y);
      }
    }
    auto publish = [&] {  // S^T as the A operand: lane = column of v, bf16 pairs along dk
      if (!SUMMARY && holds) {
#pragma unroll
        for (int x = 0; x < kCols / 2; x += 16) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float f0, f1;
            upk2(S[x + e], f0, f1);
            w[e] = tc::pack_bf16x2(f0, f1);
          }
          tmem_st16_async(pipe::tmem_quad(tmem + kTmS, a0 / 2 + x), w);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      pipe::warp_arrive(bar.s_ready);
    };
    // the three terms of diag(lam^b) K of block i: the first over K itself
    const uint32_t s0 = smem_u32(sm);
    auto weigh = [&](int i) {
      const int st = i % ST, nv = rows_of(block_of(i));
      const uint32_t sk = s0 + st * L::kStage + L::kK, sv = s0 + st * L::kStage + L::kV,
                     skt = s0 + L::kKt + (uint32_t)(i & 1) * (2 * KB * kBox);
      mbar_wait(&bar.full[st], parity(i / ST), wait);
      if (!SUMMARY) mbar_wait(&bar.k_done[i & 1], parity(i / 2), wait);
#pragma unroll
      for (int x = 0; x < 2 * KB; ++x) {
        const int e = tt + 256 * x, r = (e >> 3) & 63, cc = e & 7;
        const uint32_t off = (uint32_t)(e >> 9) * kBox + sw128_offset(r, 8 * cc);
        uint4 raw, t0 = make_uint4(0, 0, 0, 0), t1 = t0, t2 = t0;
        if (r < nv) {
          const float w = tab_st[REV ? r + 1 : nv - 1 - r];
          const uint64_t w2 = pk2(w, w);
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w)
                       : "r"(sk + off));
          split3(mul2(w2, pk2(lo_f(raw.x), hi_f(raw.x))), t0.x, t1.x, t2.x);
          split3(mul2(w2, pk2(lo_f(raw.y), hi_f(raw.y))), t0.y, t1.y, t2.y);
          split3(mul2(w2, pk2(lo_f(raw.z), hi_f(raw.z))), t0.z, t1.z, t2.z);
          split3(mul2(w2, pk2(lo_f(raw.w), hi_f(raw.w))), t0.w, t1.w, t2.w);
        }
        pipe::sts_u4(sk + off, t0);
        pipe::sts_u4(skt + off, t1);
        pipe::sts_u4(skt + KB * kBox + off, t2);
      }
      if (nv < kC) {
#pragma unroll
        for (int x = 0; x < 2 * VB; ++x) {
          const int e = tt + 256 * x, r = (e >> 3) & 63, cc = e & 7;
          if (r >= nv) pipe::sts_u4(sv + (uint32_t)(e >> 9) * kBox + sw128_offset(r, 8 * cc), make_uint4(0, 0, 0, 0));
        }
      }
      fence_async_smem();
      pipe::warp_arrive(&bar.kt_ready[i & 1]);
    };
    const float2 full = la_pow2(g, kC);
    if (nb > 0) {
      publish();
      weigh(0);
    }
    for (int i = 0; i < nb; ++i) {
      if (i + 1 < nb) weigh(i + 1);  // while the tensor core works on block i
      const int nv = rows_of(block_of(i));
      const float2 carry = nv == kC ? full : la_pow2(g, nv);
      const uint64_t chi = pk2(carry.x, carry.x), clo = pk2(carry.y, carry.y);
      // W done: so are the MMAs issued before it, which read the weighted K and S^T
      mbar_wait(bar.w_full, parity(i), wait);
      tc_fence_after();
      if (holds) {
#pragma unroll
        for (int x = 0; x < kCols; x += 32) {
          float w[32];
          tmem_ld32(pipe::tmem_quad(tmem + kTmW, a0 + x), w);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            uint64_t &t = S[x / 2 + e];
            t = fma2(t, chi, fma2(t, clo, pk2(w[2 * e], w[2 * e + 1])));
          }
        }
      }
      if (i + 1 < nb) publish();
    }
    float *out = nullptr;
    int sa = p.sa, sb = p.sb;
    if (SUMMARY) {
      out = p.seg_state + ((size_t)unit * p.H + h) * dd;
      sa = p.dv;
      sb = 1;
    } else if (!p.split && p.fin) {
      out = p.fin + ((size_t)u.seq * p.H + h) * dd;
    }
    if (out && holds && c < p.dv) {
#pragma unroll
      for (int a = 0; a < kCols; a += 2) {
        float x, y;
        upk2(S[a / 2], x, y);
        if (a0 + a < p.dk) {
          out[(size_t)(a0 + a) * sa + (size_t)c * sb] = x;
          out[(size_t)(a0 + a + 1) * sa + (size_t)c * sb] = y;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

template <int KB, int VB, bool REV, bool SUMMARY>
void run_tc(const LaPass &p, cudaStream_t s) {
  using L = Layout<KB, VB, SUMMARY>;
  static bool once = (cudaFuncSetAttribute(la_tc_kernel<KB, VB, REV, SUMMARY>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes),
                      true);
  (void)once;
  CUtensorMap tq{}, tk, tv, to{};
  if ((!SUMMARY && !encode_tmap_bf16_heads(&tq, p.q, p.dk, p.Hq, p.total, p.qs * 2, kC)) ||
      (!SUMMARY && !p.o_f32 && !encode_tmap_bf16_heads(&to, p.o, p.dv, p.H, p.total, p.os * 2, kC)) ||
      !encode_tmap_bf16_heads(&tk, p.k, p.dk, p.Hk, p.total, p.ks * 2, kC) ||
      !encode_tmap_bf16_heads(&tv, p.v, p.dv, p.Hv, p.total, p.vs * 2, kC)) {
    note_host_error();
    return;
  }
  la_tc_kernel<KB, VB, REV, SUMMARY><<<(unsigned)p.H * (unsigned)p.nunits, kThreads, L::kBytes, s>>>(tq, tk, tv, to, p);
}

template <int KB, int VB>
void run_tc_mode(const LaPass &p, bool reverse, bool summary, cudaStream_t s) {
  if (reverse)
    summary ? run_tc<KB, VB, true, true>(p, s) : run_tc<KB, VB, true, false>(p, s);
  else
    summary ? run_tc<KB, VB, false, true>(p, s) : run_tc<KB, VB, false, false>(p, s);
}

}  // namespace

void launch_la_tc(const LaPass &p, bool reverse, bool summary, cudaStream_t s) {
  if (p.dk <= 64)
    p.dv <= 64 ? run_tc_mode<1, 1>(p, reverse, summary, s) : run_tc_mode<1, 2>(p, reverse, summary, s);
  else
    p.dv <= 64 ? run_tc_mode<2, 1>(p, reverse, summary, s) : run_tc_mode<2, 2>(p, reverse, summary, s);
}

}  // namespace ssd
