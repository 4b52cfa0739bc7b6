// The gated delta rule's gradients on the 5th-generation tensor cores, from the states before the chunks and the
// gradients of those behind them (dr_tc.cu), all chunks side by side.  In the tensors' own q and k (their lengths are
// in the factors), with L_ij = e^(G_i - G_j):
//     Wq_ij = scale L_ij / |q_i| / |k_j| (dO E^T)_ij b_j   (j <= i),    Wk_ij = -L_ij / |k_i| / |k_j| b_i (Z E^T)_ij b_j   (j < i)
//     dq = qin dO S^T + Wq K,      dk = kout b E dS^T - kin b Z S^T + Wk K + Wq^T Q + Wk^T K
//     dv = b Z,  dbeta = E.Z (rows)
//     dlog_decay_t = sum_(i >= t) (qin q_i.(dO S^T)_i - kin b_i k_i.(Z S^T)_i) + sum_(i >= t > j) M_ij
//                    + sum_(j < t) kout b_j k_j.(E dS^T)_j + e^Gall <S, dS>,    M = Wq o (Q K^T) + Wk o (K K^T)
// (what passes t, as at delta.h; here the sum of q.dq - v.dv had 2% left of each token's own addition in heads that forget
// fast, with operands of bf16.  The sum over pairs goes as row sums less column sums of the same fp32 M.)
// and the division by the lengths last: dq - q (q.dq) / |q|^2, likewise dk.
//
// Persistent CTAs; a CTA takes a chunk and a head of q and k and goes through the states that share it, dq and dk
// staying in registers.  Lanes 0-63 of the accumulators are the rows of dO and dq, lanes 64-127 those of Z and dk:
//     [dO; Z] S^T,   [dO; Z] E^T,   [Q; K] K^T,   [.; E] dS^T,   [Wq; Wk] K,   [.; Wq^T Wk^T] [Q; K]
// Warps: 0 TMA producer, 1 MMA issuer, 2-9 weights and gradients, 10 the decays' suffix sums.  A state's tensors are
// loaded again as soon as their products are made, beside the weights, the last two products and the sums.  Operands are
// rounded to bf16 (the outputs are bf16).
// 2 x 8192 tokens, 32 states of 16 heads of 128: 382 us.  What bounds it: warps 2-9 take 168 registers a
// thread, so that an SM has one CTA, and a step's weights, products and gradients follow one another.
#include "delta.h"
#include "tc_pipe.cuh"
#include "tc_util.cuh"

namespace ssd {

namespace {

using bf16 = __nv_bfloat16;
using namespace sm100;
using pipe::parity;

constexpr int kThreads = 352, kTeam = 256;
constexpr uint32_t kBox = 8192;  // [64 rows x 64 columns] bf16
constexpr uint32_t kTmA = 0, kTmC = 128, kTmW = 256, kTmB = 384, kTmCols = 512;  // products with S, dS, K (before: Q K^T); with E and, later, [Q; K]

// sums of a step, by the step's parity: a step's are read while the next one's are made
struct alignas(16) Sums {
  float kb[64];         // beta / |k|
  float row[2][2][64];  // of q's and k's halves: (dO S^T).q or (Z S^T).k with their factors, and M's row
  float col[4][64];     // M's columns, by quarters of its rows (q's halves, then k's)
  float add[2][64];     // k.(E dS^T) with its factors, by halves
  float ss[8], all;     // <S, dS>, by warps; e^Gall
};
static_assert(sizeof(Sums) % 16 == 0, "kb is read 16 bytes at a time");
struct Misc {
  Sums sums[2];
  float along[2][2][64];  // of dq and dk along q and k, by halves
};
template <int KB, int VB> struct Layout {
  static constexpr uint32_t kIn = 0;                             // dO, Z, E: boxes of each 64 columns behind one another
  static constexpr uint32_t kTile = KB * VB * kBox;
  static constexpr uint32_t kS = VB * 3 * kBox, kDs = kS + kTile;  // blocks of 8 columns of dk, all rows
  static constexpr uint32_t kQK = kDs + kTile;         // Q, K: likewise pairs
  static constexpr uint32_t kQKs = KB * 2 * kBox;               // two buffers
  static constexpr uint32_t kW = kQK + 2 * kQKs;                // Wq, Wk
  static constexpr uint32_t kRows = kW + 2 * kBox;
  static constexpr uint32_t kMisc = kRows + (sizeof(DrRows) + 15) / 16 * 16;
  static constexpr uint32_t kBar = kMisc + sizeof(Misc);
  static constexpr uint32_t kEnd = kBar + 18 * 8 + 16;
  static constexpr int kBytes = (int)kEnd + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};

struct Args {
  CUtensorMap q, k, dout, z, e, dq, dk;
  DrProblem p;
  DrGrads g;
  WaitCtl wait;
};

__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t par, const WaitCtl &w) {
  const uint32_t hint = w.limit_ns < kWaitHintNs ? (uint32_t)w.limit_ns : kWaitHintNs;
  if (__builtin_expect(mbar_try_wait_hint(bar, par, hint), 1)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < w.limit_ns) {
    if (mbar_try_wait_hint(bar, par, hint)) return true;
    if (*reinterpret_cast<volatile int *>(w.status) != 0) return false;
  }
  atomicExch(w.status, 1);
  return false;
}
__device__ __forceinline__ void team_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kTeam) : "memory"); }

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
  float x[8], y[8];
  tc::unpack8(a, x);
  tc::unpack8(b, y);
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
  return s;
}

template <int KB, int VB>
__global__ void __launch_bounds__(kThreads, 1) dr_grads_tc_kernel(const __grid_constant__ Args args) {
  using L = Layout<KB, VB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = tc::aligned_smem(smem_raw);
  const DrProblem &p = args.p;
  const DrGrads &g = args.g;
  const WaitCtl wait = args.wait;
  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::kBar);
  // rows (dO, Z, E, the factors) and states loaded / read; the others' names say what they are of
  uint64_t *in_full = bar, *in_free = bar + 1, *st_full = bar + 2, *st_free = bar + 3, *b_full = bar + 4, *w_ready = bar + 5,
           *out_full = bar + 6, *acc_free = bar + 7, *drain = bar + 8, *sums_full = bar + 9, *sums_free = bar + 11,
           *qk_full = bar + 13, *qk_free = bar + 15;  // [2] each
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::kBar + 18 * 8);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (warp == 0 && lane < 7) prefetch_tmap(&args.q + lane);
  if (threadIdx.x == 32) {
    mbar_init(in_full, 1);
    mbar_init(in_free, 9);
    mbar_init(st_full, 1);
    mbar_init(st_free, 9);
    mbar_init(b_full, 1);
    mbar_init(w_ready, 8);
    mbar_init(out_full, 1);
    mbar_init(acc_free, 8);
    mbar_init(drain, 1);
    for (int e = 0; e < 2; ++e) {
      mbar_init(&sums_full[e], 8);
      mbar_init(&sums_free[e], 1);
      mbar_init(&qk_full[e], 1);
      mbar_init(&qk_free[e], 9);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tslot, kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);
  const uint32_t s0 = smem_u32(sm);
  const int nunits = p.slots * p.Hk;
  // all roles walk the same units: a chunk's heads are neighbours, so that their v, dO and states are read together
  auto unit_at = [&](int u, int &slot, int &hk, int &t0, int &n) {
    slot = u / p.Hk;
    hk = u - slot * p.Hk;
    dr_chunk(p, slot, t0, n);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t m = 0, ms = 0, c = 0;  // steps (a chunk and a state head), their states' loads, units
      bool ok = true;
#pragma unroll 1
      for (int u = blockIdx.x; u < nunits && ok; u += gridDim.x) {
        int slot, hk, t0, n;
        unit_at(u, slot, hk, t0, n);
        if (n == 0) continue;
#pragma unroll 1
        for (int y = 0; y < p.group && ok; ++y, ++m) {
          const int h = hk * p.group + y;
          const size_t at = (size_t)slot * p.H + h;
          // a unit's q and k first: they are free the longest
          if (y == 0) {
            if (c >= 2 && !wait_on(&qk_free[c & 1], parity(c / 2 - 1), wait)) {
              ok = false;
              break;
            }
            uint8_t *to = sm + L::kQK + (c & 1) * L::kQKs;
            mbar_expect_tx(&qk_full[c & 1], 2 * KB * kBox);
            for (int b = 0; b < KB; ++b) {
              tma_load_3d(to + (2 * b) * kBox, &args.q, &qk_full[c & 1], 64 * b, hk, t0);
              tma_load_3d(to + (2 * b + 1) * kBox, &args.k, &qk_full[c & 1], 64 * b, hk, t0);
            }
            ++c;
          }
          if (m > 0 && !wait_on(st_free, parity(m - 1), wait)) {
            ok = false;
            break;
          }
          mbar_expect_tx(st_full, 2 * L::kTile);
          pipe::bulk_load(sm + L::kS, reinterpret_cast<const uint8_t *>(p.S) + at * L::kTile, L::kTile, st_full);
          pipe::bulk_load(sm + L::kDs, reinterpret_cast<const uint8_t *>(p.dS) + at * L::kTile, L::kTile, st_full);
          ++ms;
          if (m > 0 && !wait_on(in_free, parity(m - 1), wait)) {
            ok = false;
            break;
          }
          mbar_expect_tx(in_full, 3 * VB * kBox + (uint32_t)sizeof(DrRows));
          pipe::bulk_load(sm + L::kRows, p.rows + at, sizeof(DrRows), in_full);
          for (int b = 0; b < VB; ++b) {
            tma_load_3d(sm + L::kIn + (3 * b) * kBox, &args.dout, in_full, 64 * b, h, t0);
            tma_load_3d(sm + L::kIn + (3 * b + 1) * kBox, &args.z, in_full, 64 * b, h, t0);
            tma_load_3d(sm + L::kIn + (3 * b + 2) * kBox, &args.e, in_full, 64 * b, h, t0);
          }
        }
      }
      // every load issued has landed before the CTA releases its shared memory
      if (m > 0) mbar_wait_drain(in_full, parity(m - 1));
      if (ms > 0) mbar_wait_drain(st_full, parity(ms - 1));
#pragma unroll 1
      for (uint32_t x = c > 2 ? c - 2 : 0; x < c; ++x) mbar_wait_drain(&qk_full[x & 1], parity(x / 2));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t el = elect_one();
    const uint64_t dIn = desc_sw128(s0 + L::kIn, 16, 1024);                                     // K-major, 128 rows
    const uint64_t dS = desc_blocks_mn(s0 + L::kS, 128, VB * 1024), dDs = desc_blocks_mn(s0 + L::kDs, 128, VB * 1024);
    const uint64_t dQK = desc_sw128(s0 + L::kQK, 2 * kBox, 1024);                               // MN-major
    const uint64_t dQKk = desc_sw128(s0 + L::kQK, 16, 1024);                                    // K-major
    const uint64_t dW = desc_sw128(s0 + L::kW, 16, 1024);
    // transposed: lanes 64-127 are its 64 columns, lanes 0-63 those of what lies two boxes before
    const uint64_t dWt = desc_sw128(s0 + L::kW - 2 * kBox, 2 * kBox, 1024);
    constexpr uint32_t iB = idesc_bf16(128, 64, false, false), iN = idesc_bf16(128, 64 * KB, false, true),
                       iT = idesc_bf16(128, 64 * KB, true, true);
    constexpr uint64_t kB = kBox / 16;
    uint32_t m = 0, c = 0;
#pragma unroll 1
    for (int u = blockIdx.x; u < nunits; u += gridDim.x) {
      int slot, hk, t0, n;
      unit_at(u, slot, hk, t0, n);
      if (n == 0) continue;
#pragma unroll 1
      for (int y = 0; y < p.group; ++y, ++m) {
        wait_on(in_full, parity(m), wait);
        if (m > 0) wait_on(acc_free, parity(m - 1), wait);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < VB; ++b)  // [dO; Z] E^T
          pipe::umma_k_el<4>(el, tmem + kTmB, dIn + 3 * b * kB, dIn + (3 * b + 2) * kB, pipe::kStepK, pipe::kStepK, iB, b > 0);
        const uint64_t qk = (uint64_t)((c & 1) * (L::kQKs / 16));
        if (y == 0) {
          wait_on(&qk_full[c & 1], parity(c / 2), wait);
          tc_fence_after();
        }
#pragma unroll
        for (int b = 0; b < KB; ++b)  // [Q; K] K^T
          pipe::umma_k_el<4>(el, tmem + kTmW, dQKk + qk + 2 * b * kB, dQKk + qk + (2 * b + 1) * kB, pipe::kStepK, pipe::kStepK, iB, b > 0);
        umma_commit_el(el, b_full);
        wait_on(st_full, parity(m), wait);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < VB; ++b)  // [dO; Z] S^T
          pipe::umma_k_el<4>(el, tmem + kTmA, dIn + 3 * b * kB, dS + b * 64, pipe::kStepK, 16, iN, b > 0);
#pragma unroll
        for (int b = 0; b < VB; ++b)  // [Z; E] dS^T
          pipe::umma_k_el<4>(el, tmem + kTmC, dIn + (3 * b + 1) * kB, dDs + b * 64, pipe::kStepK, 16, iN, b > 0);
        umma_commit_el(el, st_free);
        umma_commit_el(el, in_free);
        wait_on(w_ready, parity(m), wait);
        tc_fence_after();
        pipe::umma_k_el<4>(el, tmem + kTmW, dW, dQK + qk + kB, pipe::kStepK, pipe::kStepMN, iN, false);          // [Wq; Wk] K
        pipe::umma_k_el<8>(el, tmem + kTmB, dWt, dQK + qk, pipe::kStepMN, pipe::kStepMN, iT, false);             // [Wq^T Wk^T] [Q; K]
        umma_commit_el(el, out_full);
        if (y + 1 == p.group) {
          umma_commit_el(el, &qk_free[c & 1]);
          ++c;
        }
      }
    }
    umma_commit_el(el, drain);
    mbar_wait_drain(drain, 0);
    if (m > 0) {
      mbar_wait_drain(in_free, parity(m - 1));
      mbar_wait_drain(st_free, parity(m - 1));
      mbar_wait_drain(b_full, parity(m - 1));
      mbar_wait_drain(out_full, parity(m - 1));
#pragma unroll 1
      for (uint32_t x = c > 2 ? c - 2 : 0; x < c; ++x) mbar_wait_drain(&qk_free[x & 1], parity(x / 2));
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ sums of the decays' gradients, two rows a lane
    uint32_t m = 0;
#pragma unroll 1
    for (int u = blockIdx.x; u < nunits; u += gridDim.x) {
      int slot, hk, t0, n;
      unit_at(u, slot, hk, t0, n);
      if (n == 0) continue;
#pragma unroll 1
      for (int y = 0; y < p.group; ++y, ++m) {
        const int h = hk * p.group + y;
        const Sums &x = reinterpret_cast<const Sums *>(sm + L::kMisc)[m & 1];
        wait_on(&sums_full[m & 1], parity(m / 2), wait);
        float d[2], c[2], end = 0.f;  // what passes later tokens, and what is added before
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * lane + e;
          d[e] = c[e] = 0.f;
          if (r < n) {
            d[e] = ((x.row[0][0][r] + x.row[0][1][r]) + (x.row[1][0][r] + x.row[1][1][r])) -
                   ((x.col[0][r] + x.col[1][r]) + (x.col[2][r] + x.col[3][r]));
            c[e] = x.add[0][r] + x.add[1][r];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) end += x.ss[e];
        end *= x.all;
        pipe::warp_arrive(&sums_free[m & 1]);
        d[0] += d[1];
        float after = d[0], before = c[0] + c[1];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const float z = __shfl_down_sync(0xffffffffu, after, o), w = __shfl_up_sync(0xffffffffu, before, o);
          if (lane + o < 32) after += z;
          if (lane >= o) before += w;
        }
        // without the lane's own, which may be far larger: no decay has touched what the last row adds
        const float z = __shfl_down_sync(0xffffffffu, after, 1), w = __shfl_up_sync(0xffffffffu, before, 1);
        after = lane < 31 ? z : 0.f;
        before = lane > 0 ? w : 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * lane + e;
          if (r < n) static_cast<bf16 *>(g.dg)[(size_t)(t0 + r) * g.dgs + h] = __float2bfloat16_rn((d[e] + after) + (before + (e ? c[0] : 0.f)) + end);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ weights and gradients
    constexpr int kCols = 32 * KB;  // columns of dk of a thread
    const int et = threadIdx.x - 64, quad = warp & 3, sub = (warp - 2) >> 2;
    const bool is_k = quad >= 2;                       // lanes 64-127: rows of Z and dk
    const int i = 32 * (quad & 1) + lane;              // the thread's row
    Misc &misc = *reinterpret_cast<Misc *>(sm + L::kMisc);
    const DrRows &rw = *reinterpret_cast<const DrRows *>(sm + L::kRows);
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    uint32_t m = 0, c = 0;
#pragma unroll 1
    for (int u = blockIdx.x; u < nunits; u += gridDim.x) {
      int slot, hk, t0, n;
      unit_at(u, slot, hk, t0, n);
      if (n == 0) continue;
      const uint32_t qk0 = s0 + L::kQK + (c & 1) * L::kQKs;
      float len = 0.f;  // 1 / |q|^2 or 1 / |k|^2
      float acc[kCols], along = 0.f;  // along: q.dq or k.dk, the thread's part
#pragma unroll
      for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
#pragma unroll 1
      for (int y = 0; y < p.group; ++y, ++m) {
        const int h = hk * p.group + y;
        Sums &x = reinterpret_cast<Sums *>(sm + L::kMisc)[m & 1];
        if (m >= 2) wait_on(&sums_free[m & 1], parity(m / 2 - 1), wait);
        wait_on(in_full, parity(m), wait);
        if (et < 64) x.kb[et] = rw.rk[et] * rw.beta[et];
        if (et == 0) x.all = rw.all_hi + rw.all_lo;
        team_sync();
        // <S, dS>, while the first products are made
        wait_on(st_full, parity(m), wait);
        float ss = 0.f;
#pragma unroll 4
        for (int e = et; e < KB * VB * 512; e += kTeam)
          ss = dot8(*reinterpret_cast<const uint4 *>(sm + L::kS + 16 * e), *reinterpret_cast<const uint4 *>(sm + L::kDs + 16 * e), ss);
        pipe::warp_arrive(st_free);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) x.ss[warp - 2] = ss;
        // weights
        const float rk_i = rw.rk[i], rq_i = rw.rq[i], beta_i = rw.beta[i];
        const float fa = is_k ? -rw.kin[i] * beta_i : rw.qin[i], fc = rw.kout[i] * beta_i;
        const float hi = rw.ghi[i], lo = rw.glo[i];
        len = is_k ? rk_i * rk_i : rq_i * rq_i;
        if (y == 0) {
          if (n < kDrC) {  // rows past the end belong to another sequence
            wait_on(&qk_full[c & 1], parity(c / 2), wait);
            for (int e = et; e < (kDrC - n) * 16 * KB; e += kTeam) {
              const int b = e % (16 * KB), r = n + e / (16 * KB);
              pipe::sts_u4(qk0 + (uint32_t)(b >> 3) * kBox + sw128_offset(r, 8 * (b & 7)), make_uint4(0, 0, 0, 0));
            }
          }
        }
        wait_on(b_full, parity(m), wait);
        tc_fence_after();
        const float fw = is_k ? -rk_i * beta_i : rq_i * p.scale;
        float pairs = 0.f, own = 0.f;  // M's row, and q's own addition
        const int last = i < n ? is_k ? i - 1 : i : -1;  // the row's columns are up to this one
#pragma unroll
        for (int j0 = 32 * sub; j0 < 32 * sub + 32; j0 += 16) {
          float v[16], w8[8];
          tmem_ld16(lanes + kTmB + j0, v);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 gh = *reinterpret_cast<const float4 *>(rw.ghi + j0 + e), gl = *reinterpret_cast<const float4 *>(rw.glo + j0 + e),
                         kb = *reinterpret_cast<const float4 *>(x.kb + j0 + e);
            const float f[4] = {__expf((hi - gh.x) + (lo - gl.x)) * kb.x, __expf((hi - gh.y) + (lo - gl.y)) * kb.y,
                                __expf((hi - gh.z) + (lo - gl.z)) * kb.z, __expf((hi - gh.w) + (lo - gl.w)) * kb.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[e + j] = j0 + e + j <= last ? v[e + j] * (f[j] * fw) : 0.f;
          }
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w8[j] = v[e + j];
            pipe::sts_u4(s0 + L::kW + (is_k ? kBox : 0) + sw128_offset(i, j0 + e), tc::pack8(w8));
          }
          {
            float M[16];  // of columns before the row's
            tmem_ld16(lanes + kTmW + j0, M);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float p_ij = j0 + e <= last ? v[e] * M[e] : 0.f;
              if (j0 + e == i) own = p_ij;
              M[e] = j0 + e < i ? p_ij : 0.f;
              pairs += M[e];
            }
            // column sums over the warp's rows: halves of the columns go to halves of the lanes
#pragma unroll
            for (int k = 16, e = 8; k >= 2; k /= 2, e /= 2)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (j < e) {
                  const float give = lane & k ? M[j] : M[j + e], mine = lane & k ? M[j + e] : M[j];
                  M[j] = mine + __shfl_xor_sync(0xffffffffu, give, k);
                }
            M[0] += __shfl_xor_sync(0xffffffffu, M[0], 1);
            if (!(lane & 1)) x.col[quad][j0 + (lane >> 1)] = M[0];
          }
        }
        tc_fence_before();
        fence_async_smem();
        pipe::warp_arrive(w_ready);
        constexpr int kRounds = 2 * VB;  // 16 bytes of a row a thread and round
        // dv, dbeta: the rounds side by side
        uint4 zw[kRounds], ew[kRounds];
        float db[kRounds];
#pragma unroll
        for (int o = 0; o < kRounds; ++o) {
          const int e = et + kTeam * o, r = e / (8 * VB), b = e % (8 * VB) >> 3;
          const uint32_t at = sw128_offset(r, 8 * (e & 7));
          zw[o] = *reinterpret_cast<const uint4 *>(sm + L::kIn + (3 * b + 1) * kBox + at);
          ew[o] = *reinterpret_cast<const uint4 *>(sm + L::kIn + (3 * b + 2) * kBox + at);
        }
#pragma unroll
        for (int o = 0; o < kRounds; ++o) {
          const int e = et + kTeam * o, r = e / (8 * VB), col = 8 * (e % (8 * VB));
          db[o] = 0.f;
          if (r < n && col < p.dv) {
            db[o] = dot8(zw[o], ew[o], 0.f);
            const float beta = rw.beta[r];
            float z[8];
            tc::unpack8(zw[o], z);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] *= beta;
            *reinterpret_cast<uint4 *>(static_cast<bf16 *>(g.dv) + (size_t)(t0 + r) * g.dvs + (size_t)h * p.dv + col) = tc::pack8(z);
          }
        }
#pragma unroll
        for (int z = 4 * VB; z >= 1; z >>= 1) {
#pragma unroll
          for (int o = 0; o < kRounds; ++o) db[o] += __shfl_xor_sync(0xffffffffu, db[o], z);
        }
#pragma unroll
        for (int o = 0; o < kRounds; ++o) {
          const int e = et + kTeam * o, r = e / (8 * VB);
          if (e % (8 * VB) == 0 && r < n) static_cast<bf16 *>(g.db)[(size_t)(t0 + r) * g.dbs + h] = __float2bfloat16_rn(db[o]);
        }
        pipe::warp_arrive(in_free);
        // gradients
        wait_on(out_full, parity(m), wait);
        if (y == 0) wait_on(&qk_full[c & 1], parity(c / 2), wait);
        tc_fence_after();
        float read = 0.f, add = 0.f;  // (dO S^T).q or (Z S^T).k; k and what is added to the state
#pragma unroll
        for (int j0 = 0; j0 < kCols; j0 += 16) {
          const int col = kCols * sub + j0;
          float a[16], w[16], t[16];
          tmem_ld16(lanes + kTmA + col, a);
          tmem_ld16(lanes + kTmW + col, w);
          if (is_k) {
            tmem_ld16(lanes + kTmB + col, t);
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] += t[e];
            tmem_ld16(lanes + kTmC + col, t);
#pragma unroll
            for (int e = 0; e < 16; ++e) t[e] *= fc;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            w[e] = fmaf(fa, a[e], w[e]);
            if (is_k) w[e] += t[e];
            acc[j0 + e] += w[e];
          }
          const uint32_t tile = qk0 + (2 * (col >> 6) + is_k) * kBox;
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            float r8[8];
            tc::unpack8(pipe::lds_sw128(tile, i, ((col & 63) + e) >> 3), r8);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              read = fmaf(r8[j], a[e + j], read);
              if (is_k) {
                add = fmaf(r8[j], t[e + j], add);
                along = fmaf(r8[j], w[e + j], along);
              }
            }
          }
        }
        tc_fence_before();
        pipe::warp_arrive(acc_free);
        read = fmaf(fa, read, pairs);
        x.row[is_k][sub][i] = read;
        if (is_k)
          x.add[sub][i] = add;
        else
          along += read + own;
        pipe::warp_arrive(&sums_full[m & 1]);
      }
      // the division by the lengths, and out: through the places of q and k, which nobody reads any more
      const uint32_t tile0 = qk0 + is_k * kBox;
      float f = 0.f;
      if (p.norm) {
        misc.along[is_k][sub][i] = along;
        team_sync();
        f = (misc.along[is_k][0][i] + misc.along[is_k][1][i]) * len;
      }
#pragma unroll
      for (int e = 0; e < kCols; e += 8) {
        const int col = kCols * sub + e;
        const uint32_t at = tile0 + 2 * (col >> 6) * kBox + sw128_offset(i, col & 63);
        float v[8], r8[8];
        tc::unpack8(pipe::lds_sw128(tile0 + 2 * (col >> 6) * kBox, i, (col & 63) >> 3), r8);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = p.norm ? acc[e + j] - r8[j] * f : acc[e + j];
        pipe::sts_u4(at, tc::pack8(v));
      }
      fence_async_smem();
      team_sync();
      if (n == kDrC) {
        if (et == 0) {
          for (int b = 0; b < KB; ++b)
            if (64 * b < p.dk) {
              tma_store_3d(&args.dq, qk0 + 2 * b * kBox, 64 * b, hk, t0);
              tma_store_3d(&args.dk, qk0 + (2 * b + 1) * kBox, 64 * b, hk, t0);
            }
          bulk_commit();
          bulk_wait_read0();
        }
      } else {  // rows past the end belong to another sequence: row by row
        for (int e = et; e < n * 16 * KB; e += kTeam) {
          const int r = e / (16 * KB), b = e % (16 * KB) >> 3, ch = e & 7, col = 64 * (b >> 1) + 8 * ch;
          if (col < p.dk) {
            bf16 *out = b & 1 ? static_cast<bf16 *>(g.dk) + (size_t)(t0 + r) * g.dks : static_cast<bf16 *>(g.dq) + (size_t)(t0 + r) * g.dqs;
            *reinterpret_cast<uint4 *>(out + hk * p.dk + col) = pipe::lds_sw128(qk0 + b * kBox, r, ch);
          }
        }
      }
      pipe::warp_arrive(&qk_free[c & 1]);
      ++c;
    }
    if (et == 0) bulk_wait0();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

template <int KB, int VB> void run(Args &args, cudaStream_t s) {
  using L = Layout<KB, VB>;
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(dr_grads_tc_kernel<KB, VB>), L::kBytes, allowed);
  const int units = args.p.slots * args.p.Hk, sms = device_sm_count();
  dr_grads_tc_kernel<KB, VB><<<units < sms ? units : sms, kThreads, L::kBytes, s>>>(args);
}

}  // namespace

void launch_dr_grads_tc(const DrProblem &p, const void *dout, long long dos, const DrGrads &g, cudaStream_t s) {
  Args args;
  args.p = p;
  args.g = g;
  args.wait = {p.status, p.wait_ns};
  const uint64_t es = (uint64_t)p.H * p.dv * 2;
  if (!encode_tmap_bf16_heads(&args.q, p.q, p.dk, p.Hk, p.total, p.qs * 2, kDrC) ||
      !encode_tmap_bf16_heads(&args.k, p.k, p.dk, p.Hk, p.total, p.ks * 2, kDrC) ||
      !encode_tmap_bf16_heads(&args.dout, dout, p.dv, p.H, p.total, dos * 2, kDrC) ||
      !encode_tmap_bf16_heads(&args.z, p.Z, p.dv, p.H, p.total, es, kDrC) ||
      !encode_tmap_bf16_heads(&args.e, p.E, p.dv, p.H, p.total, es, kDrC) ||
      !encode_tmap_bf16_heads(&args.dq, g.dq, p.dk, p.Hk, p.total, g.dqs * 2, kDrC) ||
      !encode_tmap_bf16_heads(&args.dk, g.dk, p.dk, p.Hk, p.total, g.dks * 2, kDrC)) {
    note_host_error();
    return;
  }
  const int kb = la_tc_boxes(p.dk), vb = la_tc_boxes(p.dv);
  if (kb == 1)
    vb == 1 ? run<1, 1>(args, s) : run<1, 2>(args, s);
  else
    vb == 1 ? run<2, 1>(args, s) : run<2, 2>(args, s);
}

}  // namespace ssd
