// The gated delta rule on the 5th-generation tensor cores (tcgen05, accumulators and A operands in TMEM): bf16 tensors,
// widths up to 128.  The chain of chunks, forward and in reverse; the formulas are at delta.h.
//
// A CTA takes one sequence and head and walks its chunks.  Everything is formed transposed, so that dv (up to 128)
// fills the accumulators' lanes and the state stays in its warps' registers (lane = dv):
//     X^T = S^T K^T,   Y = V - kin X,   E = Y - N (b Y),   S = e^Gall S + W,   W^T = (kout b E)^T K
//     O^T = (qin S^T Q^T) + (b E)^T P^T                     (b E and P in two terms as well)
// In reverse the same four steps, with the gradient of the state for the state:
//     X^T = dS^T K^T,   dD = kout X + P^T dO,   Z = dD - N^T (b dD),   dS = e^Gall dS + W,
//     W^T = (qin dO)^T Q - (kin b Z)^T K
// What ends in a state is a sum in fp32, and an operand that is not a bf16 tensor of the user's is a sum of two bf16 terms
// (16 bits; products of the two low terms are left out), which leaves a relative error of about 3e-6 in a state: 1/1000 of
// a bf16 tensor's own rounding.  A third term would make it fp32's; it takes half as many products again of
// X and W, twice those of N, and the columns of TMEM that W has.  Outputs are 0.0017 off, by their one rounding.  (With b E
// and P in one term each they were 0.0026 off, and 0.01 where keys are nearly equal and a chunk's additions cancel; the second
// terms, made and multiplied beside W, took 3.5% more of a chain and 5% of the tables.)
//
// Warps:
//   0       TMA producer: K, Q, V (reverse: dO), and the chunk's N, P and row factors, two stages
//   1       MMA issuer
//   2, 3    a sequence's last chunk: rows past its end become zeros in shared memory
//   4-11    Y and E (reverse: dD and Z), as fragments of 16 lanes x 32 tokens
//   12-19   state
//   20-23   outputs; in reverse the two terms of (qin dO)^T
// What bounds it: the chain from state to state, its products (16 of X, 12 of N, 8 of W, 46 to 66 cycles each) and
// five hand-offs between tensor core and warps.  4 x 8192 tokens, 32 heads of 128 (128 chains of 128 chunks): 320 us,
// 2.5 us a chunk; 2 x 8192 tokens with the states and E kept 296 us, in reverse 384 us.  A CTA has an SM to
// itself (TMEM, shared memory), so fewer chains than SMs leave SMs idle: dr_segment_chunks in api_delta.cu cuts them.
#include "delta.h"
#include "tc_pipe.cuh"
#include "tc_util.cuh"

namespace ssd {

namespace {

using bf16 = __nv_bfloat16;
using namespace sm100;
using pipe::parity;

constexpr int kThreads = 768;
constexpr int kElemWarp0 = 4, kStateWarp0 = 12, kOutWarp0 = 20;
constexpr uint32_t kBox = 8192;  // [64 rows x 64 columns] bf16
constexpr int kStages = 2;

// TMEM columns: the state's terms (64 each), X and then N's product, outputs (reverse: P^T dO), the terms of b Y and then
// of the additions (32 each), those of b E for the outputs or of qin dO, W
constexpr uint32_t kTmS = 0, kTmX = 128, kTmO = 192, kTmY = 256, kTmD = 320, kTmW = 384, kTmCols = 512;

enum Mode { kOut, kStates, kReverse, kSum };  // outputs; states and E for the backward pass; the reverse chain; only the last state

template <int KB, int VB, int MODE> struct Layout {
  static constexpr uint32_t kK = 0, kQ = KB * kBox, kV = kQ + KB * kBox, kN = kV + VB * kBox, kP = kN + 2 * kBox;
  static constexpr uint32_t kRows = kP + 2 * kBox, kStage = (kRows + sizeof(DrRows) + 1023) / 1024 * 1024;
  static constexpr uint32_t kO = kStages * kStage;  // a chunk's outputs, on their way to TMA
  static constexpr uint32_t kKept = kO + VB * kBox;  // a kept state, likewise
  static constexpr uint32_t kBar = kKept + (MODE == kOut || MODE == kSum ? 0 : KB * VB * kBox);
  static constexpr int kNumBars = 2 * kStages + 14;
  static constexpr uint32_t kEnd = kBar + kNumBars * 8 + 16;
  static constexpr int kBytes = (int)kEnd + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};

struct Bars {
  uint64_t *full, *free;  // [stages] loaded / read
  uint64_t *patched;      // the last chunk's rows past the end are zeros
  uint64_t *s_ready;      // the state's terms in TMEM
  uint64_t *x_full;       // X
  uint64_t *y_ready;      // b Y's terms in TMEM
  uint64_t *n_full;       // N's product
  uint64_t *d_ready;      // the additions' terms in TMEM
  uint64_t *e_ready;      // and those for the outputs
  uint64_t *w_full;       // W
  uint64_t *q_full, *q_ready;  // outputs' part of the state formed / scaled; reverse: W's part of dO formed / its terms in TMEM
  uint64_t *o_full, *o_free;   // outputs formed / read; reverse: P^T dO
  uint64_t *drain;
  __device__ explicit Bars(uint64_t *b) {
    full = b;
    free = b + kStages;
    patched = b + 2 * kStages;
    s_ready = patched + 1;
    x_full = patched + 2;
    y_ready = patched + 3;
    n_full = patched + 4;
    d_ready = patched + 5;
    w_full = patched + 6;
    q_full = patched + 7;
    q_ready = patched + 8;
    o_full = patched + 9;
    o_free = patched + 10;
    drain = patched + 11;
    e_ready = patched + 12;
  }
};

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// a packed pair likewise (tc::split2)
__device__ __forceinline__ void split2(uint64_t v, uint32_t &a, uint32_t &b) {
  float x, y;
  upk2(v, x, y);
  tc::split2(x, y, a, b);
}

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
template <int ID, int THREADS> __device__ __forceinline__ void role_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

struct Args {
  CUtensorMap q, k, v, o;  // v: dO in reverse; o: outputs, E or Z
  DrProblem p;
  const float *first;  // states (gradients of final states) that the chain starts from, or null
  float *last;         // and where it ends, or null
  bf16 *out;           // o's rows
  long long os;
  bf16 *kept;  // the state before each chunk, the gradient of the one behind
  WaitCtl wait;
  // Sequences cut into segments of so many chunks (0: whole ones): `first` and `last` are then the segments', at their
  // places (dr_segment), but for the last segment's of a sequence, which ends in `fin`
  int seg, places;
  float *fin;
  int what;  // kSum: 0 the segment's state from zero, 1 what becomes of the unit matrix without additions, 2 both (blockIdx.y)
};

template <int KB, int VB, int MODE>
__global__ void __launch_bounds__(kThreads, 1) dr_tc_kernel(const __grid_constant__ Args args) {
  using L = Layout<KB, VB, MODE>;
  constexpr bool kRev = MODE == kReverse, kKeeps = kRev || MODE == kStates;  // what the gradients need
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = tc::aligned_smem(smem_raw);
  const DrProblem &p = args.p;
  const WaitCtl wait = args.wait;
  const Bars bar(reinterpret_cast<uint64_t *>(sm + L::kBar));
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::kBar + L::kNumBars * 8);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int place = blockIdx.x / p.H, h = blockIdx.x - place * p.H;
  int seq = place, a, len, slot0;
  bool ends = true;  // the segment is its sequence's last
  if (args.seg)
    dr_segment(p, args.seg, place, seq, a, len, slot0, ends);
  else
    dr_seq(p, seq, a, len, slot0);
  // the places of no segment; a last segment's sum is not asked for
  if (args.seg && (seq < 0 || (MODE == kSum && ends))) return;
  // the unit matrix's columns are dk
  const bool unit = MODE == kSum && (args.what == 2 ? blockIdx.y == 1 : args.what == 1);
  const int dv = unit ? p.dk : p.dv;
  const int nc = __shfl_sync(0xffffffffu, (len + kDrC - 1) / kDrC, 0);
  // processing order: the i-th chunk, its rows
  auto chunk = [&](int i) { return kRev ? nc - 1 - i : i; };
  auto live = [&](int i) { return min(kDrC, len - chunk(i) * kDrC); };
  const int tail = kRev ? 0 : nc - 1;
  const bool partial = len % kDrC != 0;  // the tail is

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&args.k);
    prefetch_tmap(&args.q);
    prefetch_tmap(&args.v);
    prefetch_tmap(&args.o);
  }
  if (threadIdx.x == 64) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      // the issuer's commit, the Y and state warps, the outputs' warps and those of a partial chunk where there are any
      mbar_init(&bar.free[i], 1 + 8 * VB + (MODE == kOut || kRev ? 2 * VB : 0) + (partial ? 2 : 0));
    }
    mbar_init(bar.patched, 2);
    mbar_init(bar.s_ready, 4 * VB);
    mbar_init(bar.x_full, 1);
    mbar_init(bar.y_ready, 4 * VB);
    mbar_init(bar.n_full, 1);
    mbar_init(bar.d_ready, 4 * VB);
    mbar_init(bar.e_ready, 4 * VB);
    mbar_init(bar.w_full, 1);
    mbar_init(bar.q_full, 1);
    mbar_init(bar.q_ready, 2 * VB);
    mbar_init(bar.o_full, 1);
    mbar_init(bar.o_free, kRev ? 4 * VB : 2 * VB);
    mbar_init(bar.drain, 1);
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
  auto stage = [&](int i) { return (uint32_t)(i % kStages) * L::kStage; };
  auto rows_of = [&](int i) { return s0 + stage(i) + L::kRows; };
  auto wait_full = [&](int i) {
    wait_on(&bar.full[i % kStages], parity(i / kStages), wait);
    if (partial && i == tail) wait_on(bar.patched, 0, wait);
  };

  // The block is launched with 768 x 80 registers, 128 x 480; the warps of Y and E and the state's take what others do not
  // need (without spills of theirs a chunk of kStates takes 2.5 us, with them 4.1).
  constexpr bool kIdle = MODE == kStates || MODE == kSum;  // the last four warps
  constexpr int kElemRegs = kIdle ? 88 : 80, kStateRegs = kIdle ? 120 : 104, kLastRegs = kIdle ? 32 : 80;
  static_assert(32 + 2 * kElemRegs + 2 * kStateRegs + kLastRegs <= 480, "registers");
  if (warp < kElemWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        const int hk = h / p.group;
        int i = 0;
#pragma unroll 1
        for (; i < nc; ++i) {
          const int st = i % kStages, row = a + chunk(i) * kDrC;
          if (i >= kStages && !wait_on(&bar.free[st], parity(i / kStages - 1), wait)) break;
          uint8_t *base = sm + stage(i);
          const size_t at = (size_t)(slot0 + chunk(i)) * p.H + h;
          const uint8_t *tiles = reinterpret_cast<const uint8_t *>(p.N) + at * (4 * kBox);
          constexpr uint32_t kQBytes = MODE == kStates || MODE == kSum ? 0 : KB * kBox;
          constexpr uint32_t kMats = MODE == kOut || MODE == kReverse ? 4 * kBox : 2 * kBox;
          mbar_expect_tx(&bar.full[st], KB * kBox + kQBytes + (unit ? 0 : VB * kBox) + kMats + (uint32_t)sizeof(DrRows));
          for (int b = 0; b < KB; ++b) tma_load_3d(base + L::kK + b * kBox, &args.k, &bar.full[st], 64 * b, hk, row);
          if (!unit)
            for (int b = 0; b < VB; ++b) tma_load_3d(base + L::kV + b * kBox, &args.v, &bar.full[st], 64 * b, h, row);
          pipe::bulk_load(base + L::kRows, p.rows + at, sizeof(DrRows), &bar.full[st]);
          pipe::bulk_load(base + L::kN, tiles, kMats, &bar.full[st]);  // N's terms, P's behind them
          if (kQBytes)
            for (int b = 0; b < KB; ++b) tma_load_3d(base + L::kQ + b * kBox, &args.q, &bar.full[st], 64 * b, hk, row);
        }
        // every load issued has landed before the CTA releases its shared memory
#pragma unroll 1
        for (int x = i > kStages ? i - kStages : 0; x < i; ++x) mbar_wait_drain(&bar.full[x % kStages], parity(x / kStages));
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t el = elect_one();
      const uint64_t dK = desc_sw128(s0 + L::kK, 16, 1024), dQ = desc_sw128(s0 + L::kQ, 16, 1024);   // K-major
      const uint64_t dKn = desc_sw128(s0 + L::kK, kBox, 1024), dQn = desc_sw128(s0 + L::kQ, kBox, 1024);  // MN-major
      const uint64_t dV = desc_sw128(s0 + L::kV, kBox, 1024), dN = desc_sw128(s0 + L::kN, 16, 1024),
                     dP = desc_sw128(s0 + L::kP, 16, 1024);
      constexpr uint32_t iKK = idesc_bf16(128, 64, false, false), iKM = idesc_bf16(128, 64, false, true),
                         iMM = idesc_bf16(128, 64, true, true), iW = idesc_bf16(128, 64 * KB, false, true);
      constexpr uint64_t kB = kBox / 16;
      constexpr uint64_t kStepN = kRev ? pipe::kStepMN : pipe::kStepK;  // N transposed in reverse
      constexpr uint32_t iN = kRev ? iKM : iKK;
      auto at = [&](int i) { return (uint64_t)(stage(i) / 16); };
      auto dO_part = [&](int i) {  // P^T dO of chunk i
        wait_full(i);
        if (i > 0) wait_on(bar.o_free, parity(i - 1), wait);
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t)
          pipe::umma_k_el<4>(el, tmem + kTmO, dV + at(i), dP + at(i) + t * kB, pipe::kStepMN, pipe::kStepMN, iMM, t > 0);
        umma_commit_el(el, bar.o_full);
      };
      if (kRev && nc > 0) dO_part(0);
#pragma unroll 1
      for (int i = 0; i < nc; ++i) {
        wait_full(i);
        wait_on(bar.s_ready, parity(i), wait);
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int b = 0; b < KB; ++b)
            pipe::umma_ts_k_el<4>(el, tmem + kTmX, tmem + kTmS + 64 * t + 32 * b, dK + at(i) + b * kB, 8, pipe::kStepK, iKK,
                                  t + b > 0);
        umma_commit_el(el, bar.x_full);
        if (MODE == kOut) {
          if (i > 0) {
            wait_on(bar.o_free, parity(i - 1), wait);
            tc_fence_after();
          }
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int b = 0; b < KB; ++b)
              pipe::umma_ts_k_el<4>(el, tmem + kTmO, tmem + kTmS + 64 * t + 32 * b, dQ + at(i) + b * kB, 8, pipe::kStepK, iKK,
                                    t + b > 0);
          umma_commit_el(el, bar.q_full);
        }
        if (kRev) {
          wait_on(bar.q_ready, parity(i), wait);
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t)
            pipe::umma_ts_k_el<4>(el, tmem + kTmW, tmem + kTmD + 32 * t, dQn + at(i), 8, pipe::kStepMN, iW, t > 0);
          umma_commit_el(el, bar.q_full);
        }
        wait_on(bar.y_ready, parity(i), wait);
        tc_fence_after();
        pipe::umma_ts_k_el<4>(el, tmem + kTmX, tmem + kTmY, dN + at(i), 8, kStepN, iN, false);
        pipe::umma_ts_k_el<4>(el, tmem + kTmX, tmem + kTmY + 32, dN + at(i), 8, kStepN, iN, true);
        pipe::umma_ts_k_el<4>(el, tmem + kTmX, tmem + kTmY, dN + at(i) + kB, 8, kStepN, iN, true);
        umma_commit_el(el, bar.n_full);
        wait_on(bar.d_ready, parity(i), wait);
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t)
          pipe::umma_ts_k_el<4>(el, tmem + kTmW, tmem + kTmY + 32 * t, dKn + at(i), 8, pipe::kStepMN, iW, kRev || t > 0);
        umma_commit_el(el, bar.w_full);
        if (MODE == kOut) {
          wait_on(bar.q_ready, parity(i), wait);
          wait_on(bar.e_ready, parity(i), wait);
          tc_fence_after();
          pipe::umma_ts_k_el<4>(el, tmem + kTmO, tmem + kTmD, dP + at(i), 8, pipe::kStepK, iKK, true);
          pipe::umma_ts_k_el<4>(el, tmem + kTmO, tmem + kTmD + 32, dP + at(i), 8, pipe::kStepK, iKK, true);
          pipe::umma_ts_k_el<4>(el, tmem + kTmO, tmem + kTmD, dP + at(i) + kB, 8, pipe::kStepK, iKK, true);
          umma_commit_el(el, bar.o_full);
        }
        umma_commit_el(el, &bar.free[i % kStages]);
        if (kRev && i + 1 < nc) dO_part(i + 1);
      }
      // every MMA and every arrival of a commit has landed before the CTA ends
      umma_commit_el(el, bar.drain);
      mbar_wait_drain(bar.drain, 0);
#pragma unroll 1
      for (int x = nc > kStages ? nc - kStages : 0; x < nc; ++x) mbar_wait_drain(&bar.free[x % kStages], parity(x / kStages));
      if (nc > 0) {
        mbar_wait_drain(bar.x_full, parity(nc - 1));
        mbar_wait_drain(bar.n_full, parity(nc - 1));
        mbar_wait_drain(bar.w_full, parity(nc - 1));
        if (MODE == kOut || kRev) {
          mbar_wait_drain(bar.q_full, parity(nc - 1));
          mbar_wait_drain(bar.o_full, parity(nc - 1));
        }
      }
    } else if (partial) {
      // ------------------------------------------------------------ rows past the end
      const int t = threadIdx.x - 64;
      constexpr int kBoxes = 2 * KB + VB;  // K, Q and V follow each other
#pragma unroll 1
      for (int i = 0; i < nc; ++i) {
        wait_on(&bar.full[i % kStages], parity(i / kStages), wait);
        if (i == tail) {
          const int nv = live(i);
          for (int e = t; e < (kDrC - nv) * 8 * kBoxes; e += 64) {
            const int y = e % (8 * kBoxes), r = nv + e / (8 * kBoxes);
            pipe::sts_u4(s0 + stage(i) + L::kK + (uint32_t)(y >> 3) * kBox + sw128_offset(r, 8 * (y & 7)), make_uint4(0, 0, 0, 0));
          }
          fence_async_smem();
          pipe::warp_arrive(bar.patched);
        }
        pipe::warp_arrive(&bar.free[i % kStages]);
      }
    }
  } else if (warp < kStateWarp0) {
    // ------------------------------------------------------------ Y and E
    if (kElemRegs > 80) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kElemRegs));
    const int quad = warp & 3, sub = (warp - kElemWarp0) >> 2;
    if (quad < 2 * VB) {
      const int tok = 32 * sub + 2 * (lane & 3);  // this lane's tokens: tok + 8 m and the next
      // addresses of the transposing loads of V: 16 tokens and 16 lanes (columns of v) at a time
      const uint32_t lr = (lane & 7) + 8 * (lane >> 4), lc = 4 * (quad & 1) + ((lane >> 3) & 1);
      const uint32_t v_at = L::kV + (uint32_t)(quad >> 1) * kBox + (32 * sub + lr) * 128;
      // and of the stores of E: row i, columns of v
      const int fi = 8 * (lane >> 4) + (lane & 7), fc = 32 * quad + 8 * ((lane >> 3) & 1);
      const uint32_t so = s0 + L::kO;
      const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
      constexpr int kTeam = 128 * VB;
      const int tt = 64 * VB * sub + 32 * quad + lane;
#pragma unroll 1
      for (int i = 0; i < nc; ++i) {
        wait_full(i);
        const uint32_t rows = rows_of(i);
        auto factors = [&](uint32_t which, uint64_t(&f)[4]) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
            asm volatile("ld.shared.b64 %0, [%1];" : "=l"(f[m]) : "r"(rows + which + (tok + 8 * m) * 4));
        };
        constexpr uint64_t kMinus = 0x8000000080000000ull, kMinusOne = 0xbf800000bf800000ull;  // signs; -1, -1
        constexpr uint32_t kIn = offsetof(DrRows, kin), kOutF = offsetof(DrRows, kout), kBeta = offsetof(DrRows, beta);
        uint64_t y[2][8], f[4], beta[4];  // pairs of tokens
        factors(kRev ? kOutF : kIn, f);
        if (!kRev) {
#pragma unroll
          for (int m = 0; m < 4; ++m) f[m] ^= kMinus;
        }
        factors(kBeta, beta);
        if (!kRev) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t w[8];
            const uint32_t at = s0 + stage(i) + v_at + (((lc + 2 * q) ^ (lane & 7)) * 16);
            ldmatrix4_trans(at, w[0], w[1], w[2], w[3]);
            ldmatrix4_trans(at + 16 * 128, w[4], w[5], w[6], w[7]);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[q][e] = unit ? 0 : pk2(lo_f(w[e]), hi_f(w[e]));
          }
        }
        wait_on(bar.x_full, parity(i), wait);
        if (kRev) wait_on(bar.o_full, parity(i), wait);
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t at = lanes + ((uint32_t)(16 * q) << 16);
          uint32_t x[16];
          tmem_ld_16x256_x4_async(at + kTmX + 32 * sub, x);
          if (kRev) {
            uint32_t g[16];
            tmem_ld_16x256_x4_async(at + kTmO + 32 * sub, g);
            tmem_wait_ld16(g);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[q][e] = pk2(__uint_as_float(g[2 * e]), __uint_as_float(g[2 * e + 1]));
          }
          tmem_wait_ld16(x);
          uint32_t t0[8], t1[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[q][e] = fma2(f[e >> 1], pk2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), y[q][e]);
            split2(mul2(beta[e >> 1], y[q][e]), t0[e], t1[e]);
          }
          tmem_st_16x128_async(at + kTmY + 16 * sub, t0);
          tmem_st_16x128_async(at + kTmY + 32 + 16 * sub, t1);
        }
        tmem_wait_st();
        tc_fence_before();
        if (kRev) pipe::warp_arrive(bar.o_free);
        pipe::warp_arrive(bar.y_ready);
        factors(kRev ? kIn : kOutF, f);
        if (kRev) {
#pragma unroll
          for (int m = 0; m < 4; ++m) f[m] ^= kMinus;
        }
        if (kKeeps) {  // the chunk before has been read out of the staging tile
          if (tt == 0) bulk_wait_read0();
          role_sync<2, kTeam>();
        }
        wait_on(bar.n_full, parity(i), wait);
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t at = lanes + ((uint32_t)(16 * q) << 16);
          uint32_t x[16];
          tmem_ld_16x256_x4_async(at + kTmX + 32 * sub, x);
          tmem_wait_ld16(x);
          uint32_t t0[8], t1[8], t2[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[q][e] = fma2(pk2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), kMinusOne, y[q][e]);
            float v0, v1;
            upk2(y[q][e], v0, v1);
            if (kKeeps) t2[e] = tc::pack_bf16x2(v0, v1);
            split2(mul2(f[e >> 1], mul2(beta[e >> 1], y[q][e])), t0[e], t1[e]);
          }
          tmem_st_16x128_async(at + kTmY + 16 * sub, t0);
          tmem_st_16x128_async(at + kTmY + 32 + 16 * sub, t1);
          if (kKeeps) {  // E or Z, rows of tokens, into the staging tile
            const int c = fc + 16 * q;
            const uint32_t to = so + (uint32_t)(c >> 6) * kBox + sw128_offset(32 * sub + fi, c & 63);
            stmatrix4_trans(to, t2[0], t2[1], t2[2], t2[3]);
            stmatrix4_trans(to + 16 * 128, t2[4], t2[5], t2[6], t2[7]);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        pipe::warp_arrive(bar.d_ready);
        if (MODE == kOut) {  // beside W
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t at = lanes + ((uint32_t)(16 * q) << 16);
            uint32_t t0[8], t1[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) split2(mul2(beta[e >> 1], y[q][e]), t0[e], t1[e]);
            tmem_st_16x128_async(at + kTmD + 16 * sub, t0);
            tmem_st_16x128_async(at + kTmD + 32 + 16 * sub, t1);
          }
          tmem_wait_st();
          tc_fence_before();
          pipe::warp_arrive(bar.e_ready);
        }
        pipe::warp_arrive(&bar.free[i % kStages]);
        if (kKeeps) {
          fence_async_smem();
          role_sync<2, kTeam>();
          const int nv = live(i);
          const long long row0 = a + (long long)chunk(i) * kDrC;
          if (nv < kDrC) {  // rows past the end belong to another sequence: row by row
            bf16 *out = args.out + row0 * args.os + (size_t)h * p.dv;
            for (int e = tt; e < nv * 8 * VB; e += kTeam) {
              const int r = e / (8 * VB), c = 8 * (e % (8 * VB));
              if (c < p.dv) *reinterpret_cast<uint4 *>(out + r * args.os + c) = pipe::lds_sw128(so + (uint32_t)(c >> 6) * kBox, r, (c & 63) / 8);
            }
          } else if (tt == 0) {
            for (int b = 0; b < VB; ++b)
              if (64 * b < p.dv) tma_store_3d(&args.o, so + b * kBox, 64 * b, h, (int)row0);
            bulk_commit();
          }
        }
      }
      if (kKeeps && tt == 0) bulk_wait0();
    }
  } else if (warp < kOutWarp0) {
    // ------------------------------------------------------------ state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
    const int quad = warp & 3, sub = (warp - kStateWarp0) >> 2;
    if (quad < 2 * VB) {
      constexpr int kCols = 32 * KB;  // state rows (dk) of a thread
      const int c = 32 * quad + lane, a0 = sub * kCols;
      const size_t dd = (size_t)p.dk * dv, item = (size_t)place * p.H + h;
      uint64_t S[kCols / 2];  // pairs along dk
      {
        const float *in = args.first ? args.first + item * dd + c : nullptr;
        const bool col = in && c < dv;
#pragma unroll
        for (int x = 0; x < kCols; x += 2) {  // dk is even
          const bool row = col && a0 + x < p.dk;
          float v0 = row ? in[(size_t)(a0 + x) * dv] : 0.f, v1 = row ? in[(size_t)(a0 + x + 1) * dv] : 0.f;
          if (unit) v0 = a0 + x == c ? 1.f : 0.f, v1 = a0 + x + 1 == c ? 1.f : 0.f;
          S[x / 2] = pk2(v0, v1);
        }
      }
      // the thread's 8 x 16 bytes of a kept state, 64 VB apart
      constexpr size_t kTile = 64 * KB * 64 * VB;
      const size_t mine = ((size_t)(a0 / 8) * (64 * VB) + c) * 8;
      constexpr int kTeam = 128 * VB;
      auto pack = [](uint64_t v) {
        float x, y;
        upk2(v, x, y);
        return tc::pack_bf16x2(x, y);
      };
      auto keep = [&](size_t at) {  // rounded as the operand's first term is
        if (sub + quad == 0 && lane == 0) bulk_wait_read0();
        role_sync<4, kTeam>();
#pragma unroll
        for (int x = 0; x < kCols; x += 8)
          pipe::sts_u4(s0 + L::kKept + 2 * (uint32_t)mine + (x / 8) * (64 * VB) * 16,
                       make_uint4(pack(S[x / 2]), pack(S[x / 2 + 1]), pack(S[x / 2 + 2]), pack(S[x / 2 + 3])));
        fence_async_smem();
        role_sync<4, kTeam>();
        if (sub + quad == 0 && lane == 0) {
          pipe::bulk_store(args.kept + at * kTile, s0 + L::kKept, (uint32_t)kTile * 2);
          bulk_commit();
        }
      };
#pragma unroll 1
      for (int i = 0; i < nc; ++i) {
        // the state's terms as A operands: lane = column of v, bf16 pairs along dk
#pragma unroll
        for (int x = 0; x < kCols; x += 16) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split2(S[x / 2 + e], hi[e], lo[e]);
          tmem_st8_async(pipe::tmem_quad(tmem + kTmS, (a0 + x) / 2), hi);
          tmem_st8_async(pipe::tmem_quad(tmem + kTmS + 64, (a0 + x) / 2), lo);
        }
        tmem_wait_st();
        tc_fence_before();
        pipe::warp_arrive(bar.s_ready);
        if (kKeeps) keep((size_t)(slot0 + chunk(i)) * p.H + h);  // beside the chunk's products
        wait_full(i);
        const float ah = pipe::lds_f(rows_of(i) + offsetof(DrRows, all_hi)), al = pipe::lds_f(rows_of(i) + offsetof(DrRows, all_lo));
        const uint64_t all_hi = pk2(ah, ah), all_lo = pk2(al, al);
        pipe::warp_arrive(&bar.free[i % kStages]);
        wait_on(bar.w_full, parity(i), wait);
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < kCols; x += 16) {
          float w[16];
          tmem_ld16(pipe::tmem_quad(tmem + kTmW, a0 + x), w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint64_t &s = S[x / 2 + e];
            s = fma2(s, all_hi, fma2(s, all_lo, pk2(w[2 * e], w[2 * e + 1])));
          }
        }
        tc_fence_before();
      }
      if (kKeeps && sub + quad == 0 && lane == 0) bulk_wait0();
      // the user's final state, or the segment's sum; M's places are behind those of all N
      float *to = args.seg && ends ? args.fin ? args.fin + ((size_t)seq * p.H + h) * dd : nullptr
                  : args.last      ? args.last + (unit ? (size_t)args.places * p.H * p.dk * p.dv : 0) + item * dd
                                   : nullptr;
      if (to && unit && c < dv) {  // M transposed, as the scan reads it
#pragma unroll
        for (int x = 0; x < kCols; x += 2)
          if (a0 + x < p.dk) *reinterpret_cast<uint64_t *>(to + (size_t)c * p.dk + a0 + x) = S[x / 2];
      } else if (to && c < dv) {
#pragma unroll
        for (int x = 0; x < kCols; x += 2) {
          float v0, v1;
          upk2(S[x / 2], v0, v1);
          if (a0 + x < p.dk) {
            to[(size_t)(a0 + x) * dv + c] = v0;
            to[(size_t)(a0 + x + 1) * dv + c] = v1;
          }
        }
      }
    }
  } else if (kIdle) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLastRegs));
  } else if (MODE == kOut) {
    // ------------------------------------------------------------ outputs
    const int quad = warp & 3, tt = threadIdx.x - 32 * kOutWarp0;
    if (quad < 2 * VB) {
      constexpr int kTeam = 64 * VB;
      const int fi = 8 * (lane >> 4) + (lane & 7), fc = 32 * quad + 8 * ((lane >> 3) & 1);
      const uint32_t so = s0 + L::kO, lanes = tmem + ((uint32_t)(32 * quad) << 16);
#pragma unroll 1
      for (int i = 0; i < nc; ++i) {
        wait_full(i);
        wait_on(bar.q_full, parity(i), wait);
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < kDrC; j += 32) {  // S^T q by e^G scale / |q|, in place
          float x[32];
          tmem_ld32(lanes + kTmO + j, x);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 f = pipe::lds_f4(rows_of(i) + offsetof(DrRows, qin) + (j + e) * 4);
            x[e] *= f.x, x[e + 1] *= f.y, x[e + 2] *= f.z, x[e + 3] *= f.w;
          }
          tmem_st32(lanes + kTmO + j, x);
        }
        tc_fence_before();
        pipe::warp_arrive(bar.q_ready);
        pipe::warp_arrive(&bar.free[i % kStages]);
        if (tt == 0) bulk_wait_read0();
        role_sync<3, kTeam>();
        wait_on(bar.o_full, parity(i), wait);
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t x[32];
          tmem_ld_16x256_async(lanes + ((uint32_t)(16 * q) << 16) + kTmO, x);
          tmem_wait_ld32(x);
          const int c = fc + 16 * q;
          const uint32_t to = so + (uint32_t)(c >> 6) * kBox + sw128_offset(fi, c & 63);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            uint32_t f[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              f[y] = tc::pack_bf16x2(__uint_as_float(x[4 * e + 2 * y]), __uint_as_float(x[4 * e + 2 * y + 1]));
            stmatrix4_trans(to + e * 1024, f[0], f[1], f[2], f[3]);
          }
        }
        tc_fence_before();
        pipe::warp_arrive(bar.o_free);
        fence_async_smem();
        role_sync<3, kTeam>();
        const int nv = live(i);
        const long long row0 = a + (long long)chunk(i) * kDrC;
        if (nv < kDrC) {
          bf16 *out = args.out + row0 * args.os + (size_t)h * p.dv;
          for (int e = tt; e < nv * 8 * VB; e += kTeam) {
            const int r = e / (8 * VB), c = 8 * (e % (8 * VB));
            if (c < p.dv) *reinterpret_cast<uint4 *>(out + r * args.os + c) = pipe::lds_sw128(so + (uint32_t)(c >> 6) * kBox, r, (c & 63) / 8);
          }
        } else if (tt == 0) {
          for (int b = 0; b < VB; ++b)
            if (64 * b < p.dv) tma_store_3d(&args.o, so + b * kBox, 64 * b, h, (int)row0);
          bulk_commit();
        }
      }
      if (tt == 0) bulk_wait0();
    }
  } else if (kRev) {
    // ------------------------------------------------------------ the terms of (qin dO)^T
    const int quad = warp & 3;
    if (quad < 2 * VB) {
      const uint32_t lr = (lane & 7) + 8 * (lane >> 4), lc = 4 * (quad & 1) + ((lane >> 3) & 1);
      const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
#pragma unroll 1
      for (int i = 0; i < nc; ++i) {
        wait_full(i);
        if (i > 0) {
          wait_on(bar.q_full, parity(i - 1), wait);
          tc_fence_after();
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float2 f[4];
#pragma unroll
          for (int m = 0; m < 4; ++m)
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                         : "=f"(f[m].x), "=f"(f[m].y)
                         : "r"(rows_of(i) + (uint32_t)offsetof(DrRows, qin) + (32 * half + 2 * (lane & 3) + 8 * m) * 4));
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t w[8], t0[8], t1[8];
            const uint32_t at = s0 + stage(i) + L::kV + (uint32_t)(quad >> 1) * kBox + (32 * half + lr) * 128 +
                                (((lc + 2 * q) ^ (lane & 7)) * 16);
            ldmatrix4_trans(at, w[0], w[1], w[2], w[3]);
            ldmatrix4_trans(at + 16 * 128, w[4], w[5], w[6], w[7]);
#pragma unroll
            for (int e = 0; e < 8; ++e) tc::split2(f[e >> 1].x * lo_f(w[e]), f[e >> 1].y * hi_f(w[e]), t0[e], t1[e]);
            const uint32_t to = lanes + ((uint32_t)(16 * q) << 16) + kTmD + 16 * half;
            tmem_st_16x128_async(to, t0);
            tmem_st_16x128_async(to + 32, t1);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        pipe::warp_arrive(bar.q_ready);
        pipe::warp_arrive(&bar.free[i % kStages]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

template <int KB, int VB, int MODE> void run(Args &args, cudaStream_t s) {
  using L = Layout<KB, VB, MODE>;
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(dr_tc_kernel<KB, VB, MODE>), L::kBytes, allowed);
  const int places = args.seg ? args.places : args.p.nseq;
  dr_tc_kernel<KB, VB, MODE><<<dim3((unsigned)(places * args.p.H), MODE == kSum && args.what == 2 ? 2 : 1), kThreads, L::kBytes, s>>>(args);
}
template <int MODE> void run_boxes(Args &args, int kb, int vb, cudaStream_t s) {
  if (kb == 1)
    vb == 1 ? run<1, 1, MODE>(args, s) : run<1, 2, MODE>(args, s);
  else
    vb == 1 ? run<2, 1, MODE>(args, s) : run<2, 2, MODE>(args, s);
}
template <int MODE> void run_boxes(Args &args, cudaStream_t s) {
  run_boxes<MODE>(args, la_tc_boxes(args.p.dk), la_tc_boxes(args.p.dv), s);
}

// the tensor maps that every chain has; v: its values or dO, with v's heads
bool fill_args(Args &args, const DrProblem &p, const void *v, long long vs, void *out, long long os) {
  args.p = p;
  args.out = static_cast<bf16 *>(out);
  args.os = os;
  args.wait = {p.status, p.wait_ns};
  args.seg = args.places = args.what = 0;
  args.fin = nullptr;
  if (!encode_tmap_bf16_heads(&args.q, p.q, p.dk, p.Hk, p.total, p.qs * 2, kDrC) ||
      !encode_tmap_bf16_heads(&args.k, p.k, p.dk, p.Hk, p.total, p.ks * 2, kDrC) ||
      !encode_tmap_bf16_heads(&args.v, v, p.dv, p.H, p.total, vs * 2, kDrC) ||
      !encode_tmap_bf16_heads(&args.o, out, p.dv, p.H, p.total, os * 2, kDrC)) {
    note_host_error();
    return false;
  }
  return true;
}

}  // namespace

void launch_dr_tc_chain(const DrProblem &p, void *o, long long os, float *fin, cudaStream_t s) {
  Args args;
  const long long es = (long long)p.H * p.dv;
  if (!fill_args(args, p, p.v, p.vs, o ? o : p.E, o ? os : es)) return;
  args.first = p.init;
  args.last = o ? fin : nullptr;
  args.kept = reinterpret_cast<bf16 *>(p.S);
  if (p.seg) {
    args.seg = p.seg;
    args.places = p.seg_places;
    args.first = p.seg_states;
    args.last = nullptr;
    args.fin = o ? fin : nullptr;
  }
  o ? run_boxes<kOut>(args, s) : run_boxes<kStates>(args, s);
}

void launch_dr_tc_sums(const DrProblem &p, cudaStream_t s) {
  Args args;
  if (!fill_args(args, p, p.v, p.vs, p.E, (long long)p.H * p.dv)) return;
  args.seg = p.seg;
  args.places = p.seg_places;
  args.first = nullptr;
  args.last = p.seg_sums;
  const int kb = la_tc_boxes(p.dk), vb = la_tc_boxes(p.dv);
  args.what = kb == vb ? 2 : 0;
  run_boxes<kSum>(args, kb, vb, s);
  if (kb != vb) {
    args.what = 1;
    run_boxes<kSum>(args, kb, kb, s);
  }
}

namespace {

// Segments' states before their first tokens: S_next = M S + N, from the initial state on.  A block has 16 columns of a
// state, a thread 8 of them in one row: the warps read M, which is transposed, row by row, and the columns are in
// shared memory.
constexpr int kScanCols = 16;
__global__ void __launch_bounds__(256) dr_scan_kernel(DrProblem p, float *fin) {
  extern __shared__ __align__(128) uint8_t smem[];  // two M
  __shared__ __align__(16) float S[128][kScanCols];
  __shared__ uint64_t full[2];
  const int seq = blockIdx.x / p.H, h = blockIdx.x - seq * p.H, c0 = blockIdx.y * kScanCols, dk = p.dk, dv = p.dv;
  const int row = threadIdx.x & 127, half = 8 * (threadIdx.x >> 7), c = c0 + half;
  const size_t dd = (size_t)dk * dv, all = (size_t)p.seg_places * p.H;
  int a, len, slot0;
  dr_seq(p, seq, a, len, slot0);
  const int n = p.seg * kDrC, place0 = dr_place0(p, p.seg, a, seq), segments = (len + n - 1) / n;
  const bool live = row < dk && c < dv;  // dv is a multiple of 8
  float4 x[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  auto get = [&](const float *from) {
    x[0] = reinterpret_cast<const float4 *>(from)[0], x[1] = reinterpret_cast<const float4 *>(from)[1];
  };
  auto put = [&](float *to) { reinterpret_cast<float4 *>(to)[0] = x[0], reinterpret_cast<float4 *>(to)[1] = x[1]; };
  const uint32_t bytes = (uint32_t)(dk * dk * 4);
  auto fetch = [&](int g) {  // thread 0
    sm100::mbar_expect_tx(&full[g & 1], bytes);
    pipe::bulk_load(smem + (g & 1) * bytes, p.seg_sums + all * dd + ((size_t)(place0 + g) * p.H + h) * ((size_t)dk * dk), bytes, &full[g & 1]);
  };
  if (threadIdx.x == 0) {
    sm100::mbar_init(&full[0], 1);
    sm100::mbar_init(&full[1], 1);
    sm100::fence_mbar_init();
    if (segments > 1) fetch(0);
  }
  __syncthreads();
  if (live && p.init) get(p.init + ((size_t)seq * p.H + h) * dd + (size_t)row * dv + c);
  if (len == 0 && fin && live) put(fin + ((size_t)seq * p.H + h) * dd + (size_t)row * dv + c);
  for (int g = 0; g < segments; ++g) {
    const size_t item = (size_t)(place0 + g) * p.H + h;
    if (live) put(p.seg_states + item * dd + (size_t)row * dv + c);
    if (g + 1 == segments) break;
    __syncthreads();  // the columns and the other M are read
    put(&S[row][half]);
    if (threadIdx.x == 0 && g + 2 < segments) fetch(g + 1);
    __syncthreads();
    sm100::mbar_wait_drain(&full[g & 1], (g >> 1) & 1);
    if (live) {
      const float *M = reinterpret_cast<const float *>(smem + (g & 1) * bytes) + row;
      get(p.seg_sums + item * dd + (size_t)row * dv + c);
#pragma unroll 8
      for (int k = 0; k < dk; ++k) {
        const float f = M[k * dk];
        const float4 s0 = *reinterpret_cast<const float4 *>(&S[k][half]), s1 = *reinterpret_cast<const float4 *>(&S[k][half + 4]);
        x[0].x = fmaf(f, s0.x, x[0].x), x[0].y = fmaf(f, s0.y, x[0].y), x[0].z = fmaf(f, s0.z, x[0].z), x[0].w = fmaf(f, s0.w, x[0].w);
        x[1].x = fmaf(f, s1.x, x[1].x), x[1].y = fmaf(f, s1.y, x[1].y), x[1].z = fmaf(f, s1.z, x[1].z), x[1].w = fmaf(f, s1.w, x[1].w);
      }
    }
  }
}

}  // namespace

void launch_dr_tc_scan(const DrProblem &p, float *fin, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(dr_scan_kernel), 2 * 128 * 128 * 4, allowed);
  dr_scan_kernel<<<dim3((unsigned)(p.nseq * p.H), (unsigned)((p.dv + kScanCols - 1) / kScanCols)), 256, 2 * p.dk * p.dk * 4, s>>>(p, fin);
}

void launch_dr_tc_reverse(const DrProblem &p, const void *dout, long long dos, const float *dfin, float *dinit, cudaStream_t s) {
  Args args;
  if (!fill_args(args, p, dout, dos, p.Z, (long long)p.H * p.dv)) return;
  args.first = dfin;
  args.last = dinit;
  args.kept = reinterpret_cast<bf16 *>(p.dS);
  run_boxes<kReverse>(args, s);
}

}  // namespace ssd
