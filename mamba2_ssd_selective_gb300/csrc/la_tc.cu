// Linear attention with a decay for each head on the 5th-generation tensor cores
// (tcgen05, accumulators and A operands in TMEM): bf16 tensors, widths up to 128.
//
// Persistent CTAs, one on an SM, take items (a segment of one sequence, one pass of
// the call, one query head) from a counter and walk each in blocks of 64 tokens.
// With P_ij = p_scale q_i . k_j lam^|i - j| inside the block (j <= i; reverse: j >= i) and
// the incoming state S (dk x dv):
//     o_i  = lam^a(i) (S^T q_i + V^T P'_i),    P'_ij = P_ij lam^-a(i)
//     S^T  = lam^nv S^T + W^T,    W^T = (V^T diag(lam^b)) K
// Everything is formed transposed, so that dv (up to 128) fills the accumulators'
// lanes, the state stays in its warps' registers (lane = dv) from block to
// block, and the products with the state take their A operands from TMEM: S^T
// from the registers, the weighted copies of V^T from shared memory through
// transposing matrix loads, so that shared memory carries the inputs, P and the outputs only.  (With
// the weighted K as a B operand in shared memory, three terms written and read back, a call of 128 items
// of 8192 tokens at widths of 128 took 325 us; as it is, 176.)
// P and S are rounded to bf16 as operands (the outputs are bf16 too); what goes
// into the state is not: V diag(lam^b) is split into three bf16 terms (24 bits), so
// that states keep fp32 precision over any length.
//
// Warps:
//   0, 1    P: scores out of TMEM (lane = row i of the block), decay and mask, P into shared memory
//   2       TMA producer: Q, K, V blocks [64 x 64 columns each], a ring of stages
//   3       TMEM owner and MMA issuer
//   4-7     outputs: O^T out of TMEM as fragments, weighed, transposed by stmatrix, stored by TMA
//   8-15    state: S = lam^nv S + W, and S^T into TMEM as the next block's operand
//   16-19   the three terms of V^T diag(lam^b) into TMEM
// The tensor core's order is scores of block i + 1, W of block i (by halves of 32 tokens,
// whose operands alternate between two buffers), outputs of block i.  So the chain
// from state to state is W's products and W's read, and the state's update and
// its way into TMEM run beside the next block's scores and W.
// P' weighs a score with a power that depends on its column alone, lam^-(j + 1) (reverse:
// lam^-(nv - 1 - j)), so that both products meet in one accumulator, which takes
// turns between two.  It is up to lam^-64: heads whose lam^64 is below 2^-40 form
// P and O beside Oi instead, and add lam^a Oi at the end.
// What bounds it: with an item on every SM, HBM (144 items of 8192 tokens at widths of 128: 190 us, 6.3 TB/s of a
// copy's 6.8).  An item by itself is bounded by its chain of blocks, 1.3 us a block of 64 tokens at widths of 128
// (1.2 us at 64, where half of the lanes have nothing to do): the tensor core's 1600 cycles (of them 770 for the
// three terms of W), the roles' hand-offs, and instructions that are not in the caches (1.2 of 9 cycles that a
// warp waits for each of its instructions).
// Segments of a cut sequence either start from states that a scan has joined before
// (few sequences: the segments run side by side), or hand their state on: the
// next segment's state warps wait for its flag, and as items are taken level by
// level, whatever an item waits for was taken before it.
// The last block of a sequence is masked: rows past its end belong to another
// sequence, so K's and V's are replaced by zeros in shared memory (0 * NaN would be
// NaN), scores with them are cut off, and nothing is stored there.
#include <type_traits>

#include "retention.h"
#include "tc_pipe.cuh"
#include "tc_util.cuh"

namespace ssd {

namespace {

using bf16 = __nv_bfloat16;
using namespace sm100;
using pipe::parity;

constexpr int kC = 64;  // tokens of a block
constexpr int kThreads = 640;
constexpr int kOutWarp0 = 4, kStateWarp0 = 8, kWeighWarp0 = 16;
constexpr uint32_t kBox = 8192;  // [64 tokens x 64 columns] bf16

// TMEM columns: scores, two accumulators of outputs (or O and Oi), W, S^T (bf16), two buffers of the three terms of half a block
constexpr uint32_t kTmQK = 0, kTmO = 64, kTmOi = 128, kTmW = 192, kTmS = 320, kTmT = 384, kTmCols = 512;
constexpr uint32_t kTmW1 = 0;  // summaries, which need nothing else: W's second buffer
constexpr uint32_t kTerm = 16, kHalf = 3 * kTerm;  // a term of half a block (32 tokens as bf16 pairs)

// Weights of a block's rows, each filled by the role that reads it.
struct Tables {
  float st[kC];   // weighted V: state scale lam^b(row)
  float out[kC];  // outputs: output scale lam^a(row)
  float p[kC];    // P: product scale lam^-a of the column, or (heads that stand apart) both scales lam^distance
};

template <int KB, int VB, bool SUMMARY, bool F32>
struct Layout {
  static constexpr int kStages = KB + VB == 2 ? 6 : KB + VB == 4 && F32 ? 3 : 4;
  static constexpr uint32_t kQ = 0, kK = SUMMARY ? 0 : KB * kBox, kV = kK + KB * kBox, kStage = kV + VB * kBox;
  static constexpr uint32_t kP = kStages * kStage;                  // two P buffers
  static constexpr uint32_t kO = kP + (SUMMARY ? 0 : 2 * kBox);     // a block's outputs, on their way to TMA
  static constexpr uint32_t kTab = kO + (SUMMARY ? 0 : (F32 ? 2 : 1) * VB * kBox);  // weights, see Tables
  static constexpr uint32_t kBar = kTab + sizeof(Tables);
  static constexpr int kNumBars = 2 * kStages + 2 + 4 + 2 + 2 + 4 + 2 + 4 + 4 + 1;
  static constexpr uint32_t kEnd = kBar + kNumBars * 8 + 16 + 2 * 48;  // and the TMEM address, two item numbers, two items
  static constexpr int kBytes = (int)kEnd + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};

template <int ST>
struct Bars {
  uint64_t *full, *free;        // [ST] stage loaded / its operands read
  uint64_t *qk_full, *qk_free;  // scores
  uint64_t *p_ready, *p_free;   // [2]
  uint64_t *s_ready, *s_free;   // S^T of the block in TMEM / read by its product
  uint64_t *v_ready, *v_free;   // [2] half a block's terms in TMEM / read by its MMAs
  uint64_t *w_full, *w_free;    // [2] W formed / read out of TMEM (summaries: two buffers, else one)
  uint64_t *o_full, *o_free;    // [2]
  pipe::UnitRing items;
  uint64_t *drain;
  __device__ explicit Bars(uint64_t *b, int *slot) {
    full = b;
    free = full + ST;
    qk_full = free + ST;
    qk_free = qk_full + 1;
    p_ready = qk_free + 1;
    p_free = p_ready + 2;
    s_ready = p_free + 2;
    s_free = s_ready + 1;
    w_free = s_free + 1;
    v_ready = w_free + 2;
    v_free = v_ready + 2;
    w_full = v_free + 2;
    o_full = w_full + 2;
    o_free = o_full + 2;
    items.full = o_free + 2;
    items.free = items.full + 2;
    items.slot = slot;
    drain = items.free + 2;
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
  a = __byte_perm(__float_as_uint(f0), __float_as_uint(f1), 0x7632);
  f0 = tc::minus_lo(f0, a);
  f1 = tc::minus_hi(f1, a);
  b = __byte_perm(__float_as_uint(f0), __float_as_uint(f1), 0x7632);
  c = tc::pack_bf16x2(tc::minus_lo(f0, b), tc::minus_hi(f1, b));
}

// The roles' loops together are more than the instruction caches hold at once, and code
// that all of them hold in line is what made them so: items are worked out by the producer alone, weights are
// filled at one place of a role, blocks of the usual kind have code of their own without the branches of the
// others.  32 heads of 4 sequences of 8192 tokens, widths of 128: 263 us with each role working out its
// items, 202 us with the producer, 181 us with one fill, 190 us without the split of the usual blocks.
// A hand-off wait as mbar_wait, kept short for the same reason: the usual case (the phase completes while the
// warp is parked) is one instruction.
__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, const WaitCtl &w) {
  const uint32_t hint = w.limit_ns < kWaitHintNs ? (uint32_t)w.limit_ns : kWaitHintNs;
  if (__builtin_expect(mbar_try_wait_hint(bar, parity, hint), 1)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < w.limit_ns) {
    if (mbar_try_wait_hint(bar, parity, hint)) return true;
    if (*reinterpret_cast<volatile int *>(w.status) != 0) return false;
  }
  atomicExch(w.status, 1);
  return false;
}
// The n-th item's number, or `stop`: as pipe::next_unit, but the slot is given back by the caller, after it has
// read the item.
__device__ __forceinline__ int next_item(const pipe::UnitRing &r, uint32_t n, int stop) {
  const bool ok = mbar_wait_drain(&r.full[n & 1], parity(n / 2));
  return __shfl_sync(0xffffffffu, ok ? *reinterpret_cast<volatile int *>(&r.slot[n & 1]) : stop, 0);
}
// barrier among a role's warps
template <int ID, int THREADS>
__device__ __forceinline__ void role_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

// a chained segment waits for its incoming state (bounded like every hand-off)
__device__ __forceinline__ bool wait_flag(const int *flag, const WaitCtl &w) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (v) return true;
    if ((i & 15u) == 15u) {
      if (*reinterpret_cast<volatile int *>(w.status) != 0) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0)
        t0 = t;
      else if (t - t0 > w.limit_ns)
        break;
    }
    __nanosleep(100);
  }
  atomicExch(w.status, 1);
  return false;
}

struct Maps {
  CUtensorMap q, k, v, o;
};
struct Args {
  Maps maps[3];
  LaBatch batch;
  LaPlanDev pl;
};

// One item: a unit, a pass, a query head.  The producer works it out and leaves it in shared memory for the
// other roles.
struct Item {
  int pass, unit, h, nb;  // nb: blocks
  int rev, apart;         // apart: lam^-64 is out of reach, products and incoming state have accumulators of their own
  float g;
  int seq, level, next, t0, len;  // of the unit
  template <bool SUMMARY>
  __device__ __forceinline__ void find(const Args &a, int x) {
    const int y = x / a.pl.H;
    h = x - y * a.pl.H;
    unit = y / a.batch.n;
    pass = y - unit * a.batch.n;
    const LaPass &p = a.batch.p[pass];
    rev = p.reverse;
    g = __ldg(p.g + h);
    apart = !(g * kC > -40.f * 0.6931f);
    const LaUnit u = la_unit(a.pl, unit, rev);
    seq = u.seq;
    level = u.level;
    next = u.next;
    t0 = u.t0;
    len = u.len;
    nb = SUMMARY && next < 0 ? 0 : (len + kC - 1) / kC;  // nothing follows a last segment
  }
  // A converged warp's copy.  What comes from memory goes through a shuffle, which tells the
  // compiler that it is the same in all lanes, so that loops and operands that depend on it may stay in
  // uniform registers.
  __device__ __forceinline__ Item uniform() const {
    Item r;
    const volatile int *from = reinterpret_cast<const volatile int *>(this);
    int *to = reinterpret_cast<int *>(&r);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Item) / 4); ++i) to[i] = __shfl_sync(0xffffffffu, from[i], 0);
    return r;
  }
  // processing order: block i is rows [64 blk, 64 blk + nv) of the segment
  __device__ __forceinline__ int block(int i) const { return rev ? nb - 1 - i : i; }
  __device__ __forceinline__ int rows(int i) const { return min(kC, len - block(i) * kC); }
};

// KB, VB: 64-column boxes of the q/k roles and of the v/o roles
// F32: passes with fp32 outputs among them
template <int KB, int VB, bool SUMMARY, bool F32>
__global__ void __launch_bounds__(kThreads, 1) la_tc_kernel(const __grid_constant__ Args args) {
  using L = Layout<KB, VB, SUMMARY, F32>;
  constexpr int ST = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = tc::aligned_smem(smem_raw);
  const LaPlanDev &pl = args.pl;
  const WaitCtl wait{pl.status, pl.wait_ns};
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::kBar + L::kNumBars * 8);
  const Bars<ST> bar(reinterpret_cast<uint64_t *>(sm + L::kBar), reinterpret_cast<int *>(tslot + 1));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  Tables &tab = *reinterpret_cast<Tables *>(sm + L::kTab);
  Item *slots = reinterpret_cast<Item *>(tslot + 4);  // [2]
  const int nitems = __shfl_sync(0xffffffffu, la_units(pl), 0) * args.batch.n * pl.H;

  if (warp == 0 && lane < args.batch.n) {
    const Maps &mp = args.maps[lane];
    prefetch_tmap(&mp.k);
    prefetch_tmap(&mp.v);
    if (!SUMMARY) prefetch_tmap(&mp.q);
    if (!SUMMARY) prefetch_tmap(&mp.o);
  }
  if (threadIdx.x == 64) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.free[i], 1);
    }
    mbar_init(bar.qk_full, 1);
    mbar_init(bar.qk_free, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.v_free[i], 1);
      mbar_init(&bar.p_ready[i], 2);
      mbar_init(&bar.p_free[i], 1);
      mbar_init(&bar.o_full[i], 1);
      mbar_init(&bar.o_free[i], 2 * VB);
      mbar_init(&bar.v_ready[i], 2 * VB);
      mbar_init(&bar.items.full[i], 1);
      mbar_init(&bar.items.free[i], SUMMARY ? 1 + 8 * VB : 3 + 8 * VB);  // every warp but the producer's that takes part
      mbar_init(&bar.w_full[i], 1);
      mbar_init(&bar.w_free[i], 4 * VB);
    }
    mbar_init(bar.s_ready, 4 * VB);
    mbar_init(bar.s_free, 1);
    mbar_init(bar.drain, 1);
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc(tslot, kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);

  // W's buffer of block m, and its use of it
  auto w_at = [&](uint32_t m) { return SUMMARY ? m & 1 : 0u; };
  auto w_use = [&](uint32_t m) { return SUMMARY ? m / 2 : m; };
  constexpr uint32_t kWBufs = SUMMARY ? 2 : 1;

  // Every role counts the blocks it has been through (m): the m-th use of a barrier is
  // its m-th completion, or for pairs and rings completion m / 2 or m / ST of one of them.
  // The block is launched with 640 x 96 registers; the state warps, which hold 64 values of the state a
  // thread, take what the others do not need: 128 x (64 + 104 + 2 * 112 + 88) = 61440.
  if (warp < kOutWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 2) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        int *counter = pl.counters + (SUMMARY ? 0 : 1);
        uint32_t m = 0;
        bool ok = true;
        int next = atomicAdd(counter, 1);
#pragma unroll 1
        for (uint32_t n = 0;; ++n) {
          const int x = ok && (uint32_t)next < (uint32_t)nitems ? next : nitems;
          Item it{};
          if (x < nitems) it.find<SUMMARY>(args, x);
          // the slot of two items ago has been read (if not, it is left alone: an item is never torn)
          if (n >= 2 && !mbar_wait_drain(&bar.items.free[n & 1], parity(n / 2 - 1))) ok = false;
          if (ok) slots[n & 1] = it;
          if (pipe::publish_unit(bar.items, n, ok ? x : nitems, nitems) >= nitems) break;
          const LaPass &p = args.batch.p[it.pass];
          const Maps &mp = args.maps[it.pass];
          const int hq = it.h / p.gq, hk = it.h / p.gk, hv = it.h / p.gv;
#pragma unroll 1
          for (int i = 0; i < it.nb; ++i) {
            const int st = m % ST, row = it.t0 + it.block(i) * kC;
            if (m >= ST && !wait_on(&bar.free[st], parity(m / ST - 1), wait)) {
              ok = false;
              break;
            }
            uint8_t *base = sm + st * L::kStage;
            mbar_expect_tx(&bar.full[st], L::kStage);
            for (int b = 0; b < KB; ++b) {
              if (!SUMMARY) tma_load_3d(base + L::kQ + b * kBox, &mp.q, &bar.full[st], 64 * b, hq, row);
              tma_load_3d(base + L::kK + b * kBox, &mp.k, &bar.full[st], 64 * b, hk, row);
            }
            for (int b = 0; b < VB; ++b) tma_load_3d(base + L::kV + b * kBox, &mp.v, &bar.full[st], 64 * b, hv, row);
            ++m;
          }
          // not earlier: an item that is claimed waits for this one, while other CTAs may be done; the ring is some
          // blocks ahead, which hides the claim
          next = atomicAdd(counter, 1);
        }
        // every load issued has landed before the CTA releases its shared memory
#pragma unroll 1
        for (uint32_t x = m > ST ? m - ST : 0; x < m; ++x) mbar_wait_drain(&bar.full[x % ST], parity(x / ST));
      }
    } else if (warp == 3) {
      // ------------------------------------------------------------ MMA issuer
      // the whole warp, so that descriptors stay in uniform registers; one lane acts
      const uint32_t el = elect_one();
      const uint32_t s0 = smem_u32(sm);
      // K-major: Q (A and B), K, P; MN-major: K as the B operand of W, V (A).  A's 128 rows run
      // past Q's 64 into the shared memory behind it; those rows of the result (and
      // the lanes past 64 when VB = 1) are not read.
      const uint64_t dQ = desc_sw128(s0 + L::kQ, 16, 1024), dK = desc_sw128(s0 + L::kK, 16, 1024),
                     dKn = desc_sw128(s0 + L::kK, kBox, 1024), dV = desc_sw128(s0 + L::kV, kBox, 1024),
                     dP = desc_sw128(s0 + L::kP, 16, 1024);
      constexpr uint32_t iQK = idesc_bf16(128, 64, false, false), iPV = idesc_bf16(128, 64, true, false),
                         iW = idesc_bf16(128, 64 * KB, false, true);
      auto stage = [&](uint32_t m) { return (uint64_t)((m % ST) * (L::kStage / 16)); };
      auto scores = [&](uint32_t m) {
        wait_on(&bar.full[m % ST], parity(m / ST), wait);
        if (m > 0) wait_on(bar.qk_free, parity(m - 1), wait);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < KB; ++b)
          pipe::umma_k_el<4>(el, tmem + kTmQK, dQ + stage(m) + b * (kBox / 16), dK + stage(m) + b * (kBox / 16),
                             pipe::kStepK, pipe::kStepK, iQK, b > 0);
        umma_commit_el(el, bar.qk_full);
      };
      // W of half a block: the three terms' two steps of 16 tokens each
      auto half_w = [&](uint32_t m, int half) {
        wait_on(&bar.v_ready[half], parity(m), wait);
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < 3; ++t)
          pipe::umma_ts_k_el<2>(el, tmem + (w_at(m) ? kTmW1 : kTmW), tmem + kTmT + half * kHalf + t * kTerm,
                                dKn + stage(m) + half * (4096 / 16), 8, pipe::kStepMN, iW, half > 0 || t > 0);
      };
      uint32_t m = 0;
      bool was_apart = false;
#pragma unroll 1
      for (uint32_t n = 0;; ++n) {
        const int x = next_item(bar.items, n, nitems);
        if (x >= nitems) break;
        const Item it = slots[n & 1].uniform();
        pipe::warp_arrive(&bar.items.free[n & 1]);
        const bool apart = it.apart;
        if (!SUMMARY && it.nb > 0) scores(m);
#pragma unroll 1
        for (int i = 0; i < it.nb; ++i, ++m) {
          if (SUMMARY)
            wait_on(&bar.full[m % ST], parity(m / ST), wait);
          else if (i + 1 < it.nb)
            scores(m + 1);
          if (m >= kWBufs) wait_on(&bar.w_free[w_at(m)], parity(w_use(m) - 1), wait);
          half_w(m, 0);
          umma_commit_el(el, &bar.v_free[0]);
          half_w(m, 1);
          umma_commit_el(el, &bar.w_full[w_at(m)]);
          umma_commit_el(el, &bar.v_free[1]);
          if (!SUMMARY) {
            wait_on(bar.s_ready, parity(m), wait);
            // the accumulator of the incoming state's part and, unless apart, of the products:
            // the one of two blocks ago, or after or before a block that uses both the last one's
            const uint32_t acc = tmem + (apart || (m & 1) ? kTmOi : kTmO);
            const uint32_t back = apart || was_apart ? 1 : 2;
            if (m >= back) wait_on(&bar.o_free[(m - back) & 1], parity((m - back) / 2), wait);
            was_apart = apart;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < KB; ++b)
              pipe::umma_ts_k_el<4>(el, acc, tmem + kTmS + 32 * b, dQ + stage(m) + b * (kBox / 16), 8, pipe::kStepK, iQK,
                                    b > 0);
            umma_commit_el(el, bar.s_free);
            wait_on(&bar.p_ready[m & 1], parity(m / 2), wait);
            tc_fence_after();
            pipe::umma_k_el<4>(el, apart ? tmem + kTmO : acc, dV + stage(m), dP + (m & 1) * (kBox / 16), pipe::kStepMN,
                               pipe::kStepK, iPV, !apart);
            umma_commit_el(el, &bar.o_full[m & 1]);
            umma_commit_el(el, &bar.p_free[m & 1]);
          }
          umma_commit_el(el, &bar.free[m % ST]);
        }
      }
      // every MMA and every arrival of a commit has landed before the CTA ends
      umma_commit_el(el, bar.drain);
      mbar_wait_drain(bar.drain, 0);
#pragma unroll 1
      for (uint32_t x = m > ST ? m - ST : 0; x < m; ++x) mbar_wait_drain(&bar.free[x % ST], parity(x / ST));
      if (m > 0) {
#pragma unroll 1
        for (uint32_t x = m > kWBufs ? m - kWBufs : 0; x < m; ++x) mbar_wait_drain(&bar.w_full[w_at(x)], parity(w_use(x)));
        mbar_wait_drain(&bar.v_free[0], parity(m - 1));
        mbar_wait_drain(&bar.v_free[1], parity(m - 1));
      }
      if (!SUMMARY && m > 0) {
        mbar_wait_drain(bar.qk_full, parity(m - 1));
        mbar_wait_drain(bar.s_free, parity(m - 1));
#pragma unroll 1
        for (uint32_t x = m > 2 ? m - 2 : 0; x < m; ++x) {
          mbar_wait_drain(&bar.p_free[x & 1], parity(x / 2));
          mbar_wait_drain(&bar.o_full[x & 1], parity(x / 2));
        }
      }
    } else if (!SUMMARY) {
      // ------------------------------------------------------------ P
      const int r = threadIdx.x;  // row of the block
      uint32_t m = 0;
#pragma unroll 1
      for (uint32_t n = 0;; ++n) {
        const int x = next_item(bar.items, n, nitems);
        if (x >= nitems) break;
        const Item it = slots[n & 1].uniform();
        pipe::warp_arrive(&bar.items.free[n & 1]);
        const LaPass &p = args.batch.p[it.pass];
        const bool rev = it.rev, apart = it.apart;
        // Masks of this row's bf16 pairs in the two 16-column groups that the diagonal
        // crosses (columns 32 warp and 32 warp + 16): masked scores may be NaN, so they
        // are cut off as bits, after weights that need not be right there.
        uint32_t keep[16];
#pragma unroll
        for (int y = 0; y < 16; ++y)
          keep[y] = ((rev ? 2 * y >= lane : 2 * y <= lane) ? 0xffffu : 0u) |
                    ((rev ? 2 * y + 1 >= lane : 2 * y + 1 <= lane) ? 0xffff0000u : 0u);
        auto fill = [&](int nv) {  // the weights of blocks of nv rows (in order they do not depend on it)
          role_sync<4, 64>();
          tab.p[r] = p.p_scale * (apart ? p.o_scale * la_pow(it.g, r) : la_pow(it.g, rev ? r + 1 - nv : -1 - r));
          role_sync<4, 64>();
        };
        // usual: not apart, all rows live
        auto block = [&](auto usual, int nv) {
          constexpr bool kUsual = decltype(usual)::value;
          if (m >= 2) wait_on(&bar.p_free[m & 1], parity(m / 2 - 1), wait);
          wait_on(bar.qk_full, parity(m), wait);
          tc_fence_after();
          const uint32_t dst = smem_u32(sm + L::kP + (m & 1) * kBox);
#pragma unroll 1
          for (int j0 = 0; j0 < kC; j0 += 16) {
            const int at = j0 - 32 * warp;  // the group's place against the diagonal: 0 and 16 cross it
            uint4 p0 = make_uint4(0, 0, 0, 0), p1 = p0;
            if (rev ? at >= 0 : at < 32) {
              float s[16], v[8];
              tmem_ld16(pipe::tmem_quad(tmem + kTmQK, j0), s);
              if (!kUsual && rev) {  // columns past the end are masked for the rows before it too
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = j0 + e < nv ? s[e] : 0.f;
              }
              if (!kUsual && apart) {
                const float *w = tab.p + (rev ? j0 - r : r - j0);  // where masked, whatever lies there
                const int step = rev ? 1 : -1;
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] *= w[step * e];
              } else {
                const ulonglong2 *w = reinterpret_cast<const ulonglong2 *>(tab.p + j0);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const ulonglong2 t = w[e / 4];
                  upk2(mul2(t.x, pk2(s[e], s[e + 1])), s[e], s[e + 1]);
                  upk2(mul2(t.y, pk2(s[e + 2], s[e + 3])), s[e + 2], s[e + 3]);
                }
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = s[e];
              p0 = tc::pack8(v);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = s[8 + e];
              p1 = tc::pack8(v);
              if (at == 0) {
                p0.x &= keep[0]; p0.y &= keep[1]; p0.z &= keep[2]; p0.w &= keep[3];
                p1.x &= keep[4]; p1.y &= keep[5]; p1.z &= keep[6]; p1.w &= keep[7];
              } else if (at == 16) {
                p0.x &= keep[8]; p0.y &= keep[9]; p0.z &= keep[10]; p0.w &= keep[11];
                p1.x &= keep[12]; p1.y &= keep[13]; p1.z &= keep[14]; p1.w &= keep[15];
              }
            }
            pipe::sts_u4(dst + sw128_offset(r, j0), p0);
            pipe::sts_u4(dst + sw128_offset(r, j0 + 8), p1);
          }
          tc_fence_before();
          pipe::warp_arrive(bar.qk_free);
          fence_async_smem();
          pipe::warp_arrive(&bar.p_ready[m & 1]);
        };
        int have = 0;  // rows that the weights are for
#pragma unroll 1
        for (int i = 0; i < it.nb; ++i, ++m) {
          const int nv = it.rows(i);
          if (nv != have) fill(have = nv);
          if (!apart && nv == kC)
            block(std::true_type{}, kC);
          else
            block(std::false_type{}, nv);
        }
      }
    }
  } else if (!SUMMARY && warp < kStateWarp0) {
    // ------------------------------------------------------------ outputs
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    if (warp < kOutWarp0 + 2 * VB) {
      constexpr int kOutThreads = 64 * VB;
      const int tt = threadIdx.x - 32 * kOutWarp0, quad = warp & 3;
      // the address this lane gives to a group of four fragments: row i, columns of v
      const int fi = 8 * (lane >> 4) + (lane & 7), fc = 32 * quad + 8 * ((lane >> 3) & 1);
      const uint32_t so = smem_u32(sm + L::kO);
      uint32_t m = 0;
#pragma unroll 1
      for (uint32_t n = 0;; ++n) {
        const int x = next_item(bar.items, n, nitems);
        if (x >= nitems) break;
        const Item it = slots[n & 1].uniform();
        pipe::warp_arrive(&bar.items.free[n & 1]);
        const LaPass &p = args.batch.p[it.pass];
        const bool rev = it.rev, apart = it.apart, f32 = F32 && p.o_f32;
        // (the kinds of output share the staging tile; the warps meet in fill)
        if (F32 && lane == 0) bulk_wait_read0();
        uint64_t w[8];  // what this lane's columns i weigh, in pairs
        auto fill = [&](int nv) {  // the weights of blocks of nv rows (in order those of a full one will do)
          role_sync<2, kOutThreads>();
          for (int r = tt; r < kC; r += kOutThreads)
            tab.out[r] = p.o_scale * la_pow(it.g, rev ? max(nv - 1 - r, 0) : r + 1);
          role_sync<2, kOutThreads>();
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = *reinterpret_cast<const uint64_t *>(tab.out + 8 * e + 2 * (lane & 3));
        };
        // usual: not apart, all rows live
        auto block = [&](auto usual, int nv, long long row0) {
          constexpr bool kUsual = decltype(usual)::value;
          if (f32) {  // the block before has been read out of the staging tile (fp32: the warp's own part)
            if (lane == 0) bulk_wait_read0();
            __syncwarp();
          } else {
            if (tt == 0) bulk_wait_read0();
            role_sync<2, kOutThreads>();
          }
          auto emit = [&](int half, const uint32_t(&a)[32]) {  // 16 lanes (columns of v) x 64 rows i
            if (f32 && kUsual) {  // a box of 16 columns x 64 rows of 64 bytes, in their swizzle
              const uint32_t to = so + (2 * (tt >> 5) + half) * 4096;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int r = 8 * (e >> 2) + 2 * (lane & 3) + (e & 1), c = (lane >> 2) + 4 * (e & 2);
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + r * 64 + (((c >> 2) ^ (lane & 3)) << 4) + (c & 3) * 4), "r"(a[e])
                             : "memory");
              }
            } else if (f32) {
              float *dst = static_cast<float *>(p.o) + row0 * p.os + (long long)it.h * p.dv;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int r = 8 * (e >> 2) + 2 * (lane & 3) + (e & 1), c = 32 * quad + 16 * half + (lane >> 2) + 4 * (e & 2);
                if (r < nv && c < p.dv) dst[r * p.os + c] = __uint_as_float(a[e]);
              }
            } else {
              const int c = fc + 16 * half;
              // 8 rows on it is the same place in the swizzle
              const uint32_t to = so + (uint32_t)(c >> 6) * kBox + sw128_offset(fi, c & 63);
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                uint32_t f[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  f[y] = tc::pack_bf16x2(__uint_as_float(a[4 * e + 2 * y]), __uint_as_float(a[4 * e + 2 * y + 1]));
                stmatrix4_trans(to + e * 1024, f[0], f[1], f[2], f[3]);
              }
            }
          };
          const uint32_t lo = pipe::tmem_quad(tmem, (!kUsual && apart) || (m & 1) ? kTmOi : kTmO), hi = lo + (16u << 16);
          wait_on(&bar.o_full[m & 1], parity(m / 2), wait);
          tc_fence_after();
          uint32_t a[32], b[32];
          tmem_ld_16x256_async(lo, a);
          tmem_ld_16x256_async(hi, b);
          tmem_wait_ld32(a);
          tmem_wait_ld32(b);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float f0, f1;
            upk2(mul2(w[e >> 2], pk2(__uint_as_float(a[e]), __uint_as_float(a[e + 1]))), f0, f1);
            a[e] = __float_as_uint(f0);
            a[e + 1] = __float_as_uint(f1);
            upk2(mul2(w[e >> 2], pk2(__uint_as_float(b[e]), __uint_as_float(b[e + 1]))), f0, f1);
            b[e] = __float_as_uint(f0);
            b[e + 1] = __float_as_uint(f1);
          }
          if (!kUsual && apart) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t t[16];
              tmem_ld_16x256_x4_async(pipe::tmem_quad(tmem, kTmO) + ((uint32_t)(16 * (q >> 1)) << 16) + 32 * (q & 1), t);
              tmem_wait_ld16(t);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                uint32_t &y = q < 2 ? a[16 * (q & 1) + e] : b[16 * (q & 1) + e];
                y = __float_as_uint(__uint_as_float(y) + __uint_as_float(t[e]));
              }
            }
          }
          tc_fence_before();
          pipe::warp_arrive(&bar.o_free[m & 1]);
          emit(0, a);
          emit(1, b);
          if (f32 && kUsual) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const int c = 32 * quad + 16 * half;
                if (c < p.dv) tma_store_3d(&args.maps[it.pass].o, so + (2 * (tt >> 5) + half) * 4096, c, it.h, (int)row0);
              }
              bulk_commit();
            }
          }
          if (!f32) {
            fence_async_smem();
            role_sync<2, kOutThreads>();
            if (!kUsual && nv < kC) {  // rows past the end belong to another sequence: row by row
              bf16 *out = static_cast<bf16 *>(p.o) + row0 * p.os + (long long)it.h * p.dv;
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
            } else if (tt == 0) {
              for (int y = 0; y < VB; ++y)
                if (64 * y < p.dv) tma_store_3d(&args.maps[it.pass].o, so + y * kBox, 64 * y, it.h, (int)row0);
              bulk_commit();
            }
          }
        };
        int have = 0;  // rows that the weights are for
#pragma unroll 1
        for (int i = 0; i < it.nb; ++i, ++m) {
          const int nv = it.rows(i);
          const long long row0 = it.t0 + (long long)it.block(i) * kC;
          if (nv != have) fill(have = nv);
          if (!apart && nv == kC)
            block(std::true_type{}, kC, row0);
          else
            block(std::false_type{}, nv, row0);
        }
      }
      if (F32 ? lane == 0 : tt == 0) bulk_wait0();
    }
  } else if (warp >= kStateWarp0 && warp < kWeighWarp0) {
    // ------------------------------------------------------------ state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    if ((warp & 3) < 2 * VB) {
      constexpr int kCols = 32 * KB;  // state rows (dk) of a thread
      const int quad = warp & 3, sub = (warp - kStateWarp0) >> 2;  // two warps share a quadrant of lanes
      const int c = 32 * quad + lane, a0 = sub * kCols;
      uint64_t S[kCols / 2];  // pairs along dk
      uint32_t m = 0;
      auto publish = [&] {  // S^T as the A operand: lane = column of v, bf16 pairs along dk
        if (!SUMMARY) {
          if (m > 0) wait_on(bar.s_free, parity(m - 1), wait);
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
          tc_fence_before();
          pipe::warp_arrive(bar.s_ready);
        }
      };
#pragma unroll 1
      for (uint32_t n = 0;; ++n) {
        const int x = next_item(bar.items, n, nitems);
        if (x >= nitems) break;
        const Item it = slots[n & 1].uniform();
        pipe::warp_arrive(&bar.items.free[n & 1]);
        const LaPass &p = args.batch.p[it.pass];
        // this item's place among the flags of the units' incoming states
        auto flag = [&](int unit) { return pl.flags + ((size_t)it.pass * pl.units + unit) * pl.H + it.h; };
        {
          int sa, sb;
          const float *in = SUMMARY ? nullptr : la_state_in(p, it.level, it.next, it.seq, it.unit, it.h, sa, sb);
          if (!SUMMARY && pl.flags && it.level > 0) wait_flag(flag(it.unit), wait);
          const bool live = in && c < p.dv;
#pragma unroll
          for (int a = 0; a < kCols; a += 2) {  // dk is even
            float f0 = 0.f, f1 = 0.f;
            if (live && a0 + a < p.dk) {
              f0 = in[(size_t)(a0 + a) * sa + (size_t)c * sb];
              f1 = in[(size_t)(a0 + a + 1) * sa + (size_t)c * sb];
            }
            S[a / 2] = pk2(f0, f1);
          }
        }
        float2 carry = make_float2(0.f, 0.f);
        int have = 0;  // rows that carry is for
#pragma unroll 1
        for (int i = 0; i < it.nb; ++i, ++m) {
          publish();
          const int nv = it.rows(i);
          if (nv != have) carry = la_pow2(it.g, have = nv);
          const uint64_t chi = pk2(carry.x, carry.x), clo = pk2(carry.y, carry.y);
          wait_on(&bar.w_full[w_at(m)], parity(w_use(m)), wait);
          tc_fence_after();
#pragma unroll
          for (int x2 = 0; x2 < kCols; x2 += 32) {
            float w[32];
            tmem_ld32(pipe::tmem_quad(tmem + (w_at(m) ? kTmW1 : kTmW), a0 + x2), w);
            if (x2 + 32 == kCols) {
              tc_fence_before();
              pipe::warp_arrive(&bar.w_free[w_at(m)]);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              uint64_t &t = S[x2 / 2 + e];
              t = fma2(t, chi, fma2(t, clo, pk2(w[2 * e], w[2 * e + 1])));
            }
          }
        }
        int sa, sb;
        const bool hand_on = SUMMARY || pl.flags;
        float *out = la_state_out(p, it.next, it.seq, it.h, hand_on, sa, sb);
        if (out && c < p.dv && (!SUMMARY || it.next >= 0)) {
#pragma unroll
          for (int a = 0; a < kCols; a += 2) {
            float f0, f1;
            upk2(S[a / 2], f0, f1);
            if (a0 + a < p.dk) {
              out[(size_t)(a0 + a) * sa + (size_t)c * sb] = f0;
              out[(size_t)(a0 + a + 1) * sa + (size_t)c * sb] = f1;
            }
          }
        }
        if (!SUMMARY && pl.flags && it.next >= 0) {  // the state warps' stores, then the flag
          __threadfence();
          role_sync<3, 128 * VB>();
          if (warp == kStateWarp0 && lane == 0)
            asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(flag(it.next)) : "memory");
        }
      }
    }
  } else {
    // ------------------------------------------------------------ weighted V
    // summaries: with the warps that have no outputs to write, each half of a block by warps of its own
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    constexpr int kTeam = SUMMARY ? 128 * VB : 64 * VB;
    const int quad = warp & 3, first = SUMMARY && warp >= kWeighWarp0 ? 1 : 0, tt = quad * 32 + lane + first * 64 * VB;
    if (quad < 2 * VB) {
      // half-blocks of 32 tokens in order; matrix loads of 8 tokens x 8 columns (lane: its
      // address), 16 tokens and 16 columns of v at a time
      const uint32_t s0 = smem_u32(sm);
      const int lr = (lane & 7) + 8 * (lane >> 4), lc = 32 * (quad & 1) + 8 * ((lane >> 3) & 1);
      uint32_t m = 0;
#pragma unroll 1
      for (uint32_t n = 0;; ++n) {
        const int x = next_item(bar.items, n, nitems);
        if (x >= nitems) break;
        const Item it = slots[n & 1].uniform();
        pipe::warp_arrive(&bar.items.free[n & 1]);
        const float st_scale = args.batch.p[it.pass].st_scale;
        auto fill = [&](int nv) {  // the weights of blocks of nv rows
          role_sync<5, kTeam>();
          for (int j = tt; j < kC; j += kTeam)
            tab.st[j] = st_scale * la_pow(it.g, it.rev ? j + 1 : max(nv - 1 - j, 0));
          role_sync<5, kTeam>();
        };
        // usual: all rows live
        auto block = [&](auto usual, int nv) {
          constexpr bool kUsual = decltype(usual)::value;
          const int st = m % ST;
          const uint32_t sv = s0 + st * L::kStage + L::kV + (uint32_t)(quad >> 1) * kBox;
          wait_on(&bar.full[st], parity(m / ST), wait);
          if (!kUsual) {  // rows past the end of K and V, which are operands as they are, become zeros
            const uint32_t sk = s0 + st * L::kStage + L::kK;  // V's boxes follow K's
            for (int e = quad * 32 + lane; e < (kC - nv) * 8 * (KB + VB); e += 64 * VB) {
              const int y = e % (8 * (KB + VB)), r = nv + e / (8 * (KB + VB));
              pipe::sts_u4(sk + (uint32_t)(y >> 3) * kBox + sw128_offset(r, 8 * (y & 7)), make_uint4(0, 0, 0, 0));
            }
            fence_async_smem();
          }
#pragma unroll 1
          for (int half = first; half < (SUMMARY ? first + 1 : 2); ++half) {
            if (m > 0) {
              wait_on(&bar.v_free[half], parity(m - 1), wait);
              tc_fence_after();
            }
            uint64_t w[4];  // weights of tokens 8 y + 2 (lane % 4) and the next of this half
#pragma unroll
            for (int y = 0; y < 4; ++y)
              w[y] = *reinterpret_cast<const uint64_t *>(tab.st + 32 * half + 8 * y + 2 * (lane & 3));
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
              uint32_t f[8], t0[8], t1[8], t2[8];
              const uint32_t row = sv + (32 * half + lr) * 128 + (uint32_t)((((lc >> 3) + 2 * q) ^ (lane & 7)) * 16);
              ldmatrix4_trans(row, f[0], f[1], f[2], f[3]);
              ldmatrix4_trans(row + 16 * 128, f[4], f[5], f[6], f[7]);
              if (!kUsual) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int j = 32 * half + 8 * (e >> 1) + 2 * (lane & 3);
                  f[e] &= (j < nv ? 0xffffu : 0u) | (j + 1 < nv ? 0xffff0000u : 0u);
                }
              }
#pragma unroll
              for (int e = 0; e < 8; ++e)
                split3(mul2(w[e >> 1], pk2(lo_f(f[e]), hi_f(f[e]))), t0[e], t1[e], t2[e]);
              const uint32_t at = pipe::tmem_quad(tmem + kTmT + half * kHalf, 0) + ((uint32_t)(16 * q) << 16);
              tmem_st_16x128_async(at, t0);
              tmem_st_16x128_async(at + kTerm, t1);
              tmem_st_16x128_async(at + 2 * kTerm, t2);
            }
            tmem_wait_st();
            tc_fence_before();
            pipe::warp_arrive(&bar.v_ready[half]);
          }
        };
        int have = 0;  // rows that the weights are for
#pragma unroll 1
        for (int i = 0; i < it.nb; ++i, ++m) {
          const int nv = it.rows(i);
          if (nv != have) fill(have = nv);
          if (nv == kC)
            block(std::true_type{}, kC);
          else
            block(std::false_type{}, nv);
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

template <int KB, int VB, bool SUMMARY, bool F32>
void run_tc(const LaPlanDev &pl, const LaBatch &b, cudaStream_t s) {
  using L = Layout<KB, VB, SUMMARY, F32>;
  static std::atomic<uint64_t> allowed{0};
  allow_smem(reinterpret_cast<const void *>(la_tc_kernel<KB, VB, SUMMARY, F32>), L::kBytes, allowed);
  Args args;
  args.batch = b;
  args.pl = pl;
  for (int i = 0; i < b.n; ++i) {
    const LaPass &p = b.p[i];
    Maps &mp = args.maps[i];
    if ((!SUMMARY && !encode_tmap_bf16_heads(&mp.q, p.q, p.dk, p.Hq, pl.total, p.qs * 2, kC)) ||
        (!SUMMARY && !(p.o_f32 ? encode_tmap_f32_heads(&mp.o, p.o, p.dv, p.H, pl.total, p.os * 4, kC)
                               : encode_tmap_bf16_heads(&mp.o, p.o, p.dv, p.H, pl.total, p.os * 2, kC))) ||
        !encode_tmap_bf16_heads(&mp.k, p.k, p.dk, p.Hk, pl.total, p.ks * 2, kC) ||
        !encode_tmap_bf16_heads(&mp.v, p.v, p.dv, p.Hv, pl.total, p.vs * 2, kC)) {
      note_host_error();
      return;
    }
  }
  const long long items = (long long)pl.units * b.n * pl.H;
  const int grid = items < device_sm_count() ? (int)items : device_sm_count();
  la_tc_kernel<KB, VB, SUMMARY, F32><<<grid, kThreads, L::kBytes, s>>>(args);
}

template <int KB, int VB>
void run_tc_mode(const LaPlanDev &pl, const LaBatch &b, bool summary, cudaStream_t s) {
  if (summary)
    run_tc<KB, VB, true, false>(pl, b, s);
  else {
    bool f32 = false;
    for (int i = 0; i < b.n; ++i) f32 = f32 || b.p[i].o_f32;
    f32 ? run_tc<KB, VB, false, true>(pl, b, s) : run_tc<KB, VB, false, false>(pl, b, s);
  }
}

}  // namespace

void launch_la_tc(const LaPlanDev &pl, const LaBatch &b, bool summary, cudaStream_t s) {
  const int kb = la_tc_boxes(b.p[0].dk), vb = la_tc_boxes(b.p[0].dv);
  if (kb == 1)
    vb == 1 ? run_tc_mode<1, 1>(pl, b, summary, s) : run_tc_mode<1, 2>(pl, b, summary, s);
  else
    vb == 1 ? run_tc_mode<2, 1>(pl, b, summary, s) : run_tc_mode<2, 2>(pl, b, summary, s);
}

}  // namespace ssd
