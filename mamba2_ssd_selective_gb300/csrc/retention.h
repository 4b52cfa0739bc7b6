// Linear attention with a decay for each head, internal: the description of one
// pass over the sequences and its launchers.
//
// Everything the forward and the backward need is one pass with three roles,
//     S_t = lam S_{t-1} + k_t^T v_t,   o_t = q_t S_t
// over the tokens in order or (reverse) from the last to the first:
//     o   = pass(q, k, v)                dq = pass(do, v, k)  (its state is S transposed)
//     dv  = reverse(k, q, do)            dk = reverse(v, do, q)  (its state transposed)
// where the reverse state R at token t is the gradient of the state after t:
//     R_t = scale q_t^T do_t + lam R_{t+1},  dinitial = lam R_0.
//
// Blocks of C tokens: with nv live tokens in a block, row r weighs what comes in
// with lam^a(r), what it adds to the outgoing state with lam^b(r), and the state
// itself is carried by lam^nv:
//     in order: a = r + 1, b = nv - 1 - r;   reverse: a = nv - 1 - r, b = r + 1.
#pragma once

#include "launch.h"

namespace ssd {

// packed calls of more sequences are never cut
constexpr int kLaMaxCutSeqs = 1024;
// work counters of a call: two for each of up to three batches of passes
constexpr int kLaCounterWords = 6;

struct LaPass {
  const void *q, *k, *v;
  void *o;
  long long qs, ks, vs, os;  // token strides (elements)
  int gq, gk, gv;            // query heads that share one head of the role's tensor
  int dk, dv;                // widths of the q/k roles and of the v/o roles
  int H, Hq, Hk, Hv;         // query heads; heads of each role's tensor
  bool reverse;
  float o_scale;   // factor of the output
  float p_scale;   // factor of the products inside a block, on top of it
  float st_scale;  // factor of what is added to the state
  const float *g;  // (H) log decays
  // states, element (a, b) of a (dk x dv) state at a * sa + b * sb
  const float *init;
  float *fin;
  int sa, sb;
  float *seg_state;  // (units, H, dk, dv): a cut sequence's segment states
  bool seg_shared;   // they are another pass's, transposed: (units, H, dv, dk), read only
  bool init_kept;    // fin is init, and the scan keeps what cut sequences start from in their first units' places
  bool o_f32;        // o is fp32 whatever the inputs' type
};

// A unit is one segment of one sequence: its level-th in processing order.  Units are
// numbered level by level (all first segments, then all second ones, ...), so
// that whoever takes them in order never waits for a unit that nobody has taken.
struct LaEntry {
  int seq, level, nseg, a, len, next;  // a, len: the sequence's rows; next: the unit after it, or -1
};
// The sequences and how they are cut; common to the passes of a call.
struct LaPlanDev {
  int nseq, seqlen, total, H;
  const int *cu;
  int seg_len;            // tokens of a segment, a multiple of the blocks' tokens
  int units;              // units, or with a table an upper bound of them
  const LaEntry *table;   // packed sequences that may be cut: written by la_table_kernel
  const int *table_units; // and their number
  int *status;            // status word
  int *counters;          // work counters of the persistent kernels: two for each batch of passes
  int *flags;             // (passes, units, H): the unit's incoming state is written (chained segments), or null
  unsigned long long wait_ns;
};
// Passes that one launch works on.
struct LaBatch {
  LaPass p[3];
  int n;
};

__device__ __forceinline__ void la_seq_bounds(const LaPlanDev &pl, int s, int &a, int &len) {
  if (pl.cu) {
    a = min(max(__ldg(pl.cu + s), 0), pl.total);
    len = max(min(max(__ldg(pl.cu + s + 1), 0), pl.total) - a, 0);
  } else {
    a = s * pl.seqlen;
    len = pl.seqlen;
  }
}
// segments of a sequence (an empty one has one empty segment, so that its state is passed on)
__host__ __device__ __forceinline__ int la_segments(int len, int seg_len) {
  return len <= seg_len ? 1 : (len - 1) / seg_len + 1;
}
__device__ __forceinline__ int la_units(const LaPlanDev &pl) { return pl.table ? *pl.table_units : pl.units; }

struct LaUnit {
  int seq, level, nseg, next, t0, len;  // rows [t0, t0 + len)
};
__device__ __forceinline__ LaUnit la_unit(const LaPlanDev &pl, int unit, bool reverse) {
  LaUnit u;
  int a, len;
  if (pl.table) {
    const LaEntry &e = pl.table[unit];
    u.seq = e.seq;
    u.level = e.level;
    u.nseg = e.nseg;
    u.next = e.next;
    a = e.a;
    len = e.len;
  } else {
    u.level = unit / pl.nseq;
    u.seq = unit - u.level * pl.nseq;
    la_seq_bounds(pl, u.seq, a, len);
    u.nseg = pl.cu ? 1 : la_segments(len, pl.seg_len);
    u.next = u.level + 1 < u.nseg ? unit + pl.nseq : -1;
  }
  const int seg = reverse ? u.nseg - 1 - u.level : u.level;
  u.t0 = a + seg * pl.seg_len;
  u.len = u.nseg == 1 ? len : min(pl.seg_len, len - seg * pl.seg_len);
  return u;
}

// The state before the unit's first token in processing order, or null (zero), and its strides: the segment's, or
// the user's for a sequence's first segment (unless that is where its last segment's state goes).
__device__ __forceinline__ const float *la_state_in(const LaPass &p, int level, int next, int seq, int unit, int h,
                                                    int &sa, int &sb) {
  const size_t dd = (size_t)p.dk * p.dv;
  sa = p.sa;
  sb = p.sb;
  if (level == 0 && !(p.init_kept && next >= 0)) return p.init ? p.init + ((size_t)seq * p.H + h) * dd : nullptr;
  sa = p.seg_shared ? 1 : p.dv;
  sb = p.seg_shared ? p.dk : 1;
  return p.seg_state + ((size_t)unit * p.H + h) * dd;
}
// Where the unit's state goes, or null: with to_next the next unit's incoming state, else (and for the last
// segment) the user's final state.
__device__ __forceinline__ float *la_state_out(const LaPass &p, int next, int seq, int h, bool to_next, int &sa, int &sb) {
  const size_t dd = (size_t)p.dk * p.dv;
  const bool last = next < 0;
  sa = last ? p.sa : p.dv;
  sb = last ? p.sb : 1;
  if (!last) return to_next ? p.seg_state + ((size_t)next * p.H + h) * dd : nullptr;
  return p.fin ? p.fin + ((size_t)seq * p.H + h) * dd : nullptr;
}

// lam^n in fp32; lam^0 is 1 even for a log decay of -inf
__device__ __forceinline__ float la_pow(float g, int n) { return n == 0 ? 1.f : expf(g * (float)n); }
// lam^n as a sum of two fp32 values: a state is multiplied by it once per block,
// for as many blocks as it lives, so that an error of its own would add up.  A
// state lives for about 1 / (1 - lam^n) blocks, so the error has to be small
// against 1 - lam^n, which expm1 gives.
__device__ __forceinline__ float2 la_pow2(float g, int n) {
  const float e = n == 0 ? 0.f : expm1f(g * (float)n), hi = 1.f + e;
  return make_float2(hi, e - (hi - 1.f));
}

// la_plan.cu: clears status, counters and flags; writes the table of units
void launch_la_table(const LaPlanDev &pl, LaEntry *table, int *table_units, int nflags, cudaStream_t s);
// la_simt.cu: any type and width of the envelope.  summary: the segments' own states
// (from zero), each where the next segment's incoming state will be
template <typename T> void launch_la_simt(const LaPlanDev &pl, const LaBatch &b, bool summary, cudaStream_t s);
// la_tc.cu: bf16, both widths at most 128 (all passes of a batch of the same boxes)
inline bool la_tc_envelope(int dk, int dv) { return dk <= 128 && dv <= 128; }
inline int la_tc_boxes(int width) { return width <= 64 ? 1 : 2; }
void launch_la_tc(const LaPlanDev &pl, const LaBatch &b, bool summary, cudaStream_t s);
// segments' own states -> incoming states, in place (either path)
void launch_la_scan(const LaPlanDev &pl, const LaBatch &b, cudaStream_t s);
// sums fp32 (rows, H, d) over groups of query heads into (rows, Hkv, d), for two tensors
struct LaHeadSum {
  const float *in;
  void *out;
  long long os;
  int d;
};
template <typename T>
void launch_la_sum_heads(const LaHeadSum &x, const LaHeadSum &y, long long rows, int Hkv, int group, cudaStream_t s);
// la_step.cu
template <typename T>
void launch_la_step(const LaPass &p, int rows, float *states, int nslots, const int *slot_idx, cudaStream_t s);

}  // namespace ssd
