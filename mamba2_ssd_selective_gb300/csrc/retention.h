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

struct LaPass {
  const void *q, *k, *v;
  void *o;
  long long qs, ks, vs, os;  // token strides (elements)
  int gq, gk, gv;            // query heads that share one head of the role's tensor
  int dk, dv;                // widths of the q/k roles and of the v/o roles
  int H, Hq, Hk, Hv;         // query heads; heads of each role's tensor
  float o_scale;             // factor of the output
  float p_scale;             // factor of the products inside a block, on top of it
  float st_scale;            // factor of what is added to the state
  const float *g;            // (H) log decays
  // states, element (a, b) of a (dk x dv) state at a * sa + b * sb
  const float *init;
  float *fin;
  int sa, sb;
  // sequences
  int nseq, seqlen, total;
  const int *cu;
  int seg_len;  // tokens of a segment (a multiple of the blocks' tokens)
  int nunits;   // upper bound of the segments of all sequences
  bool split;   // sequences longer than seg_len are cut: seg_state[u, h] holds their segments' states
  float *seg_state;
  bool o_f32;  // o is fp32 whatever the inputs' type
  int *status;
  unsigned long long wait_ns;
};

// One segment of a sequence: tokens [t0, t0 + len) of the rows, seg-th of its sequence.
struct LaUnit {
  int seq, seg, nseg, t0, len;
};

__device__ __forceinline__ void la_seq_bounds(const LaPass &p, int s, int &a, int &len) {
  if (p.cu) {
    a = min(max(__ldg(p.cu + s), 0), p.total);
    len = max(min(max(__ldg(p.cu + s + 1), 0), p.total) - a, 0);
  } else {
    a = s * p.seqlen;
    len = p.seqlen;
  }
}
// segments of a sequence (an empty one has one empty segment, so that its state is passed on)
__device__ __forceinline__ int la_segments(const LaPass &p, int len) {
  return len <= p.seg_len ? 1 : (len - 1) / p.seg_len + 1;
}

// Segment u of all sequences in order; by a full warp.  false: there is no such segment.
__device__ __forceinline__ bool la_find_unit(const LaPass &p, int u, LaUnit &out) {
  int s, seg, a, len;
  if (!p.cu) {
    const int per = la_segments(p, p.seqlen);
    s = u / per;
    seg = u - s * per;
    if (s >= p.nseq) return false;
  } else {
    const int lane = threadIdx.x & 31;
    int base = 0;
    s = -1;
    seg = 0;
    for (int s0 = 0; s0 < p.nseq; s0 += 32) {
      int n = 0;
      if (s0 + lane < p.nseq) {
        la_seq_bounds(p, s0 + lane, a, len);
        n = la_segments(p, len);
      }
      int inc = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += x;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + inc > u);
      if (hit) {
        const int l = __ffs(hit) - 1;
        s = s0 + l;
        seg = u - base - __shfl_sync(0xffffffffu, inc - n, l);
        break;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (s < 0) return false;
  }
  la_seq_bounds(p, s, a, len);
  out.seq = s;
  out.seg = seg;
  out.t0 = a + seg * p.seg_len;
  out.len = min(p.seg_len, len - seg * p.seg_len);
  out.nseg = la_segments(p, len);
  return true;
}

// The state before the unit's first token in processing order, or null (zero), and its strides: the segment's, or
// the user's for a sequence that is not cut.
__device__ __forceinline__ const float *la_state_in(const LaPass &p, const LaUnit &u, int unit, int h, int &sa, int &sb) {
  const size_t dd = (size_t)p.dk * p.dv;
  sa = p.sa;
  sb = p.sb;
  if (u.nseg == 1) return p.init ? p.init + ((size_t)u.seq * p.H + h) * dd : nullptr;
  sa = p.dv;
  sb = 1;
  return p.seg_state + ((size_t)unit * p.H + h) * dd;
}
// whether the unit is its sequence's last in processing order
__device__ __forceinline__ bool la_is_last(const LaUnit &u, bool reverse) {
  return reverse ? u.seg == 0 : u.seg == u.nseg - 1;
}
// Where the unit's state goes, or null: the summary's segment state, the user's final state of a sequence.
__device__ __forceinline__ float *la_state_out(const LaPass &p, const LaUnit &u, int unit, int h, bool reverse,
                                               bool summary, int &sa, int &sb) {
  const size_t dd = (size_t)p.dk * p.dv;
  sa = summary ? p.dv : p.sa;
  sb = summary ? 1 : p.sb;
  if (summary) return p.seg_state + ((size_t)unit * p.H + h) * dd;
  return p.fin && la_is_last(u, reverse) ? p.fin + ((size_t)u.seq * p.H + h) * dd : nullptr;
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

// la_simt.cu: any type and width of the envelope
template <typename T> void launch_la_simt(const LaPass &p, bool reverse, bool summary, cudaStream_t s);
// la_tc.cu: bf16, both widths at most 128
inline bool la_tc_envelope(int dk, int dv) { return dk <= 128 && dv <= 128; }
void launch_la_tc(const LaPass &p, bool reverse, bool summary, cudaStream_t s);
// segment states -> incoming segment states, in place (either path)
void launch_la_scan(const LaPass &p, bool reverse, cudaStream_t s);
// sums fp32 (rows, H, d) over groups of query heads into (rows, Hkv, d)
template <typename T>
void launch_la_sum_heads(const float *in, void *out, long long os, long long rows, int Hkv, int group, int d,
                         cudaStream_t s);
// la_step.cu
template <typename T>
void launch_la_step(const LaPass &p, float *states, int nslots, const int *slot_idx, cudaStream_t s);

}  // namespace ssd
