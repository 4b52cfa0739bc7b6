// The gated delta rule, internal: a call's description, the chunks' tables and their launchers.
//
// Per state head, with a_t = exp(log_decay_t), b_t = beta_t and k, q of length 1 where qk_norm says so:
//     S' = a_t S_{t-1},   S_t = S' + b_t k_t^T (v_t - k_t S'),   o_t = scale q_t S_t
// Chunks of 64 tokens.  G_i: the sum of the chunk's log decays up to token i, S: the state before the chunk.
//     A_ij = e^(G_i - G_j) k_i.k_j (j < i),    N = (I + A diag(b))^-1 A    (strictly lower triangular, as A)
//     P_ij = scale e^(G_i - G_j) q_i.k_j (j <= i)
//     Y = V - diag(e^G) K S,   E = Y - N (b Y),   D = b E
//     O = scale diag(e^G) Q S + P D,   S_next = e^Gall S + K^T diag(e^(Gall - G)) D
// N and P do not depend on the state: they are made for all chunks side by side, and what runs from chunk
// to chunk is four products.  Writing the inverse as I - N diag(b) keeps its identity exact, and b = 0 harmless.
// Backward, dS: the gradient of the state behind the chunk:
//     dD = P^T dO + diag(e^(Gall - G)) K dS,   Z = dD - N^T (b dD),   dV = b Z,   dbeta_i = E_i.Z_i
//     dS_prev = e^Gall dS + scale Q^T diag(e^G) dO - K^T diag(e^G) dV
//     dA = -dV D^T,   dP = dO D^T (each where its matrix is not zero), and with L_ij = e^(G_i - G_j)
//     dQ = scale diag(e^G) dO S^T + (scale dP L) K
//     dK = diag(e^(Gall - G)) D dS^T - diag(e^G) dV S^T + (scale dP L)^T Q + (dA L) K + (dA L)^T K
//     dlog_decay_t = sum_{i >= t} (r_i + sum_j (M_ij - M_ji)) + sum_{j < t} w_j + e^Gall <S, dS>,   M = dP o P + dA o A (j < i)
//     r_i = e^G_i (scale q_i.(S dO_i) - k_i.(S dV_i)),   w_j = e^(Gall - G_j) k_j.(dS D_j)
// The last lines count what passes t, which is what a decay at t scales: what tokens from t on read and write over of the
// state before the chunk (r), what they have of tokens before t (M: the pairs behind t cancel), and what the state behind the
// chunk has of those (w) and of the state before it.  sum_{i >= t} (q_i.dq_i - v_i.dv_i) + <S_next, dS> is the same, but each
// token's own addition, which no decay touches, is in both terms and leaves its rounding error: in fp32, of a
// gradient 0.1% to 1% at log decays of -8, and 3% to 10% at -12.
// q and k stay as they are (exact as bf16 operands): 1 / |q| and 1 / |k| are part of the rows' factors and of A, P.
#pragma once

#include "retention.h"

namespace ssd {

constexpr int kDrC = 64;  // tokens of a chunk
constexpr uint32_t kDrTile = kDrC * kDrC * 2;  // bytes of a (64, 64) bf16 tile

// Factors of a chunk's rows.  Rows past the sequence's end have zeros.
struct alignas(16) DrRows {
  float kin[kDrC];   // e^G / |k|
  float kout[kDrC];  // e^(Gall - G) / |k|
  float qin[kDrC];   // scale e^G / |q|
  float beta[kDrC];
  float rk[kDrC], rq[kDrC];      // 1 / |k|, 1 / |q| (1 without qk_norm)
  float ghi[kDrC], glo[kDrC];    // G as a sum of two values
  float all_hi, all_lo, pad[2];  // e^Gall, likewise: a state is multiplied by it in every chunk that it lives
};
static_assert(sizeof(DrRows) % 16 == 0, "moved in units of 16 bytes");

struct DrProblem {
  int nseq, seqlen, total, H, Hk, group, dk, dv;
  int slots;      // places for chunks (dr_seq says where a sequence's start)
  const int *cu;  // or null: sequences of seqlen tokens
  const void *q, *k, *v, *g, *b;
  long long qs, ks, vs, gs, bs;  // token strides (elements)
  float scale, eps;
  int norm;
  const float *init;
  // tables, of chunk (slot, head) at slot * H + head
  DrRows *rows;
  float *N, *P, *A;  // CUDA cores: (64, 64) fp32, element (i, j) at 64 i + j; A for the gradients only, else null
  // backward: the states before the chunks and the gradients of those behind them (dk, dv), E and Z (total, H, dv).
  // Tensor cores: N's and P's two bf16 terms as four tiles of (64, 64) in the 128-byte swizzle, at N; E and Z are bf16,
  // and so are the states, at S and dS, in blocks of 8 columns: element (m, c) of (dk, dv), both padded to 64 or 128, at
  // (m / 8) 8 dv + 8 c + m % 8.
  float *S, *dS, *E, *Z;
  float *dqp, *dkp;  // (total, H, dk): gradients of the unit q and k of each state head
  // Tensor cores: sequences cut into segments of `seg` chunks (0: not cut), their places (dr_place0), the states before
  // them, and for all but last ones N, the state that a segment makes of zero, and M, so that S_next = M S + N (at
  // seg_sums: N of all places, then M)
  int seg, seg_places;
  float *seg_states, *seg_sums;
  int *status;       // device status word, cleared by the first kernel
  unsigned long long wait_ns;
};

// padded width of a state's side
__host__ __device__ __forceinline__ int dr_padded(int width) { return width <= 64 ? 64 : 128; }

__host__ __device__ __forceinline__ int dr_slots(long long rows, int nseq, int seqlen, bool packed) {
  return packed ? (int)(rows / kDrC) + nseq : nseq * ((seqlen + kDrC - 1) / kDrC);
}
// A sequence's rows, and the place of its first chunk.  Packed: ceil(len / 64) chunks fit between the places of
// sequences that start at a and a + len, a / 64 + s and (a + len) / 64 + s + 1, whatever the lengths are.
__device__ __forceinline__ void dr_seq(const DrProblem &p, int s, int &a, int &len, int &slot0) {
  if (p.cu) {
    a = min(max(__ldg(p.cu + s), 0), p.total);
    len = max(min(max(__ldg(p.cu + s + 1), 0), p.total) - a, 0);
    slot0 = a / kDrC + s;
  } else {
    a = s * p.seqlen;
    len = p.seqlen;
    slot0 = s * ((p.seqlen + kDrC - 1) / kDrC);
  }
}
// The rows of the chunk at a place: [t0, t0 + n), n = 0 where there is none
__device__ __forceinline__ void dr_chunk(const DrProblem &p, int slot, int &t0, int &n) {
  int a, len, slot0, s = 0;
  if (p.cu) {  // the last sequence whose place is not behind this one
    int lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (min(max(__ldg(p.cu + mid), 0), p.total) / kDrC + mid <= slot)
        lo = mid;
      else
        hi = mid - 1;
    }
    s = lo;
  } else {
    s = slot / ((p.seqlen + kDrC - 1) / kDrC);
  }
  dr_seq(p, s, a, len, slot0);
  const long long off = (long long)(slot - slot0) * kDrC;
  t0 = a + (int)(off < 0 || off > len ? len : off);
  n = off < 0 || off >= len ? 0 : min(kDrC, len - (int)off);
}

// The place of a sequence's first segment, as of its first chunk; and the segment at a place: seq < 0 where there is none
__device__ __forceinline__ int dr_place0(const DrProblem &p, int seg, int a, int s) {
  const int n = seg * kDrC;
  return p.cu ? a / n + s : s * ((p.seqlen + n - 1) / n);
}
__device__ __forceinline__ void dr_segment(const DrProblem &p, int seg, int place, int &seq, int &a, int &len, int &slot0, bool &ends) {
  const int n = seg * kDrC;
  if (p.cu) {
    int lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (min(max(__ldg(p.cu + mid), 0), p.total) / n + mid <= place)
        lo = mid;
      else
        hi = mid - 1;
    }
    seq = lo;
  } else {
    seq = place / ((p.seqlen + n - 1) / n);
  }
  dr_seq(p, seq, a, len, slot0);
  const long long off = (long long)(place - dr_place0(p, seg, a, seq)) * n;
  if (off < 0 || off >= len) {  // (empty sequences have no segment either: the scan sees to their states)
    seq = -1;
    return;
  }
  ends = off + n >= len;
  slot0 += (int)(off / kDrC);
  a += (int)off;
  len = min(n, len - (int)off);
}

// dr_prep.cu: rows' factors, N and P of every chunk
template <typename T> void launch_dr_prep(const DrProblem &p, cudaStream_t s);
// dr_prep_tc.cu: the same for the tensor-core chains
void launch_dr_prep_tc(const DrProblem &p, cudaStream_t s);
// dr_tc.cu: the chains for bf16, both widths at most 128
void launch_dr_tc_chain(const DrProblem &p, void *o, long long os, float *fin, cudaStream_t s);
// cut sequences: the segments' M and N, then the states before them, and the final ones of empty sequences
void launch_dr_tc_sums(const DrProblem &p, cudaStream_t s);
void launch_dr_tc_scan(const DrProblem &p, float *fin, cudaStream_t s);
void launch_dr_tc_reverse(const DrProblem &p, const void *dout, long long dos, const float *dfin, float *dinit, cudaStream_t s);
// dr_simt.cu: the chain of chunks (o null: only S and E, for backward), its reverse, and the gradients
template <typename T> void launch_dr_chain(const DrProblem &p, void *o, long long os, float *fin, cudaStream_t s);
template <typename T>
void launch_dr_reverse(const DrProblem &p, const void *dout, long long dos, const float *dfin, float *dinit, cudaStream_t s);
struct DrGrads {
  void *dq, *dk, *dv, *dg, *db;
  long long dqs, dks, dvs, dgs, dbs;
};
template <typename T>
void launch_dr_grads(const DrProblem &p, const void *dout, long long dos, const DrGrads &g, cudaStream_t s);
// dq and dk out of their parts: summed over the states that share a head, and through the division by the length
template <typename T> void launch_dr_finish(const DrProblem &p, const DrGrads &g, cudaStream_t s);
// dr_grads_tc.cu: all gradients of the tensor-core path
void launch_dr_grads_tc(const DrProblem &p, const void *dout, long long dos, const DrGrads &g, cudaStream_t s);
// dr_step.cu
template <typename T>
void launch_dr_step(const DrProblem &p, void *o, long long os, float *states, int nslots, const int *slot_idx, cudaStream_t s);

}  // namespace ssd
