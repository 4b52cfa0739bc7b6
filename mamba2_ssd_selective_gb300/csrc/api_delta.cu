// C ABI of the gated delta rule and of the norms around a block: argument checks, workspace carving and launch
// sequences.  Nothing here allocates or synchronises.
#include <cmath>

#include "block_norm.h"
#include "delta.h"

using namespace ssd;

namespace {

// two of these outputs that start at the same place, or one where one of the inputs does
bool outputs_meet(std::initializer_list<const void *> outputs, std::initializer_list<const void *> inputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    if (on_input(*o, inputs)) return true;
    for (auto other = outputs.begin(); other != o; ++other)
      if (*o && *o == *other) return true;
  }
  return false;
}

// ---------------------------------------------------------------- gated delta rule

struct DrPlan {
  bool tc;
  int slots, seg, places;  // seg: chunks of a segment, 0: sequences are not cut
  size_t seg_states, seg_sums, status, rows, N, P, A, S, dS, E, Z, dqp, dkp, total;  // workspace offsets
};

long long dr_rows(const ssd_delta_rule_dims *d) { return d->packed ? d->total_tokens : (long long)d->nseq * d->seqlen; }

ssd_status dr_check_dims(const ssd_delta_rule_dims *d) {
  if (!d) return SSD_ERR_NULL_PTR;
  if (d->nseq <= 0 || d->nheads <= 0 || d->nheads_qk <= 0 || d->headdim_k <= 0 || d->headdim_v <= 0 ||
      (d->packed != 0 && d->packed != 1) || (d->qk_norm != 0 && d->qk_norm != 1) || d->nheads % d->nheads_qk)
    return SSD_ERR_INVALID_DIMS;
  if (d->packed ? d->total_tokens <= 0 : d->seqlen <= 0) return SSD_ERR_INVALID_DIMS;
  if (d->dtype != SSD_BF16 && d->dtype != SSD_F32) return SSD_ERR_DTYPE;
  const long long rows = dr_rows(d);
  if (!d->packed && d->total_tokens != 0 && d->total_tokens != rows) return SSD_ERR_INVALID_DIMS;
  if (d->headdim_k % 8 || d->headdim_v % 8 || d->headdim_k > 256 || d->headdim_v > 256 || rows > kMaxRows ||
      d->nseq > kMaxSeqs || (long long)d->nseq * d->nheads > (1LL << 28) ||
      (long long)d->nheads * d->headdim_k > kMaxChannels || (long long)d->nheads * d->headdim_v > kMaxChannels)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

// bf16 within its widths takes the tensor-core kernels, everything else the CUDA-core ones
bool dr_use_tc(const ssd_delta_rule_dims *d) { return d->dtype == SSD_BF16 && la_tc_envelope(d->headdim_k, d->headdim_v); }

// Chunks of a segment, or 0: whether sequences are cut is a matter of their number, since a chain is an SM's however few
// there are.  Times measured here with states of 128 x 128 (and taken for narrower ones too), in us: a chunk of a chain 2.7,
// a chunk of a segment's sums 2.4 (there are two, for all segments but the last), the scan 4 a segment, two launches more
// 12.  Lengths of packed sequences are not known: the longest of n is taken for its mean where sequences end at random.  (A
// workspace's size may be asked for where there is no GPU: the SMs are not asked.)
int dr_segment_chunks(const ssd_delta_rule_dims *d) {
  const long long sms = 152, items = (long long)d->nseq * d->nheads, n = d->nseq;
  const double part = d->packed ? (std::log((double)n) + 0.577 + 0.5 / (double)n) / (double)n : 1.;
  const long long chunks = (long long)((double)(d->packed ? d->total_tokens : d->seqlen) * (part < 1. ? part : 1.) / kDrC) + 1;
  auto rounds = [&](long long x) { return (double)((x + sms - 1) / sms); };
  double best = rounds(items) * 2.7 * (double)chunks;
  int seg = 0;
  for (long long k = 2; k <= 64 && 4 * k <= chunks; ++k) {
    const long long len = (chunks + k - 1) / k;
    const double cost = rounds(2 * items * (k - 1)) * 2.4 * (double)len + rounds(items * k) * 2.7 * (double)len + 4. * (double)k + 12.;
    if (cost < best) {
      best = cost;
      seg = (int)len;
    }
  }
  return seg;
}

DrPlan dr_plan(const ssd_delta_rule_dims *d, bool backward) {
  DrPlan pl{};
  pl.tc = dr_use_tc(d);
  pl.slots = dr_slots(dr_rows(d), d->nseq, d->seqlen, d->packed != 0);
  const size_t chunks = (size_t)pl.slots * d->nheads, state = (size_t)d->headdim_k * d->headdim_v,
               tokens = (size_t)dr_rows(d) * d->nheads;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  pl.status = take(256);
  pl.rows = take(chunks * sizeof(DrRows));
  pl.N = take(chunks * (pl.tc ? 4 * kDrTile : kDrC * kDrC * 4));
  pl.P = take(pl.tc ? 0 : chunks * kDrC * kDrC * 4);
  if (pl.tc && !backward) pl.seg = dr_segment_chunks(d);
  if (pl.seg) {
    const long long n = (long long)pl.seg * kDrC, rows = dr_rows(d);
    pl.places = (int)(d->packed ? rows / n + d->nseq : d->nseq * ((d->seqlen + n - 1) / n));
    const size_t items = (size_t)pl.places * d->nheads;
    pl.seg_states = take(items * state * 4);
    pl.seg_sums = take(items * (state + (size_t)d->headdim_k * d->headdim_k) * 4);
  }
  if (backward) {
    const size_t eb = pl.tc ? 2 : 4, padded = (size_t)dr_padded(d->headdim_k) * dr_padded(d->headdim_v);
    pl.S = take(chunks * (pl.tc ? padded * 2 : state * 4));
    pl.dS = take(chunks * (pl.tc ? padded * 2 : state * 4));
    pl.E = take(tokens * d->headdim_v * eb);
    pl.Z = take(tokens * d->headdim_v * eb);
    pl.dqp = take(pl.tc ? 0 : tokens * d->headdim_k * 4);
    pl.dkp = take(pl.tc ? 0 : tokens * d->headdim_k * 4);
    pl.A = take(pl.tc ? 0 : chunks * kDrC * kDrC * 4);
  }
  pl.total = off;
  return pl;
}

// a (T, width) tensor of the activation type, 16-byte aligned rows
ssd_status dr_check_rows(const ssd_delta_rule_dims *d, const void *p, int64_t stride, long long width) {
  if (!p) return SSD_ERR_NULL_PTR;
  if (stride < width) return SSD_ERR_INVALID_DIMS;
  return aligned(p, 16) && stride % (16 / elem_bytes(d->dtype)) == 0 ? SSD_OK : SSD_ERR_ALIGNMENT;
}
// a (T, nheads) tensor: one number for each head
ssd_status dr_check_numbers(const ssd_delta_rule_dims *d, const void *p, int64_t stride) {
  if (!p) return SSD_ERR_NULL_PTR;
  if (stride < d->nheads) return SSD_ERR_INVALID_DIMS;
  return aligned(p, elem_bytes(d->dtype)) ? SSD_OK : SSD_ERR_ALIGNMENT;
}

ssd_status dr_check_inputs(const ssd_delta_rule_dims *d, const ssd_delta_rule_inputs *in) {
  if (!in) return SSD_ERR_NULL_PTR;
  const long long qk = (long long)d->nheads_qk * d->headdim_k;
  ssd_status st = dr_check_rows(d, in->q, in->q_tok_stride, qk);
  if (st == SSD_OK) st = dr_check_rows(d, in->k, in->k_tok_stride, qk);
  if (st == SSD_OK) st = dr_check_rows(d, in->v, in->v_tok_stride, (long long)d->nheads * d->headdim_v);
  if (st == SSD_OK) st = dr_check_numbers(d, in->log_decay, in->log_decay_tok_stride);
  if (st == SSD_OK) st = dr_check_numbers(d, in->beta, in->beta_tok_stride);
  if (st != SSD_OK) return st;
  if (d->packed && !in->cu_seqlens) return SSD_ERR_NULL_PTR;
  if (!d->packed && in->cu_seqlens) return SSD_ERR_INVALID_DIMS;  // would be ignored: rejected instead
  if (!(in->scale > -1e30f && in->scale < 1e30f)) return SSD_ERR_INVALID_DIMS;
  if (d->qk_norm && !(in->norm_eps >= 0.f && in->norm_eps < 1e30f)) return SSD_ERR_INVALID_DIMS;
  return aligned(in->initial_states, 16) && aligned(in->cu_seqlens, 4) ? SSD_OK : SSD_ERR_ALIGNMENT;
}

ssd_status dr_check_workspace(const DrPlan &pl, const void *ws, size_t bytes) {
  if (!ws || bytes < pl.total) return SSD_ERR_WORKSPACE;
  return aligned(ws, 256) ? SSD_OK : SSD_ERR_ALIGNMENT;
}

// what a call of any kind has; the tables and a backward pass's buffers where there is a workspace
DrProblem dr_problem(const ssd_delta_rule_dims *d, const ssd_delta_rule_inputs *in, const DrPlan *pl, char *ws) {
  DrProblem p{};
  p.nseq = d->nseq;
  p.seqlen = d->seqlen;
  p.total = (int)dr_rows(d);
  p.H = d->nheads;
  p.Hk = d->nheads_qk;
  p.group = d->nheads / d->nheads_qk;
  p.dk = d->headdim_k;
  p.dv = d->headdim_v;
  p.cu = in->cu_seqlens;
  p.q = in->q, p.qs = in->q_tok_stride;
  p.k = in->k, p.ks = in->k_tok_stride;
  p.v = in->v, p.vs = in->v_tok_stride;
  p.g = in->log_decay, p.gs = in->log_decay_tok_stride;
  p.b = in->beta, p.bs = in->beta_tok_stride;
  p.scale = in->scale;
  p.eps = in->norm_eps;
  p.norm = d->qk_norm;
  p.init = in->initial_states;
  if (pl) {
    p.slots = pl->slots;
    p.status = reinterpret_cast<int *>(ws + pl->status);
    p.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
    p.rows = reinterpret_cast<DrRows *>(ws + pl->rows);
    auto at = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    p.N = at(pl->N), p.P = at(pl->P);
    p.seg = pl->seg, p.seg_places = pl->places;
    p.seg_states = at(pl->seg_states), p.seg_sums = at(pl->seg_sums);
    p.S = at(pl->S), p.dS = at(pl->dS), p.E = at(pl->E), p.Z = at(pl->Z);
    p.dqp = at(pl->dqp), p.dkp = at(pl->dkp);
    p.A = pl->A ? at(pl->A) : nullptr;
  }
  return p;
}

template <typename T>
ssd_status dr_forward_impl(const DrProblem &p, bool tc, void *o, int64_t os, float *fin, cudaStream_t s) {
  SSD_LAUNCH("dr_prep", tc ? launch_dr_prep_tc(p, s) : launch_dr_prep<T>(p, s));
  if (p.seg) {
    SSD_LAUNCH("dr_sums", launch_dr_tc_sums(p, s));
    SSD_LAUNCH("dr_scan", launch_dr_tc_scan(p, fin, s));
  }
  SSD_LAUNCH("dr_chain", tc ? launch_dr_tc_chain(p, o, os, fin, s) : launch_dr_chain<T>(p, o, os, fin, s));
  return launch_status();
}

template <typename T>
ssd_status dr_backward_impl(const DrProblem &p, bool tc, const void *dout, int64_t dos, const float *dfin,
                            const ssd_delta_rule_grads *g, cudaStream_t s) {
  const DrGrads out{g->dq, g->dk, g->dv, g->dlog_decay, g->dbeta, g->dq_tok_stride, g->dk_tok_stride, g->dv_tok_stride,
                    g->dlog_decay_tok_stride, g->dbeta_tok_stride};
  if (tc) {
    SSD_LAUNCH("dr_prep", launch_dr_prep_tc(p, s));
    SSD_LAUNCH("dr_chain", launch_dr_tc_chain(p, nullptr, 0, nullptr, s));
    SSD_LAUNCH("dr_reverse", launch_dr_tc_reverse(p, dout, dos, dfin, g->dinitial_states, s));
    SSD_LAUNCH("dr_grads", launch_dr_grads_tc(p, dout, dos, out, s));
  } else {
    SSD_LAUNCH("dr_prep", launch_dr_prep<T>(p, s));
    SSD_LAUNCH("dr_chain", launch_dr_chain<T>(p, nullptr, 0, nullptr, s));
    SSD_LAUNCH("dr_reverse", launch_dr_reverse<T>(p, dout, dos, dfin, g->dinitial_states, s));
    SSD_LAUNCH("dr_grads", launch_dr_grads<T>(p, dout, dos, out, s));
    SSD_LAUNCH("dr_finish", launch_dr_finish<T>(p, out, s));
  }
  return launch_status();
}

// ---------------------------------------------------------------- block norm

bool flag(int32_t x) { return x == 0 || x == 1; }

ssd_status bn_check_dims(const ssd_block_norm_dims *d) {
  if (!d) return SSD_ERR_NULL_PTR;
  if (d->rows <= 0 || d->channels <= 0 || !flag(d->post_norm) || !flag(d->gate) || !flag(d->residual) || !flag(d->pre_norm))
    return SSD_ERR_INVALID_DIMS;
  if ((d->dtype != SSD_BF16 && d->dtype != SSD_F32) || (d->residual_dtype != d->dtype && d->residual_dtype != SSD_F32))
    return SSD_ERR_DTYPE;
  if (d->rows > kMaxRows || d->channels > kBnMaxChannels) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

// Rows of a tensor, and how many channels the tensors so far allow at once: 8 (16 bytes of bf16, twice 16 of fp32), 2 or 1
ssd_status bn_check_rows(const ssd_block_norm_dims *d, int dtype, const void *p, int64_t stride, int &vec) {
  if (!p) return SSD_ERR_NULL_PTR;
  if (stride < d->channels) return SSD_ERR_INVALID_DIMS;
  if (stride > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype);
  if (!aligned(p, eb)) return SSD_ERR_ALIGNMENT;
  const int w = aligned(p, 16) && stride % 8 == 0 ? 8 : aligned(p, 2 * eb) && stride % 2 == 0 ? 2 : 1;
  if (w < vec) vec = w;
  return SSD_OK;
}
// the same for a tensor that is there exactly with its flag
ssd_status bn_check_with(const ssd_block_norm_dims *d, bool with, int dtype, const void *p, int64_t stride, int &vec) {
  if (with) return bn_check_rows(d, dtype, p, stride, vec);
  return p ? SSD_ERR_INVALID_DIMS : SSD_OK;  // would be ignored: rejected instead
}
int bn_vec(const ssd_block_norm_dims *d) { return d->channels % 8 == 0 ? 8 : d->channels % 2 == 0 ? 2 : 1; }

ssd_status bn_check_inputs(const ssd_block_norm_dims *d, const ssd_block_norm_inputs *in, bool backward, int &vec) {
  if (!in) return SSD_ERR_NULL_PTR;
  ssd_status st = bn_check_rows(d, d->dtype, in->x, in->x_row_stride, vec);
  if (st == SSD_OK) st = bn_check_with(d, d->gate, d->dtype, in->z, in->z_row_stride, vec);
  if (st == SSD_OK)
    st = bn_check_with(d, d->residual && !backward, d->residual_dtype, in->residual, in->residual_row_stride, vec);
  if (st != SSD_OK) return st;
  if ((in->post_weight && !d->post_norm) || (in->pre_weight && !d->pre_norm)) return SSD_ERR_INVALID_DIMS;
  if (!aligned(in->post_weight, 4) || !aligned(in->branch_scale, 4) || !aligned(in->pre_weight, 4)) return SSD_ERR_ALIGNMENT;
  return in->eps >= 0.f && in->eps < 1e30f ? SSD_OK : SSD_ERR_INVALID_DIMS;
}

BnProblem bn_problem(const ssd_block_norm_dims *d, const ssd_block_norm_inputs *in) {
  BnProblem p{};
  p.rows = d->rows;
  p.C = d->channels;
  p.post = d->post_norm;
  p.gate = d->gate;
  p.pre = d->pre_norm;
  p.x = in->x, p.xs = in->x_row_stride;
  p.z = in->z, p.zs = in->z_row_stride;
  p.res = in->residual, p.rs = in->residual_row_stride;
  p.pw = in->post_weight;
  p.sc = in->branch_scale;
  p.w = in->pre_weight;
  p.eps = in->eps;
  return p;
}

}  // namespace

extern "C" {

size_t ssd_delta_rule_workspace_size(const ssd_delta_rule_dims *dims, int backward) {
  if (dr_check_dims(dims) != SSD_OK) return 0;
  return dr_plan(dims, backward != 0).total;
}

ssd_status ssd_delta_rule_forward(const ssd_delta_rule_dims *dims, const ssd_delta_rule_inputs *in, void *o,
                                  int64_t o_tok_stride, float *final_states, void *workspace, size_t ws_bytes,
                                  ssd_stream_t stream) {
  ssd_status st = dr_check_dims(dims);
  if (st == SSD_OK) st = dr_check_inputs(dims, in);
  if (st == SSD_OK) st = dr_check_rows(dims, o, o_tok_stride, (long long)dims->nheads * dims->headdim_v);
  if (st != SSD_OK) return st;
  if (!aligned(final_states, 16)) return SSD_ERR_ALIGNMENT;
  const DrPlan pl = dr_plan(dims, false);
  st = dr_check_workspace(pl, workspace, ws_bytes);
  if (st != SSD_OK) return st;
  if (outputs_meet({o, final_states}, {in->q, in->k, in->v, in->log_decay, in->beta, in->cu_seqlens}) ||
      on_input(o, {in->initial_states}))
    return SSD_ERR_INVALID_DIMS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const DrProblem p = dr_problem(dims, in, &pl, static_cast<char *>(workspace));
  return dims->dtype == SSD_BF16 ? dr_forward_impl<__nv_bfloat16>(p, pl.tc, o, o_tok_stride, final_states, s)
                                 : dr_forward_impl<float>(p, pl.tc, o, o_tok_stride, final_states, s);
}

ssd_status ssd_delta_rule_backward(const ssd_delta_rule_dims *dims, const ssd_delta_rule_inputs *in, const void *dout,
                                   int64_t dout_tok_stride, const float *dfinal_states,
                                   const ssd_delta_rule_grads *grads, void *workspace, size_t ws_bytes,
                                   ssd_stream_t stream) {
  ssd_status st = dr_check_dims(dims);
  if (st == SSD_OK) st = dr_check_inputs(dims, in);
  if (st != SSD_OK) return st;
  const long long qk = (long long)dims->nheads_qk * dims->headdim_k, hv = (long long)dims->nheads * dims->headdim_v;
  if (!grads) return SSD_ERR_NULL_PTR;
  st = dr_check_rows(dims, dout, dout_tok_stride, hv);
  if (st == SSD_OK) st = dr_check_rows(dims, grads->dq, grads->dq_tok_stride, qk);
  if (st == SSD_OK) st = dr_check_rows(dims, grads->dk, grads->dk_tok_stride, qk);
  if (st == SSD_OK) st = dr_check_rows(dims, grads->dv, grads->dv_tok_stride, hv);
  if (st == SSD_OK) st = dr_check_numbers(dims, grads->dlog_decay, grads->dlog_decay_tok_stride);
  if (st == SSD_OK) st = dr_check_numbers(dims, grads->dbeta, grads->dbeta_tok_stride);
  if (st != SSD_OK) return st;
  if (!aligned(dfinal_states, 16) || !aligned(grads->dinitial_states, 16)) return SSD_ERR_ALIGNMENT;
  const DrPlan pl = dr_plan(dims, true);
  st = dr_check_workspace(pl, workspace, ws_bytes);
  if (st != SSD_OK) return st;
  if (outputs_meet({grads->dq, grads->dk, grads->dv, grads->dlog_decay, grads->dbeta, grads->dinitial_states},
                   {in->q, in->k, in->v, in->log_decay, in->beta, in->initial_states, in->cu_seqlens, dout, dfinal_states}))
    return SSD_ERR_INVALID_DIMS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const DrProblem p = dr_problem(dims, in, &pl, static_cast<char *>(workspace));
  return dims->dtype == SSD_BF16 ? dr_backward_impl<__nv_bfloat16>(p, pl.tc, dout, dout_tok_stride, dfinal_states, grads, s)
                                 : dr_backward_impl<float>(p, pl.tc, dout, dout_tok_stride, dfinal_states, grads, s);
}

ssd_status ssd_delta_rule_step(const ssd_delta_rule_dims *dims, const ssd_delta_rule_inputs *in, float *states,
                               int32_t nslots, const int32_t *slot_idx, void *o, int64_t o_tok_stride,
                               ssd_stream_t stream) {
  ssd_status st = dr_check_dims(dims);
  if (st != SSD_OK) return st;
  if (dims->packed || dims->seqlen != 1) return SSD_ERR_INVALID_DIMS;
  st = dr_check_inputs(dims, in);
  if (st == SSD_OK) st = dr_check_rows(dims, o, o_tok_stride, (long long)dims->nheads * dims->headdim_v);
  if (st != SSD_OK) return st;
  if (in->initial_states) return SSD_ERR_INVALID_DIMS;  // the cache is the state
  if (!states) return SSD_ERR_NULL_PTR;
  if (nslots <= 0) return SSD_ERR_INVALID_DIMS;
  if (!aligned(states, 16) || !aligned(slot_idx, 4)) return SSD_ERR_ALIGNMENT;
  if (outputs_meet({o, states}, {in->q, in->k, in->v, in->log_decay, in->beta, slot_idx})) return SSD_ERR_INVALID_DIMS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const DrProblem p = dr_problem(dims, in, nullptr, nullptr);
  if (dims->dtype == SSD_BF16)
    SSD_LAUNCH("dr_step", launch_dr_step<__nv_bfloat16>(p, o, o_tok_stride, states, nslots, slot_idx, s));
  else
    SSD_LAUNCH("dr_step", launch_dr_step<float>(p, o, o_tok_stride, states, nslots, slot_idx, s));
  return launch_status();
}

size_t ssd_block_norm_workspace_size(const ssd_block_norm_dims *dims) {
  if (bn_check_dims(dims) != SSD_OK) return 0;
  return align_up((size_t)bn_blocks(dims->rows, dims->channels, 8) * 3 * dims->channels * 4, 256);
}

ssd_status ssd_block_norm_forward(const ssd_block_norm_dims *dims, const ssd_block_norm_inputs *in, void *h,
                                  int64_t h_row_stride, void *y, int64_t y_row_stride, float *rstd_post,
                                  float *rstd_pre, ssd_stream_t stream) {
  ssd_status st = bn_check_dims(dims);
  if (st != SSD_OK) return st;
  int vec = bn_vec(dims);
  st = bn_check_inputs(dims, in, false, vec);
  if (st == SSD_OK && (h || !dims->pre_norm)) st = bn_check_rows(dims, dims->residual_dtype, h, h_row_stride, vec);
  if (st == SSD_OK) st = bn_check_with(dims, dims->pre_norm, dims->dtype, y, y_row_stride, vec);
  if (st != SSD_OK) return st;
  if ((rstd_post && !dims->post_norm) || (rstd_pre && !dims->pre_norm)) return SSD_ERR_INVALID_DIMS;
  if (!aligned(rstd_post, 4) || !aligned(rstd_pre, 4)) return SSD_ERR_ALIGNMENT;
  if (outputs_meet({h, y, rstd_post, rstd_pre}, {in->x, in->z, in->post_weight, in->branch_scale, in->pre_weight}) ||
      outputs_meet({y, rstd_post, rstd_pre}, {in->residual}) ||
      (h && h == in->residual && h_row_stride != in->residual_row_stride))
    return SSD_ERR_INVALID_DIMS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  BnProblem p = bn_problem(dims, in);
  p.h = h, p.hs = h_row_stride;
  p.y = y, p.ys = y_row_stride;
  p.rstd_post = rstd_post;
  p.rstd_pre = rstd_pre;
  if (dims->dtype == SSD_F32)
    SSD_LAUNCH("bn_forward", (launch_bn_forward<float, float>(p, vec, s)));
  else if (dims->residual_dtype == SSD_F32)
    SSD_LAUNCH("bn_forward", (launch_bn_forward<__nv_bfloat16, float>(p, vec, s)));
  else
    SSD_LAUNCH("bn_forward", (launch_bn_forward<__nv_bfloat16, __nv_bfloat16>(p, vec, s)));
  return launch_status();
}

ssd_status ssd_block_norm_backward(const ssd_block_norm_dims *dims, const ssd_block_norm_inputs *in,
                                   const ssd_block_norm_saved *saved, const ssd_block_norm_grads *grads,
                                   void *workspace, size_t ws_bytes, ssd_stream_t stream) {
  ssd_status st = bn_check_dims(dims);
  if (st != SSD_OK) return st;
  int vec = bn_vec(dims);
  st = bn_check_inputs(dims, in, true, vec);
  if (st != SSD_OK) return st;
  if (!saved || !grads) return SSD_ERR_NULL_PTR;
  st = bn_check_with(dims, dims->pre_norm, dims->residual_dtype, saved->h, saved->h_row_stride, vec);
  if (st == SSD_OK) st = bn_check_with(dims, dims->pre_norm, dims->dtype, saved->dy, saved->dy_row_stride, vec);
  if (st == SSD_OK && saved->dh) st = bn_check_rows(dims, dims->residual_dtype, saved->dh, saved->dh_row_stride, vec);
  if (st == SSD_OK) st = bn_check_rows(dims, dims->dtype, grads->dx, grads->dx_row_stride, vec);
  if (st == SSD_OK) st = bn_check_with(dims, dims->gate, dims->dtype, grads->dz, grads->dz_row_stride, vec);
  if (st == SSD_OK)
    st = bn_check_with(dims, dims->residual, dims->residual_dtype, grads->dresidual, grads->dresidual_row_stride, vec);
  if (st != SSD_OK) return st;
  if ((dims->post_norm && !saved->rstd_post) || (dims->pre_norm && !saved->rstd_pre)) return SSD_ERR_NULL_PTR;
  if ((grads->dpost_weight && !dims->post_norm) || (grads->dpre_weight && !dims->pre_norm)) return SSD_ERR_INVALID_DIMS;
  for (const void *q : {(const void *)saved->rstd_post, (const void *)saved->rstd_pre, (const void *)grads->dpost_weight,
                        (const void *)grads->dbranch_scale, (const void *)grads->dpre_weight})
    if (!aligned(q, 4)) return SSD_ERR_ALIGNMENT;
  if (!workspace || ws_bytes < ssd_block_norm_workspace_size(dims)) return SSD_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SSD_ERR_ALIGNMENT;
  // (the parameters' sums are written when everything has been read)
  if (outputs_meet({grads->dx, grads->dz, grads->dresidual},
                   {in->x, in->z, in->post_weight, in->branch_scale, in->pre_weight, saved->h, saved->dy, saved->rstd_post,
                    saved->rstd_pre}) ||
      outputs_meet({grads->dx, grads->dz, grads->dresidual, grads->dpost_weight, grads->dbranch_scale, grads->dpre_weight}, {}) ||
      on_input(saved->dh, {grads->dx, grads->dz}) ||
      (on_input(saved->dh, {grads->dresidual}) && saved->dh_row_stride != grads->dresidual_row_stride))
    return SSD_ERR_INVALID_DIMS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  BnProblem p = bn_problem(dims, in);
  p.h = const_cast<void *>(saved->h), p.hs = saved->h_row_stride;
  p.dh = saved->dh, p.dhs = saved->dh_row_stride;
  p.dy = saved->dy, p.dys = saved->dy_row_stride;
  p.rstd_post = const_cast<float *>(saved->rstd_post);
  p.rstd_pre = const_cast<float *>(saved->rstd_pre);
  p.dx = grads->dx, p.dxs = grads->dx_row_stride;
  p.dz = grads->dz, p.dzs = grads->dz_row_stride;
  p.dres = grads->dresidual, p.drs = grads->dresidual_row_stride;
  p.dpw = grads->dpost_weight;
  p.dsc = grads->dbranch_scale;
  p.dw = grads->dpre_weight;
  p.part = static_cast<float *>(workspace);
  if (dims->dtype == SSD_F32)
    SSD_LAUNCH("bn_backward", (launch_bn_backward<float, float>(p, vec, s)));
  else if (dims->residual_dtype == SSD_F32)
    SSD_LAUNCH("bn_backward", (launch_bn_backward<__nv_bfloat16, float>(p, vec, s)));
  else
    SSD_LAUNCH("bn_backward", (launch_bn_backward<__nv_bfloat16, __nv_bfloat16>(p, vec, s)));
  if (p.dpw || p.dsc || p.dw) SSD_LAUNCH("bn_sums", launch_bn_sums(p, vec, s));
  return launch_status();
}

}  // extern "C"
