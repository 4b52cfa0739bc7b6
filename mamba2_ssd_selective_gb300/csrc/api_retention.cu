// C ABI of linear attention with a decay for each head and of group norm with
// an activation: argument checks, workspace carving and launch sequences.
// Nothing here allocates or synchronises.
#include "group_norm.h"
#include "retention.h"

using namespace ssd;

namespace {

constexpr long long kMaxRows = 1LL << 30, kMaxChannels = 1 << 16;
constexpr int kMaxSeqs = 1 << 20;

// ---------------------------------------------------------------- linear attention

struct LaPlan {
  bool split;
  int seg_len, nunits;
  size_t status, seg, part, total;  // workspace offsets
};

long long la_rows(const ssd_linear_attn_dims *d) {
  return d->packed ? d->total_tokens : (long long)d->nseq * d->seqlen;
}

ssd_status la_check_dims(const ssd_linear_attn_dims *d) {
  if (!d) return SSD_ERR_NULL_PTR;
  if (d->nseq <= 0 || d->nheads <= 0 || d->nheads_kv <= 0 || d->headdim_k <= 0 || d->headdim_v <= 0 ||
      (d->packed != 0 && d->packed != 1) || d->nheads % d->nheads_kv)
    return SSD_ERR_INVALID_DIMS;
  if (d->packed ? d->total_tokens <= 0 : d->seqlen <= 0) return SSD_ERR_INVALID_DIMS;
  if (d->dtype != SSD_BF16 && d->dtype != SSD_F32) return SSD_ERR_DTYPE;
  const long long rows = la_rows(d);
  if (!d->packed && d->total_tokens != 0 && d->total_tokens != rows) return SSD_ERR_INVALID_DIMS;
  if (d->headdim_k % 8 || d->headdim_v % 8 || d->headdim_k > 256 || d->headdim_v > 256 || rows > kMaxRows ||
      d->nseq > kMaxSeqs || (long long)d->nseq * d->nheads > (1LL << 30) || (long long)d->nheads * d->headdim_k > kMaxChannels ||
      (long long)d->nheads * d->headdim_v > kMaxChannels)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

// bf16 within its widths takes the tensor-core kernel, everything else the CUDA-core one
bool la_use_tc(const ssd_linear_attn_dims *d) {
  return d->dtype == SSD_BF16 && la_tc_envelope(d->headdim_k, d->headdim_v);
}

// Whether and where sequences are cut, and the workspace.  A cut sequence costs
// a second read of k and v (the segments' own states) and two more launches, so
// it is only made when whole sequences leave most of the GPU without work.
LaPlan la_plan(const ssd_linear_attn_dims *d, bool backward) {
  LaPlan pl{};
  const bool tc = la_use_tc(d);
  const long long rows = la_rows(d), H = d->nheads, sms = 152;
  // blocks of a whole sequence, and blocks that fill the GPU (one or four on an SM)
  const long long blocks = H * (tc ? 1 : (d->headdim_v + 63) / 64), want = tc ? sms : 4 * sms;
  const long long longest = d->packed ? rows : d->seqlen;
  const long long cuts = want / (d->nseq * blocks);
  long long seg = d->packed ? rows * blocks / want : cuts > 0 ? (longest + cuts - 1) / cuts : longest;
  seg = (seg + 63) / 64 * 64;
  if (seg < 256) seg = 256;
  pl.split = seg < longest && cuts >= 2;
  if (!pl.split) seg = (longest + 63) / 64 * 64;
  pl.seg_len = (int)seg;
  pl.nunits = (int)(!pl.split ? d->nseq : d->packed ? rows / seg + d->nseq : d->nseq * ((longest + seg - 1) / seg));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  pl.status = take(256);
  pl.seg = take(pl.split ? (size_t)pl.nunits * H * d->headdim_k * d->headdim_v * 4 : 0);
  const int wide = d->headdim_k > d->headdim_v ? d->headdim_k : d->headdim_v;
  pl.part = take(backward && d->nheads != d->nheads_kv ? (size_t)rows * H * wide * 4 : 0);
  pl.total = off;
  return pl;
}

ssd_status la_check_inputs(const ssd_linear_attn_dims *d, const ssd_linear_attn_inputs *in) {
  if (!in) return SSD_ERR_NULL_PTR;
  if (!in->q || !in->k || !in->v || !in->log_decay || (d->packed && !in->cu_seqlens)) return SSD_ERR_NULL_PTR;
  if (!d->packed && in->cu_seqlens) return SSD_ERR_INVALID_DIMS;  // would be ignored: rejected instead
  const long long vec = 16 / elem_bytes(d->dtype);
  if (in->q_tok_stride < (long long)d->nheads * d->headdim_k ||
      in->k_tok_stride < (long long)d->nheads_kv * d->headdim_k ||
      in->v_tok_stride < (long long)d->nheads_kv * d->headdim_v)
    return SSD_ERR_INVALID_DIMS;
  if (!(in->scale > -1e30f && in->scale < 1e30f)) return SSD_ERR_INVALID_DIMS;
  if (!aligned(in->q, 16) || !aligned(in->k, 16) || !aligned(in->v, 16) || in->q_tok_stride % vec ||
      in->k_tok_stride % vec || in->v_tok_stride % vec || !aligned(in->log_decay, 4) ||
      !aligned(in->initial_states, 16) || !aligned(in->cu_seqlens, 4))
    return SSD_ERR_ALIGNMENT;
  return SSD_OK;
}

// a (T, heads * width) tensor of the activation type with its own token stride
ssd_status la_check_rows(const ssd_linear_attn_dims *d, const void *p, int64_t stride, long long width) {
  if (!p) return SSD_ERR_NULL_PTR;
  if (stride < width) return SSD_ERR_INVALID_DIMS;
  return aligned(p, 16) && stride % (16 / elem_bytes(d->dtype)) == 0 ? SSD_OK : SSD_ERR_ALIGNMENT;
}

ssd_status la_check_workspace(const LaPlan &pl, const void *ws, size_t bytes) {
  if (!ws || bytes < pl.total) return SSD_ERR_WORKSPACE;
  return aligned(ws, 256) ? SSD_OK : SSD_ERR_ALIGNMENT;
}

// what every pass of a call has in common
LaPass la_base(const ssd_linear_attn_dims *d, const ssd_linear_attn_inputs *in, const LaPlan &pl, char *ws) {
  LaPass p{};
  p.H = d->nheads;
  p.g = in->log_decay;
  p.nseq = d->nseq;
  p.seqlen = d->seqlen;
  p.total = (int)la_rows(d);
  p.cu = in->cu_seqlens;
  p.seg_len = pl.seg_len;
  p.nunits = pl.nunits;
  p.split = pl.split;
  p.seg_state = ws ? reinterpret_cast<float *>(ws + pl.seg) : nullptr;
  p.status = ws ? reinterpret_cast<int *>(ws + pl.status) : nullptr;
  p.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  return p;
}

// one role's tensor: its rows, the query heads that share a head, its heads
struct Role {
  const void *p;
  long long stride;
  int group, heads;
};
void la_roles(LaPass &p, const Role &q, const Role &k, const Role &v, int dk, int dv) {
  p.q = q.p;
  p.qs = q.stride;
  p.gq = q.group;
  p.Hq = q.heads;
  p.k = k.p;
  p.ks = k.stride;
  p.gk = k.group;
  p.Hk = k.heads;
  p.v = v.p;
  p.vs = v.stride;
  p.gv = v.group;
  p.Hv = v.heads;
  p.dk = dk;
  p.dv = dv;
}
// states of the pass: element (a, b) of the user's state, or of its transpose
void la_states(LaPass &p, const float *init, float *fin, bool transposed) {
  p.init = init;
  p.fin = fin;
  p.sa = transposed ? 1 : p.dv;
  p.sb = transposed ? p.dk : 1;
}

template <typename T>
void la_run(const LaPass &p, bool reverse, cudaStream_t s) {
  const bool tc = sizeof(T) == 2 && la_tc_envelope(p.dk, p.dv);
  auto pass = [&](bool summary) { tc ? launch_la_tc(p, reverse, summary, s) : launch_la_simt<T>(p, reverse, summary, s); };
  if (p.split) {
    SSD_LAUNCH("la_segment_states", pass(true));
    SSD_LAUNCH("la_scan", launch_la_scan(p, reverse, s));
  }
  SSD_LAUNCH("la_pass", pass(false));
}

template <typename T>
ssd_status la_backward_impl(const ssd_linear_attn_dims *d, const ssd_linear_attn_inputs *in, const void *dout,
                            int64_t dout_stride, const float *dfinal, const ssd_linear_attn_grads *g, char *ws,
                            const LaPlan &pl, cudaStream_t s) {
  const int group = d->nheads / d->nheads_kv, H = d->nheads, Hkv = d->nheads_kv, dk = d->headdim_k,
            dv = d->headdim_v;
  const Role q{in->q, in->q_tok_stride, 1, H}, k{in->k, in->k_tok_stride, group, Hkv},
      v{in->v, in->v_tok_stride, group, Hkv}, o{dout, dout_stride, 1, H};
  float *part = reinterpret_cast<float *>(ws + pl.part);
  const long long rows = la_rows(d);
  const LaPass base = la_base(d, in, pl, ws);

  LaPass p = base;  // dq
  la_roles(p, o, v, k, dv, dk);
  la_states(p, in->initial_states, nullptr, true);
  p.o_scale = in->scale;
  p.p_scale = p.st_scale = 1.f;
  p.o = g->dq;
  p.os = g->dq_tok_stride;
  la_run<T>(p, false, s);

  p = base;  // dk
  la_roles(p, v, o, q, dv, dk);
  la_states(p, dfinal, nullptr, true);
  p.p_scale = p.st_scale = in->scale;
  p.o_scale = 1.f;
  p.o_f32 = group > 1;
  p.o = group > 1 ? part : g->dk;
  p.os = group > 1 ? (long long)H * dk : g->dk_tok_stride;
  la_run<T>(p, true, s);
  if (group > 1)
    SSD_LAUNCH("la_sum_heads", launch_la_sum_heads<T>(part, g->dk, g->dk_tok_stride, rows, Hkv, group, dk, s));

  p = base;  // dv, and the gradient of the initial states
  la_roles(p, k, q, o, dk, dv);
  la_states(p, dfinal, g->dinitial_states, false);
  p.p_scale = p.st_scale = in->scale;
  p.o_scale = 1.f;
  p.o_f32 = group > 1;
  p.o = group > 1 ? part : g->dv;
  p.os = group > 1 ? (long long)H * dv : g->dv_tok_stride;
  la_run<T>(p, true, s);
  if (group > 1)
    SSD_LAUNCH("la_sum_heads", launch_la_sum_heads<T>(part, g->dv, g->dv_tok_stride, rows, Hkv, group, dv, s));
  return launch_status();
}

// ---------------------------------------------------------------- group norm

ssd_status gn_check_dims(const ssd_group_norm_dims *d) {
  if (!d) return SSD_ERR_NULL_PTR;
  if (d->nsamples <= 0 || d->nrows <= 0 || d->channels <= 0 || d->groups <= 0 || d->channels % d->groups)
    return SSD_ERR_INVALID_DIMS;
  if (d->activation != SSD_ACT_NONE && d->activation != SSD_ACT_SILU && d->activation != SSD_ACT_GATE)
    return SSD_ERR_INVALID_DIMS;
  if (d->dtype != SSD_BF16 && d->dtype != SSD_F32) return SSD_ERR_DTYPE;
  if ((long long)d->nsamples * d->nrows > kMaxRows || d->channels > kMaxChannels ||
      (long long)d->nsamples * d->groups > (1LL << 30))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd_status gn_check_rows(const ssd_group_norm_dims *d, const void *p, int64_t stride) {
  if (!p) return SSD_ERR_NULL_PTR;
  if (stride < d->channels) return SSD_ERR_INVALID_DIMS;
  if (stride > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  return aligned(p, elem_bytes(d->dtype)) ? SSD_OK : SSD_ERR_ALIGNMENT;
}

ssd_status gn_check_inputs(const ssd_group_norm_dims *d, const ssd_group_norm_inputs *in) {
  if (!in) return SSD_ERR_NULL_PTR;
  ssd_status st = gn_check_rows(d, in->x, in->x_row_stride);
  if (st != SSD_OK) return st;
  if (d->activation == SSD_ACT_GATE) {
    st = gn_check_rows(d, in->z, in->z_row_stride);
    if (st != SSD_OK) return st;
  } else if (in->z) {
    return SSD_ERR_INVALID_DIMS;  // a gate that would be ignored: rejected instead
  }
  if (!aligned(in->weight, 4) || !aligned(in->bias, 4)) return SSD_ERR_ALIGNMENT;
  if (!(in->eps >= 0.f && in->eps < 1e30f)) return SSD_ERR_INVALID_DIMS;
  return SSD_OK;
}

// channels that rows of the tensor allow at once, at most `widest`: 8 (16 bytes of bf16, twice 16 of fp32), 2 or 1
int gn_width(const void *p, int64_t stride, int eb, int widest) {
  const int w = aligned(p, 16) && stride % 8 == 0 ? 8 : aligned(p, 2 * eb) && stride % 2 == 0 ? 2 : 1;
  return w < widest ? w : widest;
}

GnProblem gn_problem(const ssd_group_norm_dims *d, const ssd_group_norm_inputs *in) {
  GnProblem p{};
  p.n = d->nsamples;
  p.m = d->nrows;
  p.C = d->channels;
  p.G = d->groups;
  p.cg = d->channels / d->groups;
  p.act = d->activation;
  if (in) {
    p.x = in->x;
    p.xs = (int)in->x_row_stride;
    p.z = in->z;
    p.zs = (int)in->z_row_stride;
    p.w = in->weight;
    p.b = in->bias;
    p.eps = in->eps;
  }
  return p;
}

}  // namespace

extern "C" {

size_t ssd_linear_attn_workspace_size(const ssd_linear_attn_dims *dims, int backward) {
  if (la_check_dims(dims) != SSD_OK) return 0;
  return la_plan(dims, backward != 0).total;
}

ssd_status ssd_linear_attn_forward(const ssd_linear_attn_dims *dims, const ssd_linear_attn_inputs *in, void *o,
                                   int64_t o_tok_stride, float *final_states, void *workspace, size_t ws_bytes,
                                   ssd_stream_t stream) {
  ssd_status st = la_check_dims(dims);
  if (st == SSD_OK) st = la_check_inputs(dims, in);
  if (st == SSD_OK) st = la_check_rows(dims, o, o_tok_stride, (long long)dims->nheads * dims->headdim_v);
  if (st != SSD_OK) return st;
  if (!aligned(final_states, 16)) return SSD_ERR_ALIGNMENT;
  const LaPlan pl = la_plan(dims, false);
  st = la_check_workspace(pl, workspace, ws_bytes);
  if (st != SSD_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int group = dims->nheads / dims->nheads_kv;
  LaPass p = la_base(dims, in, pl, static_cast<char *>(workspace));
  la_roles(p, Role{in->q, in->q_tok_stride, 1, dims->nheads}, Role{in->k, in->k_tok_stride, group, dims->nheads_kv},
           Role{in->v, in->v_tok_stride, group, dims->nheads_kv}, dims->headdim_k, dims->headdim_v);
  la_states(p, in->initial_states, final_states, false);
  p.o_scale = in->scale;
  p.p_scale = p.st_scale = 1.f;
  p.o = o;
  p.os = o_tok_stride;
  cudaMemsetAsync(p.status, 0, 64, s);
  if (dims->dtype == SSD_BF16)
    la_run<__nv_bfloat16>(p, false, s);
  else
    la_run<float>(p, false, s);
  return launch_status();
}

ssd_status ssd_linear_attn_backward(const ssd_linear_attn_dims *dims, const ssd_linear_attn_inputs *in,
                                    const void *dout, int64_t dout_tok_stride, const float *dfinal_states,
                                    const ssd_linear_attn_grads *grads, void *workspace, size_t ws_bytes,
                                    ssd_stream_t stream) {
  ssd_status st = la_check_dims(dims);
  if (st == SSD_OK) st = la_check_inputs(dims, in);
  if (st != SSD_OK) return st;
  const long long HK = (long long)dims->nheads * dims->headdim_k, HV = (long long)dims->nheads * dims->headdim_v,
                  KK = (long long)dims->nheads_kv * dims->headdim_k, KV = (long long)dims->nheads_kv * dims->headdim_v;
  if (!grads) return SSD_ERR_NULL_PTR;
  st = la_check_rows(dims, dout, dout_tok_stride, HV);
  if (st == SSD_OK) st = la_check_rows(dims, grads->dq, grads->dq_tok_stride, HK);
  if (st == SSD_OK) st = la_check_rows(dims, grads->dk, grads->dk_tok_stride, KK);
  if (st == SSD_OK) st = la_check_rows(dims, grads->dv, grads->dv_tok_stride, KV);
  if (st != SSD_OK) return st;
  if (!aligned(dfinal_states, 16) || !aligned(grads->dinitial_states, 16)) return SSD_ERR_ALIGNMENT;
  const LaPlan pl = la_plan(dims, true);
  st = la_check_workspace(pl, workspace, ws_bytes);
  if (st != SSD_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  cudaMemsetAsync(ws + pl.status, 0, 64, s);
  if (dims->dtype == SSD_BF16)
    return la_backward_impl<__nv_bfloat16>(dims, in, dout, dout_tok_stride, dfinal_states, grads, ws, pl, s);
  return la_backward_impl<float>(dims, in, dout, dout_tok_stride, dfinal_states, grads, ws, pl, s);
}

ssd_status ssd_linear_attn_step(const ssd_linear_attn_dims *dims, const ssd_linear_attn_inputs *in, float *states,
                                int32_t nslots, const int32_t *slot_idx, void *o, int64_t o_tok_stride,
                                ssd_stream_t stream) {
  ssd_status st = la_check_dims(dims);
  if (st != SSD_OK) return st;
  if (dims->packed || dims->seqlen != 1) return SSD_ERR_INVALID_DIMS;
  st = la_check_inputs(dims, in);
  if (st == SSD_OK) st = la_check_rows(dims, o, o_tok_stride, (long long)dims->nheads * dims->headdim_v);
  if (st != SSD_OK) return st;
  if (in->initial_states) return SSD_ERR_INVALID_DIMS;  // the cache is the state
  if (!states) return SSD_ERR_NULL_PTR;
  if (nslots <= 0) return SSD_ERR_INVALID_DIMS;
  if (!aligned(states, 16) || !aligned(slot_idx, 4)) return SSD_ERR_ALIGNMENT;
  const int group = dims->nheads / dims->nheads_kv;
  LaPass p = la_base(dims, in, LaPlan{}, nullptr);
  la_roles(p, Role{in->q, in->q_tok_stride, 1, dims->nheads}, Role{in->k, in->k_tok_stride, group, dims->nheads_kv},
           Role{in->v, in->v_tok_stride, group, dims->nheads_kv}, dims->headdim_k, dims->headdim_v);
  p.o_scale = in->scale;
  p.o = o;
  p.os = o_tok_stride;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dims->dtype == SSD_BF16)
    SSD_LAUNCH("la_step", launch_la_step<__nv_bfloat16>(p, states, nslots, slot_idx, s));
  else
    SSD_LAUNCH("la_step", launch_la_step<float>(p, states, nslots, slot_idx, s));
  return launch_status();
}

size_t ssd_group_norm_workspace_size(const ssd_group_norm_dims *dims, int backward) {
  if (gn_check_dims(dims) != SSD_OK) return 0;
  return gn_workspace(gn_problem(dims, nullptr), backward != 0);
}

ssd_status ssd_group_norm_forward(const ssd_group_norm_dims *dims, const ssd_group_norm_inputs *in, void *y,
                                  int64_t y_row_stride, float *mean, float *rstd, void *workspace, size_t ws_bytes,
                                  ssd_stream_t stream) {
  ssd_status st = gn_check_dims(dims);
  if (st == SSD_OK) st = gn_check_inputs(dims, in);
  if (st == SSD_OK) st = gn_check_rows(dims, y, y_row_stride);
  if (st != SSD_OK) return st;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return SSD_ERR_ALIGNMENT;
  GnProblem p = gn_problem(dims, in);
  if (!workspace || ws_bytes < gn_workspace(p, false)) return SSD_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SSD_ERR_ALIGNMENT;
  const int eb = elem_bytes(dims->dtype);
  int widest = gn_width(y, y_row_stride, eb, gn_width(in->x, in->x_row_stride, eb, 8));
  if (dims->activation == SSD_ACT_GATE) widest = gn_width(in->z, in->z_row_stride, eb, widest);
  const GnPlan pl = gn_plan(p, false, widest);
  p.y = y;
  p.ys = (int)y_row_stride;
  p.mean = mean;
  p.rstd = rstd;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dims->dtype == SSD_BF16)
    run_gn_forward<__nv_bfloat16>(p, pl, static_cast<char *>(workspace), s);
  else
    run_gn_forward<float>(p, pl, static_cast<char *>(workspace), s);
  return launch_status();
}

ssd_status ssd_group_norm_backward(const ssd_group_norm_dims *dims, const ssd_group_norm_inputs *in, const void *dy,
                                   int64_t dy_row_stride, const float *mean, const float *rstd,
                                   const ssd_group_norm_grads *grads, void *workspace, size_t ws_bytes,
                                   ssd_stream_t stream) {
  ssd_status st = gn_check_dims(dims);
  if (st == SSD_OK) st = gn_check_inputs(dims, in);
  if (st == SSD_OK) st = gn_check_rows(dims, dy, dy_row_stride);
  if (st != SSD_OK) return st;
  if (!grads || !mean || !rstd) return SSD_ERR_NULL_PTR;
  st = gn_check_rows(dims, grads->dx, grads->dx_row_stride);
  if (st == SSD_OK && dims->activation == SSD_ACT_GATE) st = gn_check_rows(dims, grads->dz, grads->dz_row_stride);
  if (st != SSD_OK) return st;
  if (dims->activation != SSD_ACT_GATE && grads->dz) return SSD_ERR_INVALID_DIMS;
  if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(grads->dweight, 4) || !aligned(grads->dbias, 4))
    return SSD_ERR_ALIGNMENT;
  GnProblem p = gn_problem(dims, in);
  if (!workspace || ws_bytes < gn_workspace(p, true)) return SSD_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SSD_ERR_ALIGNMENT;
  const int eb = elem_bytes(dims->dtype);
  int widest = gn_width(in->x, in->x_row_stride, eb, gn_width(dy, dy_row_stride, eb, 8));
  widest = gn_width(grads->dx, grads->dx_row_stride, eb, widest);
  if (dims->activation == SSD_ACT_GATE)
    widest = gn_width(in->z, in->z_row_stride, eb, gn_width(grads->dz, grads->dz_row_stride, eb, widest));
  const GnPlan pl = gn_plan(p, true, widest);
  p.dy = dy;
  p.dys = (int)dy_row_stride;
  p.mean = const_cast<float *>(mean);  // read only on this path
  p.rstd = const_cast<float *>(rstd);
  p.dx = grads->dx;
  p.dxs = (int)grads->dx_row_stride;
  p.dz = grads->dz;
  p.dzs = (int)grads->dz_row_stride;
  p.dw = grads->dweight;
  p.db = grads->dbias;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dims->dtype == SSD_BF16)
    run_gn_backward<__nv_bfloat16>(p, pl, static_cast<char *>(workspace), s);
  else
    run_gn_backward<float>(p, pl, static_cast<char *>(workspace), s);
  return launch_status();
}

}  // extern "C"
