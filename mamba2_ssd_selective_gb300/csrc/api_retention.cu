// C ABI of linear attention with a decay for each head and of group norm with
// an activation: argument checks, workspace carving and launch sequences.
// Nothing here allocates or synchronises.
#include <cmath>
#include <initializer_list>

#include "group_norm.h"
#include "retention.h"

using namespace ssd;

namespace {

constexpr long long kMaxRows = 1LL << 30, kMaxChannels = 1 << 16;
constexpr int kMaxSeqs = 1 << 20;

// an output that starts where one of these inputs does
bool on_input(const void *out, std::initializer_list<const void *> inputs) {
  for (const void *p : inputs)
    if (out && out == p) return true;
  return false;
}

// ---------------------------------------------------------------- linear attention

struct LaPlan {
  enum Cut { kWhole, kChained, kSideBySide } cut;
  bool table;
  int seg_len, units, passes;
  size_t status, flags, table_at, seg, part, total;  // workspace offsets
  size_t seg_bytes;                                  // of one pass
};
// words at the start of the workspace: the status, the work counters, the table's number of units
constexpr int kLaCounters = 16, kLaTableUnits = kLaCounters + kLaCounterWords;

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
      d->nseq > kMaxSeqs || (long long)d->nseq * d->nheads > (1LL << 28) || (long long)d->nheads * d->headdim_k > kMaxChannels ||
      (long long)d->nheads * d->headdim_v > kMaxChannels)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

// bf16 within its widths takes the tensor-core kernel, everything else the CUDA-core one
bool la_use_tc(const ssd_linear_attn_dims *d) {
  return d->dtype == SSD_BF16 && la_tc_envelope(d->headdim_k, d->headdim_v);
}

// Whether and where sequences are cut, and the workspace.
//
// Cut side by side, a sequence's segments run at once: their own states first (a second read of k and v), a scan,
// then the pass.  Chained (tensor cores), segments of all sequences are items of a queue in order of their
// level, a segment's state handed to the next: nothing is done twice, and SMs that finish early take over, but a
// sequence still takes its time.  Which one, and the length of a segment, are those of the least cost by the
// times measured here, in us:
//   tensor cores, a block of 64 tokens on an SM: 1.3 (1.33 at widths of 128, 1.19 at 64); of segments' states 0.9;
//   CUDA cores, a block of 32 tokens and 64 columns: 6.3 for one by itself, 5 where the SM has others;
//   handing a state on: 3 blocks; a scan and a launch more: 17; the table of packed sequences' segments: 8.
// Lengths of packed sequences are not known here: the longest of n is taken for its mean where
// sequences end at random, (1 + 1/2 + ... + 1/n) / n of all tokens.
// Whole against side by side: one sequence of 31991 tokens, 16 heads of 128, bf16, 616 us against 165 in 9 segments;
// four of 8192, 169 against 170 in 2; fp32, 4 x 2048 tokens, 12 heads of 64, 460 us against 171; 8 x 4096, 32
// heads of 128, 4440 us against 5560.
// Whole against chained: 192 items of 8192 tokens of 128 (two sequences' backward pass, 32 heads) 349 us against 288 in
// 4 segments, 301 in 8 and 262 in 3; 24 packed sequences of 1 to 4487 tokens, 16 heads, 107 us against 104 in
// segments of 1024 and 94 in segments of 2048.
LaPlan la_plan(const ssd_linear_attn_dims *d, bool backward) {
  LaPlan pl{};
  const bool tc = la_use_tc(d);
  pl.passes = backward ? 3 : 1;
  const int wide = d->headdim_k > d->headdim_v ? d->headdim_k : d->headdim_v, wide64 = (wide + 63) / 64;
  // (the SMs are not asked for: a workspace's size may be, where there is no GPU, and is that of the same plan)
  const long long rows = la_rows(d), H = d->nheads, n = d->nseq, sms = 152;
  const long long longest = d->packed ? rows : d->seqlen;
  // blocks (CTAs or items) of a whole sequence of every head and pass, all of them, and those with states to sum
  // (both reverse passes share theirs)
  const long long each = H * pl.passes * (tc ? 1 : wide64), all = n * each;
  const double summing = backward ? 2. / 3. : 1.;
  const int kb = tc ? 64 : 32;
  // in blocks of kb tokens: an SM's share of all work, and the longest sequence
  const double share = (double)(d->packed ? rows * each : longest * all) / sms / kb;
  const double part = d->packed ? (std::log((double)n) + 0.577 + 0.5 / (double)n) / (double)n : 1.;
  const double chain = (double)longest / kb * (part < 1. ? part : 1.);
  const bool cuttable = !d->packed || n <= kLaMaxCutSeqs;
  const double table = d->packed ? 8. : 0.;
  auto up = [](long long x, long long y) { return (x + y - 1) / y; };
  long long seg = 0;
  double best = 0.;
  auto take_if = [&](LaPlan::Cut cut, long long length, double cost) {
    const bool fits = length < longest && (rows / length + n) * each < (1LL << 28);  // item numbers are 32-bit
    if (cut == LaPlan::kWhole || (fits && cuttable && cost < best)) {
      pl.cut = cut;
      seg = length;
      best = cost;
    }
  };
  if (tc && !d->packed) {
    const long long tiles = up(longest, kb);
    take_if(LaPlan::kWhole, longest, 1.3 * (double)(up(all, sms) * (tiles + 3)));
    for (long long c = 2; c <= 152 && 4 * c <= tiles; ++c) {
      const long long len = up(tiles, c), rounds = up(all * c, sms);
      take_if(LaPlan::kChained, len * kb, 1.3 * (double)((rounds > c ? rounds : c) * (len + 3)));
      const double sums = (double)up((long long)((double)(all * (c - 1)) * summing), sms);
      take_if(LaPlan::kSideBySide, len * kb, 1.3 * ((double)(rounds * (len + 3)) + sums * (0.7 * (double)len + 3.)) + 17.);
    }
  } else if (tc) {
    const double longer = share > chain ? share : chain;
    take_if(LaPlan::kWhole, longest, 1.3 * (longer + 0.5 * share));
    // hand-overs in all against the last items' idle SMs
    long long len = (long long)std::sqrt(6. * share) * kb;
    if (len < 2048) len = 2048;
    take_if(LaPlan::kChained, len, 1.3 * (longer + 3. * chain * kb / (double)len) + table);
    len = ((long long)share + 1) * kb;
    if (len < 512) len = 512;
    const double of = share > (double)len / kb ? share : (double)len / kb;
    take_if(LaPlan::kSideBySide, len, 1.3 * (of + 3.) * (1. + 0.7 * summing) + 17. + table);
  } else {
    const double alone = 6.3 * wide64, among = 5. * wide64;
    auto time = [&](double blocks) { return alone * blocks > among * share ? alone * blocks : among * share; };
    take_if(LaPlan::kWhole, longest, time(chain));
    // segments enough for every SM's places (by shared memory), twice over as they are short
    const long long want = 2 * sms * (wide64 == 1 ? 4 : wide64 == 2 ? 2 : 1);
    long long len = up(d->packed ? rows * each / want : up(longest * all, want), 64) * 64;
    if (len < 64) len = 64;
    take_if(LaPlan::kSideBySide, len, time((double)len / kb) * (1. + 0.5 * summing) + 17. + table);
  }
  if (pl.cut == LaPlan::kWhole) seg = (longest + 63) / 64 * 64;
  const bool cut = pl.cut != LaPlan::kWhole;
  pl.seg_len = (int)seg;
  pl.table = cut && d->packed;
  pl.units = (int)(!cut ? n : d->packed ? rows / seg + n : n * ((longest + seg - 1) / seg));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  pl.status = take(256);
  pl.flags = take(pl.cut == LaPlan::kChained ? (size_t)pl.passes * pl.units * H * 4 : 0);
  pl.table_at = take(pl.table ? (size_t)pl.units * sizeof(LaEntry) : 0);
  pl.seg_bytes = align_up((size_t)pl.units * H * d->headdim_k * d->headdim_v * 4, 256);
  pl.seg = take(cut ? pl.passes * pl.seg_bytes : 0);
  pl.part = take(backward && d->nheads != d->nheads_kv ? (size_t)rows * H * (d->headdim_k + d->headdim_v) * 4 : 0);
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

LaPlanDev la_plan_dev(const ssd_linear_attn_dims *d, const ssd_linear_attn_inputs *in, const LaPlan &pl, char *ws) {
  LaPlanDev v{};
  v.nseq = d->nseq;
  v.seqlen = d->seqlen;
  v.total = (int)la_rows(d);
  v.H = d->nheads;
  v.cu = in->cu_seqlens;
  v.seg_len = pl.seg_len;
  v.units = pl.units;
  v.status = reinterpret_cast<int *>(ws + pl.status);
  v.counters = v.status + kLaCounters;
  if (pl.table) {
    v.table = reinterpret_cast<const LaEntry *>(ws + pl.table_at);
    v.table_units = v.status + kLaTableUnits;
  }
  if (pl.cut == LaPlan::kChained) v.flags = reinterpret_cast<int *>(ws + pl.flags);
  v.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  return v;
}

// pass i of a call; the tensors, scales and states follow
LaPass la_pass(const ssd_linear_attn_dims *d, const ssd_linear_attn_inputs *in, const LaPlan &pl, char *ws, int i) {
  LaPass p{};
  p.H = d->nheads;
  p.g = in->log_decay;
  p.seg_state = reinterpret_cast<float *>(ws + pl.seg + i * pl.seg_bytes);
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

// The passes of a call: status, counters and flags cleared (and the table of units written), then the passes, in
// batches that share a kernel.
template <typename T>
void la_run(const ssd_linear_attn_dims *d, const LaPlan &pl, const LaPlanDev &dev, const LaPass *p, int n, char *ws,
            cudaStream_t s) {
  const int nflags = pl.cut == LaPlan::kChained ? pl.passes * pl.units * d->nheads : 0;
  if (pl.table)
    SSD_LAUNCH("la_table", launch_la_table(dev, reinterpret_cast<LaEntry *>(ws + pl.table_at),
                                           dev.status + kLaTableUnits, nflags, s));
  else
    cudaMemsetAsync(ws, 0, pl.flags + (size_t)nflags * 4, s);
  const bool tc = sizeof(T) == 2 && la_use_tc(d);
  // batches of passes that one kernel takes: on the tensor cores those of the same boxes
  auto batches = [&](bool summary, auto launch) {
    int number = 0;
    for (int done = 0; done < n;) {
      LaBatch b{};
      LaPlanDev v = dev;
      v.counters += 2 * number++;
      if (v.flags) v.flags += (size_t)done * pl.units * d->nheads;
      auto kernel = [](const LaPass &x) { return 2 * la_tc_boxes(x.dk) + la_tc_boxes(x.dv); };
      for (; done < n; ++done) {
        if (summary && p[done].seg_shared) continue;
        if (tc && b.n > 0 && kernel(p[done]) != kernel(b.p[0])) break;
        b.p[b.n++] = p[done];
      }
      launch(v, b);
    }
  };
  if (pl.cut == LaPlan::kSideBySide)
    batches(true, [&](const LaPlanDev &v, const LaBatch &b) {
      SSD_LAUNCH("la_segment_states", tc ? launch_la_tc(v, b, true, s) : launch_la_simt<T>(v, b, true, s));
      SSD_LAUNCH("la_scan", launch_la_scan(v, b, s));
    });
  batches(false, [&](const LaPlanDev &v, const LaBatch &b) {
    SSD_LAUNCH("la_pass", tc ? launch_la_tc(v, b, false, s) : launch_la_simt<T>(v, b, false, s));
  });
}

template <typename T>
ssd_status la_backward_impl(const ssd_linear_attn_dims *d, const ssd_linear_attn_inputs *in, const void *dout,
                            int64_t dout_stride, const float *dfinal, const ssd_linear_attn_grads *g, char *ws,
                            const LaPlan &pl, cudaStream_t s) {
  const int group = d->nheads / d->nheads_kv, H = d->nheads, Hkv = d->nheads_kv, dk = d->headdim_k,
            dv = d->headdim_v;
  const Role q{in->q, in->q_tok_stride, 1, H}, k{in->k, in->k_tok_stride, group, Hkv},
      v{in->v, in->v_tok_stride, group, Hkv}, o{dout, dout_stride, 1, H};
  const long long rows = la_rows(d);
  float *part_k = reinterpret_cast<float *>(ws + pl.part), *part_v = part_k + (size_t)rows * H * dk;
  LaPass p[3] = {la_pass(d, in, pl, ws, 0), la_pass(d, in, pl, ws, 1), la_pass(d, in, pl, ws, 2)};
  // dq
  la_roles(p[0], o, v, k, dv, dk);
  la_states(p[0], in->initial_states, nullptr, true);
  p[0].o_scale = in->scale;
  p[0].p_scale = p[0].st_scale = 1.f;
  p[0].o = g->dq;
  p[0].os = g->dq_tok_stride;
  // dk
  la_roles(p[1], v, o, q, dv, dk);
  la_states(p[1], dfinal, nullptr, true);
  p[1].o = group > 1 ? part_k : g->dk;
  p[1].os = group > 1 ? (long long)H * dk : g->dk_tok_stride;
  // dv, and the gradient of the initial states
  la_roles(p[2], k, q, o, dk, dv);
  la_states(p[2], dfinal, g->dinitial_states, false);
  p[2].o = group > 1 ? part_v : g->dv;
  p[2].os = group > 1 ? (long long)H * dv : g->dv_tok_stride;
  for (int i = 1; i < 3; ++i) {
    p[i].reverse = true;
    p[i].o_scale = 1.f;
    p[i].p_scale = p[i].st_scale = in->scale;
    p[i].o_f32 = group > 1;
  }
  if (pl.cut == LaPlan::kSideBySide) {  // both reverse passes carry the same state, one of them transposed
    p[1].seg_state = p[2].seg_state;
    p[1].seg_shared = true;
  }
  la_run<T>(d, pl, la_plan_dev(d, in, pl, ws), p, 3, ws, s);
  if (group > 1)
    SSD_LAUNCH("la_sum_heads", launch_la_sum_heads<T>({part_k, g->dk, g->dk_tok_stride, dk},
                                                      {part_v, g->dv, g->dv_tok_stride, dv}, rows, Hkv, group, s));
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
  if (on_input(o, {in->q, in->k, in->v})) return SSD_ERR_INVALID_DIMS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int group = dims->nheads / dims->nheads_kv;
  char *ws = static_cast<char *>(workspace);
  LaPass p = la_pass(dims, in, pl, ws, 0);
  la_roles(p, Role{in->q, in->q_tok_stride, 1, dims->nheads}, Role{in->k, in->k_tok_stride, group, dims->nheads_kv},
           Role{in->v, in->v_tok_stride, group, dims->nheads_kv}, dims->headdim_k, dims->headdim_v);
  la_states(p, in->initial_states, final_states, false);
  p.o_scale = in->scale;
  p.p_scale = p.st_scale = 1.f;
  p.init_kept = pl.cut == LaPlan::kSideBySide && final_states && final_states == in->initial_states;
  p.o = o;
  p.os = o_tok_stride;
  const LaPlanDev dev = la_plan_dev(dims, in, pl, ws);
  if (dims->dtype == SSD_BF16)
    la_run<__nv_bfloat16>(dims, pl, dev, &p, 1, ws, s);
  else
    la_run<float>(dims, pl, dev, &p, 1, ws, s);
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
  for (const void *out : {grads->dq, grads->dk, grads->dv})
    if (on_input(out, {in->q, in->k, in->v, dout})) return SSD_ERR_INVALID_DIMS;
  if (on_input(grads->dinitial_states, {in->initial_states, dfinal_states})) return SSD_ERR_INVALID_DIMS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
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
  if (on_input(o, {in->q, in->k, in->v})) return SSD_ERR_INVALID_DIMS;
  const int group = dims->nheads / dims->nheads_kv;
  LaPass p{};
  p.H = dims->nheads;
  p.g = in->log_decay;
  la_roles(p, Role{in->q, in->q_tok_stride, 1, dims->nheads}, Role{in->k, in->k_tok_stride, group, dims->nheads_kv},
           Role{in->v, in->v_tok_stride, group, dims->nheads_kv}, dims->headdim_k, dims->headdim_v);
  p.o_scale = in->scale;
  p.o = o;
  p.os = o_tok_stride;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dims->dtype == SSD_BF16)
    SSD_LAUNCH("la_step", launch_la_step<__nv_bfloat16>(p, dims->nseq, states, nslots, slot_idx, s));
  else
    SSD_LAUNCH("la_step", launch_la_step<float>(p, dims->nseq, states, nslots, slot_idx, s));
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
  if ((y == in->x && y_row_stride != in->x_row_stride) || (y == in->z && y_row_stride != in->z_row_stride))
    return SSD_ERR_INVALID_DIMS;  // in place, but at other places
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
  if (on_input(grads->dx, {in->x, in->z, dy, grads->dz}) || on_input(grads->dz, {in->x, in->z, dy}))
    return SSD_ERR_INVALID_DIMS;
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
