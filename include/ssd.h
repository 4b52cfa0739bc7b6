/*
 * ssd.h -- C ABI of libssd: the Mamba2 mixer core (conv1d + SiLU over xBC,
 * chunked SSD, causal segments with affine summaries, exclusive segment scan,
 * correction), forward and backward, on one GB300 (sm_103a).
 *
 * Method.  Megatron-LM PR #6808 "Add state-passing context parallelism for
 * Mamba2" (description): the SSD transform of one causal segment is affine in
 * its initial state, S_out = a_block * S_in + S_ext; every segment computes its
 * (S_ext, a_block) from a zero initial state, an exclusive causal scan over the
 * summaries recovers each segment's true initial state, and a correction pass
 * applies it; the conv halo is the previous segment's last d_conv-1 tokens;
 * backward mirrors this with a reverse boundary scan and recomputes everything
 * that scales with the sequence length.  Resets at packed-sequence boundaries
 * follow seq_idx derived from cu_seqlens (NeMo Automodel PR #1441 "feat:
 * context-parallel with nemotron v3", Key changes).  The per-token model is the
 * Mamba2 selective SSM:
 *     u      = SiLU(causal depthwise conv1d(xBC) + conv_b)      (x, B, C parts)
 *     dt_t   = softplus(dt_raw_t + dt_bias),  A = -exp(A_log)
 *     h_t    = exp(dt_t*A) * h_{t-1} + dt_t * x_t (outer) B_t    (P x N per head)
 *     y_t    = h_t . C_t + D * x_t
 * with the state zeroed where seq_idx changes and the conv taps masked there.
 *
 * Conventions shared by every call:
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *    never allocates, frees or synchronises the host; every call only enqueues
 *    work on `stream` (a cudaStream_t; NULL = the legacy default stream).
 *  - Arguments are validated before anything is launched.  A rejected call
 *    returns a negative ssd_status and launches nothing.  SSD_ERR_CUDA means a
 *    launch failed; the CUDA error is then also left for cudaGetLastError().
 *  - Activations (x, B, C, dt_raw, y, dy and their grads) use `dims.dtype`;
 *    parameters, states and parameter grads are fp32.  Arithmetic is fp32
 *    (bf16 tensor-core operands with fp32 accumulation on the bf16 path).
 *  - Shapes: b = batch, L = seqlen, H = nheads, P = headdim, N = dstate,
 *    G = ngroups (head h reads group h / (H/G)), Q = chunk, S = n_segments.
 *    Token-major layouts: element (b, t, c) of a tensor with token stride ts
 *    lives at ptr[(b*L + t)*ts + c].  Channels within a token are contiguous.
 */
#ifndef SSD_H
#define SSD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *ssd_stream_t; /* == cudaStream_t */

typedef enum {
  SSD_OK = 0,
  SSD_ERR_INVALID_DIMS = -1,   /* a dimension is <= 0, H % G != 0, or d_conv != 4 */
  SSD_ERR_SEGMENT_ALIGN = -2,  /* L % (n_segments * chunk) != 0 */
  SSD_ERR_NULL_PTR = -3,       /* a required pointer is NULL */
  SSD_ERR_ALIGNMENT = -4,      /* pointer or token stride violates the alignment rules below */
  SSD_ERR_DTYPE = -5,          /* dims.dtype is not an ssd_dtype */
  SSD_ERR_WORKSPACE = -6,      /* workspace NULL or smaller than ssd_workspace_size() */
  SSD_ERR_UNSUPPORTED = -7,    /* valid but outside the supported envelope (see ssd_forward) */
  SSD_ERR_CUDA = -8,           /* a kernel launch failed */
  SSD_ERR_DEVICE_TIMEOUT = -9  /* a bounded device-side wait gave up (see ssd_device_status) */
} ssd_status;

typedef enum { SSD_BF16 = 0, SSD_F32 = 1 } ssd_dtype;

typedef struct {
  int32_t batch, seqlen, nheads, headdim, dstate, ngroups;
  int32_t d_conv;     /* must be 4 */
  int32_t chunk;      /* Q: SSD chunk length */
  int32_t n_segments; /* S: equal causal segments; each must be a multiple of chunk */
  int32_t dtype;      /* ssd_dtype of the activations */
  int32_t gated_norm; /* 1: y is the gated RMSNorm of the mixer output (needs z and
                         norm_weight in ssd_inputs; at most 4096 channels per group), 0: none */
} ssd_dims;

/* Pre-conv activations as laid out by the in-projection (zero-copy views into
 * one zxBCdt buffer are fine: pass each part's pointer and token stride).
 *   x  (b, L, H*P)  B (b, L, G*N)  C (b, L, G*N)  dt (b, L, H)
 * x, B, C: 16-byte aligned, token strides a multiple of 8 elements (bf16) or
 * 4 elements (fp32).  dt: element aligned, any token stride >= H.
 * Parameters (fp32, contiguous): dt_bias, A_log, D (H); conv_w (Cd, 4),
 * 16-byte aligned, where tap 3 multiplies the current token; conv_b (Cd);
 * Cd = H*P + 2*G*N and the conv channel order is [x | B | C].
 * seq_idx (b, L) int32, 16-byte aligned (the tensor-core kernels copy it into
 * shared memory in 16-byte units), non-decreasing within a row, or NULL (one
 * sequence per row).  The state and the conv taps are reset where it changes.
 * initial_states (b, H, P, N) fp32, 16-byte aligned, or NULL (zero): each row's
 * state before its first token, to which that token's decay applies (the
 * Mamba2 chunked-scan convention; the pages list initial states as not
 * supported yet: "Add state-passing context parallelism for Mamba2", "Not
 * supported yet").  With packed rows it seeds the row's first sequence only;
 * later sequences start from zero.  The exclusive segment scan starts from it.
 * Gated RMSNorm (dims.gated_norm = 1; else z and norm_weight must be NULL): the
 * step after the mixer core in a Mamba2 block, which the Megatron-LM PR keeps
 * outside its fused function (description); Mamba2's gated norm with one norm
 * group per B/C group of heads (H*P/G channels):
 *     g = y * silu(z),   out = g * norm_weight / sqrt(mean_group(g^2) + norm_eps)
 * z (b, L, H*P) activation dtype with its own token stride (a view into the
 * zxBCdt buffer), 16-byte aligned, stride a multiple of 8 (bf16) or 4 (fp32)
 * elements; norm_weight (H*P) fp32, 16-byte aligned; norm_eps >= 0. */
typedef struct {
  const void *x;  int64_t x_tok_stride;
  const void *B;  int64_t B_tok_stride;
  const void *C;  int64_t C_tok_stride;
  const void *dt; int64_t dt_tok_stride;
  const float *dt_bias, *A_log, *D, *conv_w, *conv_b;
  const int32_t *seq_idx;
  const float *initial_states;
  const void *z;  int64_t z_tok_stride;
  const float *norm_weight;
  float norm_eps;
} ssd_inputs;

/* Gradients, written (not accumulated).  dx, dB, dC, ddt have the layout and
 * alignment rules of x, B, C, dt, with their own token strides (they may be
 * views into one d(zxBCdt) buffer).  ddt_bias, dA_log, dD (H), dconv_w (Cd,4),
 * dconv_b (Cd) are fp32 and summed over batch and tokens.  dinitial_states
 * (b, H, P, N) fp32, 16-byte aligned: the gradient of the initial states, the
 * reverse segment scan carried one step past the first segment; written only
 * when the inputs have initial_states, and may be NULL.  With the gated norm:
 * dz (layout rules of z, its own token stride) and dnorm_weight (H*P) fp32,
 * both required. */
typedef struct {
  void *dx;  int64_t dx_tok_stride;
  void *dB;  int64_t dB_tok_stride;
  void *dC;  int64_t dC_tok_stride;
  void *ddt; int64_t ddt_tok_stride;
  float *ddt_bias, *dA_log, *dD, *dconv_w, *dconv_b;
  float *dinitial_states;
  void *dz;  int64_t dz_tok_stride;
  float *dnorm_weight;
} ssd_grads;

/* Bytes of device workspace ssd_forward (backward = 0) or ssd_backward
 * (backward = 1) needs for `dims`; 0 if dims are invalid.  The workspace is
 * scratch: its contents need not survive between calls. */
size_t ssd_workspace_size(const ssd_dims *dims, int backward);

/* Forward.  y (b, L, H*P) activation dtype, contiguous (with the gated norm: its
 * output; the mixer output itself is not written); final_state (b, H, P, N)
 * fp32 = the state after each row's last token (with packing: of the row's last
 * sequence), or NULL; seg_init_states (b, S, H, P, N) fp32 = each segment's true
 * initial state recovered by the exclusive scan (what ssd_backward may reuse),
 * or NULL.  Supported envelope: P and N multiples of 8 and <= 256, chunk a
 * multiple of 32 and <= 256, n_segments <= 1024; otherwise SSD_ERR_UNSUPPORTED. */
ssd_status ssd_forward(const ssd_dims *dims, const ssd_inputs *in, void *y, float *final_state,
                       float *seg_init_states, void *workspace, size_t ws_bytes, ssd_stream_t stream);

/* Forward of a packed row of sequences (THD layout, dims.batch = 1) that also
 * returns the state after every sequence's last token: seq_final_states
 * (nseq, H, P, N) fp32, 16-byte aligned, sequence s covering tokens
 * [cu_seqlens[s], cu_seqlens[s+1]) (cu_seqlens: nseq + 1 int32 device values, the
 * layout of "feat: context-parallel with nemotron v3", Key changes).  in->seq_idx
 * is required and must describe the same sequences (ssd_cu_seqlens_to_seq_idx
 * makes it; neither is checked against the other on the host).  Sequences
 * that are empty or fall outside [0, seqlen) get a zero state.  Everything else
 * as ssd_forward, same workspace size.  No gradient flows back through
 * seq_final_states (ssd_backward's dfinal_state is the row's last token's). */
ssd_status ssd_forward_varlen(const ssd_dims *dims, const ssd_inputs *in, void *y, float *final_state,
                              float *seg_init_states, const int32_t *cu_seqlens, int32_t nseq,
                              float *seq_final_states, void *workspace, size_t ws_bytes, ssd_stream_t stream);

/* Backward of  L = <dy, y> + <dfinal_state, final_state>  (y the forward's output:
 * with the gated norm, the normalised output; the mixer output is recomputed).
 * dy (b, L, H*P) activation dtype, contiguous; dfinal_state (b, H, P, N) fp32 or
 * NULL (zero); seg_init_states from ssd_forward on the same inputs, or NULL to
 * have them recomputed.  Everything that scales with L is recomputed. */
ssd_status ssd_backward(const ssd_dims *dims, const ssd_inputs *in, const void *dy, const float *dfinal_state,
                        const float *seg_init_states, const ssd_grads *grads, void *workspace, size_t ws_bytes,
                        ssd_stream_t stream);

/* Forward without any workspace argument, for callers that cannot allocate
 * device memory: code running inside a host framework that owns every device
 * allocation and forbids new ones after start-up (inference plugins, real-time
 * serving loops), or code for which a cudaMalloc would synchronise the device
 * and break its latency budget.  Same arguments, results and rules as
 * ssd_forward minus the workspace.  The scratch is one fixed array of
 * SSD_STATIC_SCRATCH_BYTES in the library's device memory (each GPU that loads
 * the library holds it until the process exits); problems whose forward needs
 * more (ssd_workspace_size(dims, 0) > SSD_STATIC_SCRATCH_BYTES) are rejected
 * with SSD_ERR_WORKSPACE before anything is launched.  The first call on each
 * device looks up the array's device address (make that first call before any
 * stream capture); no call allocates or frees memory.  All calls share the one
 * array, so calls whose GPU work may overlap (other streams, other host
 * threads) race on it and must be serialised by the caller.  The array's
 * status word (a device-side wait that gave up) is read with
 * ssd_device_status(NULL, stream).  This entry point has no counterpart in the
 * pages the method comes from. */
#define SSD_STATIC_SCRATCH_BYTES (32u << 20)
ssd_status ssd_forward_static(const ssd_dims *dims, const ssd_inputs *in, void *y, float *final_state,
                              float *seg_init_states, ssd_stream_t stream);

/* seq_idx[t] = i for cu_seqlens[i] <= t < cu_seqlens[i+1], t in [0, total_tokens)
 * (NeMo Automodel PR #1441, Key changes: seq_idx computed from cu_seqlens).
 * cu_seqlens (nseq + 1) int32 device array, non-decreasing, cu_seqlens[0] = 0 and
 * cu_seqlens[nseq] = total_tokens (not checked on the host: tokens outside every
 * range get seq_idx -1). */
ssd_status ssd_cu_seqlens_to_seq_idx(const int32_t *cu_seqlens, int32_t nseq, int32_t *seq_idx,
                                     int32_t total_tokens, ssd_stream_t stream);

/* Reads the device status word kept in `workspace` by the last call that used
 * it (synchronises `stream`): SSD_OK, or SSD_ERR_DEVICE_TIMEOUT if a bounded
 * device-side wait gave up (the outputs of that call are then garbage; the
 * context stays usable and the next call starts from a cleared word).
 * workspace = NULL reads the word of ssd_forward_static's fixed scratch array
 * on the current device instead.  Returns SSD_ERR_CUDA if the read fails. */
ssd_status ssd_device_status(const void *workspace, ssd_stream_t stream);

/* Failure detection.  Every wait of one role of a kernel on another (mbarrier
 * hand-offs inside the tensor-core kernels) gives up after this limit,
 * raises the status word that ssd_device_status reads and lets the kernel
 * finish: it drains the copies and tensor-core operations it started, frees
 * its tensor memory and returns, so the process can carry on.  Applies to the
 * calls made after it, from any host thread; returns the previous limit.  The
 * default, SSD_DEFAULT_WAIT_LIMIT_NS (1.5 s), is far above any real hand-off;
 * a limit of 0 makes every wait that is not already satisfied give up (a way
 * to exercise the failure path). */
#define SSD_DEFAULT_WAIT_LIMIT_NS 1500000000ull
uint64_t ssd_set_wait_limit_ns(uint64_t limit_ns);

/* Per-kernel timing for benchmarks.  After ssd_profile_begin(), every kernel
 * that ssd_forward / ssd_backward launch (from this host thread) is bracketed
 * by a pair of CUDA events recorded on the launch stream (events come from a
 * fixed pool created on the first begin; at most 65536 launches are recorded,
 * later ones run unrecorded).  ssd_profile_end() waits for the recorded events,
 * writes up to max_entries per-kernel totals (name, launches, summed
 * milliseconds) in first-launch order, stops recording and returns the number
 * of entries, or a negative ssd_status.  Not for use during stream capture. */
typedef struct {
  const char *name; /* static string */
  int32_t launches;
  float total_ms;
} ssd_kernel_time;

ssd_status ssd_profile_begin(void);
int32_t ssd_profile_end(ssd_kernel_time *out, int32_t max_entries);

/* ======================= retention: linear attention with a decay for each head, and the norm behind it
 *
 * Linear attention.  Per query head h, with lam = exp(log_decay[h]) and kv = h / (nheads / nheads_kv), for the
 * tokens t of one sequence in order:
 *     S_t = lam S_{t-1} + k_{t,kv}^T v_{t,kv}      (headdim_k x headdim_v; S_{-1}: the initial state, or zero)
 *     o_t = scale q_{t,h} S_t
 * Sequences either all have dims.seqlen tokens (cu_seqlens NULL; token t of sequence s is row s * seqlen + t), or
 * are packed into dims.total_tokens rows: sequence s covers rows [cu_seqlens[s], cu_seqlens[s+1]), cu_seqlens
 * (nseq + 1) int32 device values, non-decreasing, from 0 to total_tokens (not checked on the host; values outside
 * [0, total_tokens] are clamped, a bound below the one before gives an empty sequence, what rows of several
 * sequences get is undefined, rows outside every sequence are neither read as data nor written).  Sequences may
 * be empty or of one token; with no token the final state is the initial state.
 * Tensors are token-major with their own token strides, heads and channels contiguous within a token:
 *   q (T, nheads * headdim_k), k (T, nheads_kv * headdim_k), v (T, nheads_kv * headdim_v), o (T, nheads * headdim_v)
 * in dims.dtype, 16-byte aligned, strides a multiple of 8 (bf16) or 4 (fp32) elements, so views into one
 * projection output are read in place.  log_decay (nheads) fp32, at most 0 (-inf: the state forgets everything at
 * each token).  States (nseq, nheads, headdim_k, headdim_v) fp32, contiguous, 16-byte aligned.
 * Arithmetic: fp32; on the bf16 tensor-core path (headdim_k and headdim_v at most 128) the products take bf16
 * operands with fp32 accumulation, and what reaches the state is split into three bf16 terms, so that states keep
 * fp32 precision.  There a head's scores q.k (backward: do.v, and with the scale) are weighed by up to 2^40 before they
 * are rounded, so scores beyond 2^87 overflow; elsewhere the limit is that of fp32.  A NaN or infinity in a token can
 * reach every output of the same 64-token block of its own sequence and head, and those of later tokens (dk and dv:
 * of earlier ones); other sequences are not affected.
 * Envelope: headdim_k and headdim_v multiples of 8, at most 256; nheads * headdim and total rows as in ssd_dims; at
 * most 2^20 sequences and 2^28 sequences x heads; else SSD_ERR_UNSUPPORTED.  All sums have a fixed order: equal inputs give equal bits. */
typedef struct {
  int32_t nseq;
  int32_t seqlen;       /* tokens of every sequence; ignored when packed */
  int32_t total_tokens; /* packed: rows of the token-major tensors; else 0 or nseq * seqlen */
  int32_t packed;       /* 1: cu_seqlens gives the sequences */
  int32_t nheads, nheads_kv, headdim_k, headdim_v;
  int32_t dtype; /* ssd_dtype of q, k, v, o and their gradients */
} ssd_linear_attn_dims;

typedef struct {
  const void *q; int64_t q_tok_stride;
  const void *k; int64_t k_tok_stride;
  const void *v; int64_t v_tok_stride;
  const float *log_decay;
  const float *initial_states; /* or NULL: zero */
  const int32_t *cu_seqlens;   /* exactly when dims.packed */
  float scale;
} ssd_linear_attn_inputs;

/* Gradients, written (not accumulated).  dq, dk, dv: layout rules of q, k, v, own token strides; dk and dv are
 * summed over the query heads that share a key/value head.  dinitial_states fp32: written when not NULL (it does
 * not need initial_states to be given).  log_decay is a constant of the model and has no gradient. */
typedef struct {
  void *dq; int64_t dq_tok_stride;
  void *dk; int64_t dk_tok_stride;
  void *dv; int64_t dv_tok_stride;
  float *dinitial_states;
} ssd_linear_attn_grads;

/* Bytes of device workspace of ssd_linear_attn_forward (backward = 0) or _backward (1); 0 if dims are invalid. */
size_t ssd_linear_attn_workspace_size(const ssd_linear_attn_dims *dims, int backward);

/* Forward.  final_states: the state after each sequence's last token, or NULL; it may be initial_states itself, which
 * are then updated in place.  o must not overlap an input: one that starts where an input does is refused
 * (SSD_ERR_INVALID_DIMS). */
ssd_status ssd_linear_attn_forward(const ssd_linear_attn_dims *dims, const ssd_linear_attn_inputs *in, void *o,
                                   int64_t o_tok_stride, float *final_states, void *workspace, size_t ws_bytes,
                                   ssd_stream_t stream);

/* Backward of <do, o> + <dfinal_states, final_states> (dfinal_states NULL: zero).  do is named dout here: layout
 * rules of o.  Nothing but the inputs is needed from the forward pass.  Gradients must not overlap what is read:
 * dinitial_states = dfinal_states is refused (SSD_ERR_INVALID_DIMS), as is any output that starts where an input does. */
ssd_status ssd_linear_attn_backward(const ssd_linear_attn_dims *dims, const ssd_linear_attn_inputs *in,
                                    const void *dout, int64_t dout_tok_stride, const float *dfinal_states,
                                    const ssd_linear_attn_grads *grads, void *workspace, size_t ws_bytes,
                                    ssd_stream_t stream);

/* One token of each of dims.nseq rows (dims.seqlen must be 1, dims.packed 0), against a cache of states
 * (nslots, nheads, headdim_k, headdim_v) fp32, updated in place: row r uses slot slot_idx[r] (slot_idx NULL: slot
 * r).  A row whose slot is outside [0, nslots) leaves the cache alone and writes zeros to its o; no two rows may
 * share a slot (which of them would win is undefined).  in->initial_states and in->cu_seqlens must be NULL.  o must
 * not overlap an input, as in the forward pass.  No workspace. */
ssd_status ssd_linear_attn_step(const ssd_linear_attn_dims *dims, const ssd_linear_attn_inputs *in, float *states,
                                int32_t nslots, const int32_t *slot_idx, void *o, int64_t o_tok_stride,
                                ssd_stream_t stream);

/* Group norm with an activation, channels last.  x (nsamples, nrows, channels): row r of sample n is row
 * n * nrows + r of a row-major tensor with its own row stride (channels contiguous).  Per sample and group of
 * channels / groups consecutive channels, over its nrows * channels / groups values:
 *     u = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(var + eps)   (var: the mean squared deviation)
 *     y = u (SSD_ACT_NONE), u sigmoid(u) (SSD_ACT_SILU), u z sigmoid(z) (SSD_ACT_GATE, z a tensor like x)
 * nrows = 1 is the norm of each head of each token that retention uses.  weight and bias (channels) fp32, or NULL
 * (1 and 0).  Row strides below 2^31 elements.  mean and rstd (nsamples, groups) fp32 are written by the forward pass (each may be NULL) and read by
 * the backward pass.  Any number of channels per group; rows of 16-byte aligned tensors whose strides and group
 * widths are multiples of 8 elements move as 16-byte vectors, even ones two elements at a time, others one by one.
 * Statistics are summed in fp32 as deviations (no difference of large sums).  y may be x or z itself, with its row stride; gradients must not
 * overlap what the backward pass reads (tiles are read twice): what starts where an input does is refused otherwise
 * (SSD_ERR_INVALID_DIMS). */
typedef enum { SSD_ACT_NONE = 0, SSD_ACT_SILU = 1, SSD_ACT_GATE = 2 } ssd_activation;

typedef struct {
  int32_t nsamples, nrows, channels, groups;
  int32_t dtype;      /* ssd_dtype of x, z, y and their gradients */
  int32_t activation; /* ssd_activation */
} ssd_group_norm_dims;

typedef struct {
  const void *x; int64_t x_row_stride;
  const void *z; int64_t z_row_stride; /* exactly with SSD_ACT_GATE */
  const float *weight, *bias;
  float eps;
} ssd_group_norm_inputs;

/* Gradients, written (not accumulated); dz exactly with SSD_ACT_GATE; dweight and dbias may be NULL. */
typedef struct {
  void *dx; int64_t dx_row_stride;
  void *dz; int64_t dz_row_stride;
  float *dweight, *dbias;
} ssd_group_norm_grads;

size_t ssd_group_norm_workspace_size(const ssd_group_norm_dims *dims, int backward);

ssd_status ssd_group_norm_forward(const ssd_group_norm_dims *dims, const ssd_group_norm_inputs *in, void *y,
                                  int64_t y_row_stride, float *mean, float *rstd, void *workspace, size_t ws_bytes,
                                  ssd_stream_t stream);

ssd_status ssd_group_norm_backward(const ssd_group_norm_dims *dims, const ssd_group_norm_inputs *in, const void *dy,
                                   int64_t dy_row_stride, const float *mean, const float *rstd,
                                   const ssd_group_norm_grads *grads, void *workspace, size_t ws_bytes,
                                   ssd_stream_t stream);

/* ======================= the gated delta rule, and the norms around a block
 *
 * Gated delta rule.  Per state head h, with a_t = exp(log_decay_t), b_t = beta_t and the rows k and q of head
 * h / (nheads / nheads_qk), for the tokens t of one sequence in order:
 *     S' = a_t S_{t-1},   S_t = S' + b_t k_t^T (v_t - k_t S')     (headdim_k x headdim_v; S_{-1}: the initial state, or zero)
 *     o_t = scale q_t S_t
 * With dims.qk_norm, q and k are divided by sqrt(|.|^2 + norm_eps) first (gradients go through the division); without
 * it the keys should be short (b |k|^2 at most 2), or states grow from token to token.
 * Sequences, cu_seqlens, empty sequences and rows outside every sequence are as in ssd_linear_attn_dims (with bounds out
 * of order what any sequence but an empty one gets is undefined, and stays inside the tensors), and so are the layouts:
 * token-major tensors with their own token strides, heads and channels contiguous within a token,
 *   q, k (T, nheads_qk * headdim_k), v, o (T, nheads * headdim_v), log_decay, beta (T, nheads)
 * all in dims.dtype; q, k, v, o 16-byte aligned with strides a multiple of 8 (bf16) or 4 (fp32) elements, log_decay and
 * beta element aligned with any stride of at least nheads.  log_decay is at most 0 (below -256 it counts as -256, which
 * forgets everything; -inf is allowed).  States (nseq, nheads, headdim_k, headdim_v) fp32, contiguous, 16-byte aligned.
 * Arithmetic: fp32.  bf16 tensors with both widths at most 128 take products of bf16 operands with fp32 sums; what ends in
 * a state or an output is a sum of products of two bf16 terms each (states within about 3e-6 of their size; fp32 tensors:
 * 3e-7; outputs within their one rounding, 0.0017), operands of gradients are rounded once (0.004).  Where keys are nearly
 * equal, additions cancel and errors add up: states 2e-5, gradients 0.01; with beta |k|^2 near 2 as well, where the rule itself
 * magnifies errors, 1e-3 and 0.02 (fp32 tensors: 2e-5 and 4e-5).
 * A NaN or infinity in a token can reach every output of the same 64-token chunk of its own sequence and head, and those
 * of later tokens (gradients: of all tokens); other sequences are not affected.
 * Envelope: headdim_k and headdim_v multiples of 8, at most 256; otherwise as linear attention, else
 * SSD_ERR_UNSUPPORTED.  All sums have a fixed order: equal inputs give equal bits. */
typedef struct {
  int32_t nseq;
  int32_t seqlen;       /* tokens of every sequence; ignored when packed */
  int32_t total_tokens; /* packed: rows of the token-major tensors; else 0 or nseq * seqlen */
  int32_t packed;       /* 1: cu_seqlens gives the sequences */
  int32_t nheads, nheads_qk, headdim_k, headdim_v;
  int32_t dtype;   /* ssd_dtype of q, k, v, log_decay, beta, o and their gradients */
  int32_t qk_norm; /* 1: q and k of each head are divided by their length */
} ssd_delta_rule_dims;

typedef struct {
  const void *q; int64_t q_tok_stride;
  const void *k; int64_t k_tok_stride;
  const void *v; int64_t v_tok_stride;
  const void *log_decay; int64_t log_decay_tok_stride;
  const void *beta; int64_t beta_tok_stride;
  const float *initial_states; /* or NULL: zero */
  const int32_t *cu_seqlens;   /* exactly when dims.packed */
  float scale;
  float norm_eps; /* with qk_norm: at least 0 */
} ssd_delta_rule_inputs;

/* Gradients, written (not accumulated), layout rules of the tensors they belong to, own token strides; dq and dk are
 * summed over the states that share a head.  dinitial_states fp32: written when not NULL (it does not need
 * initial_states to be given). */
typedef struct {
  void *dq; int64_t dq_tok_stride;
  void *dk; int64_t dk_tok_stride;
  void *dv; int64_t dv_tok_stride;
  void *dlog_decay; int64_t dlog_decay_tok_stride;
  void *dbeta; int64_t dbeta_tok_stride;
  float *dinitial_states;
} ssd_delta_rule_grads;

/* Bytes of device workspace of ssd_delta_rule_forward (backward = 0) or _backward (1); 0 if dims are invalid. */
size_t ssd_delta_rule_workspace_size(const ssd_delta_rule_dims *dims, int backward);

/* Forward.  final_states: the state after each sequence's last token, or NULL; it may be initial_states itself, which
 * are then updated in place.  Outputs must not overlap each other or anything else that is read: one that starts where
 * an input or another output does is refused (SSD_ERR_INVALID_DIMS). */
ssd_status ssd_delta_rule_forward(const ssd_delta_rule_dims *dims, const ssd_delta_rule_inputs *in, void *o,
                                  int64_t o_tok_stride, float *final_states, void *workspace, size_t ws_bytes,
                                  ssd_stream_t stream);

/* Backward of <do, o> + <dfinal_states, final_states> (dfinal_states NULL: zero).  do is named dout here: layout rules
 * of o.  Nothing but the inputs is needed from the forward pass.  Gradients must not overlap each other or what is read:
 * one that starts where an input or another gradient does is refused (SSD_ERR_INVALID_DIMS). */
ssd_status ssd_delta_rule_backward(const ssd_delta_rule_dims *dims, const ssd_delta_rule_inputs *in, const void *dout,
                                   int64_t dout_tok_stride, const float *dfinal_states,
                                   const ssd_delta_rule_grads *grads, void *workspace, size_t ws_bytes,
                                   ssd_stream_t stream);

/* One token of each of dims.nseq rows (dims.seqlen must be 1, dims.packed 0), against a cache of states (nslots, nheads,
 * headdim_k, headdim_v) fp32, updated in place: slots, rows without one, and refusals are those of
 * ssd_linear_attn_step; o and the cache are refused where they meet each other or an input, too.  No workspace. */
ssd_status ssd_delta_rule_step(const ssd_delta_rule_dims *dims, const ssd_delta_rule_inputs *in, float *states,
                               int32_t nslots, const int32_t *slot_idx, void *o, int64_t o_tok_stride,
                               ssd_stream_t stream);

/* Block norm: the norms behind and before a block, joined with its gate, its scale and the residual stream.  Per row of
 * `channels` values, rms(v) = sqrt(mean of v^2 + eps):
 *     u = x / rms(x) * post_weight          (dims.post_norm; else u = x)
 *     t = u z sigmoid(z)                    (dims.gate, z a tensor like x; else t = u)
 *     h = residual + branch_scale t         (dims.residual; else h = branch_scale t)
 *     y = h / rms(h) * pre_weight           (dims.pre_norm: the input of the next block)
 * x, z, y in dims.dtype, residual and h in dims.residual_dtype (that of x, or fp32), rows with their own strides
 * (channels contiguous), element aligned; tensors that are 16-byte aligned with strides and channels a multiple of 8
 * move as 16-byte vectors, even ones two elements at a time, others one by one.  post_weight, branch_scale, pre_weight
 * (channels) fp32, or NULL (1).  y is made of h before it is rounded.
 * h: may be NULL with pre_norm, and may be the residual itself, with its stride (the stream updated in place); other
 * outputs that start where an input or another output does are refused (SSD_ERR_INVALID_DIMS).  rstd_post (rows) and rstd_pre (rows) fp32,
 * 1 / rms, are written with their norm, each may be NULL; the backward pass reads them.
 * Envelope: at most 16384 channels and 2^30 rows, row strides below 2^31 elements; else SSD_ERR_UNSUPPORTED.  All sums
 * have a fixed order. */
typedef struct {
  int32_t rows, channels;
  int32_t dtype;          /* ssd_dtype of x, z, y and their gradients */
  int32_t residual_dtype; /* ssd_dtype of residual, h and their gradients */
  int32_t post_norm, gate, residual, pre_norm; /* each 0 or 1 */
} ssd_block_norm_dims;

typedef struct {
  const void *x; int64_t x_row_stride;
  const void *z; int64_t z_row_stride;               /* exactly with dims.gate */
  const void *residual; int64_t residual_row_stride; /* forward: exactly with dims.residual; backward: NULL */
  const float *post_weight;  /* NULL without post_norm */
  const float *branch_scale;
  const float *pre_weight;   /* NULL without pre_norm */
  float eps;
} ssd_block_norm_inputs;

/* What the backward pass reads besides the inputs.  h: the forward pass's h (without post_norm, gate, residual and
 * branch_scale that is x, of the same type), needed with pre_norm.  dh: the gradient of h from elsewhere, or NULL
 * (zero).  dy: the gradient of y, exactly with pre_norm. */
typedef struct {
  const void *h; int64_t h_row_stride;
  const void *dh; int64_t dh_row_stride;
  const void *dy; int64_t dy_row_stride;
  const float *rstd_post, *rstd_pre;
} ssd_block_norm_saved;

/* Gradients, written (not accumulated).  dz exactly with dims.gate, dresidual exactly with dims.residual; dresidual may
 * be dh itself, with its stride; else rows' gradients that start where an input does, and any two that start at the same
 * place, are refused (SSD_ERR_INVALID_DIMS).  Parameter gradients (channels) fp32, each may be NULL; dpost_weight only with
 * post_norm, dpre_weight only with pre_norm. */
typedef struct {
  void *dx; int64_t dx_row_stride;
  void *dz; int64_t dz_row_stride;
  void *dresidual; int64_t dresidual_row_stride;
  float *dpost_weight, *dbranch_scale, *dpre_weight;
} ssd_block_norm_grads;

/* Bytes of device workspace of ssd_block_norm_backward; the forward pass needs none. */
size_t ssd_block_norm_workspace_size(const ssd_block_norm_dims *dims);

ssd_status ssd_block_norm_forward(const ssd_block_norm_dims *dims, const ssd_block_norm_inputs *in, void *h,
                                  int64_t h_row_stride, void *y, int64_t y_row_stride, float *rstd_post,
                                  float *rstd_pre, ssd_stream_t stream);

ssd_status ssd_block_norm_backward(const ssd_block_norm_dims *dims, const ssd_block_norm_inputs *in,
                                   const ssd_block_norm_saved *saved, const ssd_block_norm_grads *grads,
                                   void *workspace, size_t ws_bytes, ssd_stream_t stream);

/* Static description of a status code. */
const char *ssd_status_string(ssd_status status);

#ifdef __cplusplus
}
#endif
#endif /* SSD_H */
