"""The operators of a gated delta rule block as cases to measure: the delta rule with a decay and a write strength for
each token (prompt, gradients, single tokens), and the norms before and after a block joined with its gate, its
scale and the residual stream (forward, gradients).

Each case runs in one of two forms on the same inputs: the plain form, in elementary torch operations in 32 bits,
and the framework's own entry points.

Notation: T tokens of n sequences, H heads with a state each, K heads of q and k (each shared by H / K states),
a_t = exp(log_decay_t), b_t = beta_t, k a row:
    S' = a_t S_(t-1),   S_t = S' + b_t k_t^T (v_t - k_t S'),   o_t = scale q_t S_t          (S: dk x dv)
with q and k divided by their length where qk_norm says so.
"""
import math
import random

import torch

own = False  # True: the framework's entry points; False: the plain form

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64  # tokens per block of the plain form
_QK_EPS = 1e-6
_EPS = 1e-6


# ------------------------------------------------------------------ cases

def _dr(op, name, n, tokens, heads, qk, dk, dv, dtype="bf16", packed=False, init=False, norm=True):
    """tokens: of each sequence, or of all sequences together when packed."""
    return {"name": name, "op": op, "n": n, "tokens": tokens, "heads": heads, "qk": qk, "dk": dk, "dv": dv,
            "dtype": dtype, "packed": packed, "init": init, "norm": norm}


def _step(name, rows, slots, heads, qk, dk, dv, dtype="bf16", norm=True):
    return {"name": name, "op": "dr_step", "rows": rows, "slots": slots, "heads": heads, "qk": qk, "dk": dk, "dv": dv,
            "dtype": dtype, "norm": norm}


def _bn(op, name, rows, channels, post, gate, residual, scaled, pre, dtype="bf16", res="bf16"):
    return {"name": name, "op": op, "rows": rows, "channels": channels, "post": post, "gate": gate,
            "residual": residual, "scaled": scaled, "pre": pre, "dtype": dtype, "res": res}


def listed():
    return [
        # a short prompt of one user: latency
        _dr("dr_forward", "delta_short", 1, 77, 8, 8, 64, 64),
        # one long document, few heads: there is little to do side by side
        _dr("dr_forward", "delta_long", 1, 16411, 16, 8, 128, 128),
        # a training batch's forward
        _dr("dr_forward", "delta_batch", 4, 8192, 32, 16, 128, 128),
        # prompts of different lengths packed into one row, continued from cached states
        _dr("dr_forward", "delta_packed", 24, 16384, 16, 4, 64, 128, packed=True, init=True),
        # a training step's backward
        _dr("dr_backward", "delta_grad", 2, 8192, 32, 16, 128, 128),
        # fine-tuning in 32 bits on packed samples
        _dr("dr_backward", "delta_grad_f32", 7, 5003, 12, 4, 64, 64, dtype="f32", packed=True, init=True),
        # one user's next token
        _step("delta_token", 1, 4, 16, 16, 64, 64),
        # a serving batch's next token, states in a larger cache
        _step("delta_tokens", 256, 320, 32, 16, 128, 128),
        # a block's output normed, gated, scaled, added to the stream, and the stream normed for the next block
        _bn("bn_forward", "join_batch", 16384, 4096, True, True, True, True, True),
        # one user's next token: a block's output added to a stream of 32 bits, and the norm of the next block
        _bn("bn_forward", "join_token", 1, 2048, False, False, True, False, True, res="f32"),
        # gradients of the whole join, the stream in 32 bits
        _bn("bn_backward", "join_grad", 8192, 4096, True, True, True, True, True, res="f32"),
        # gradients in 32 bits, odd sizes, no norm on the block's output
        _bn("bn_backward", "join_grad_f32", 3001, 1003, False, False, True, True, True, dtype="f32", res="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dr_forward", "dr_forward", "dr_backward", "dr_step", "bn_forward", "bn_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("bn"):
        res = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        channels = rng.choice([_log_int(rng, 24, 6000), 8 * _log_int(rng, 8, 1024)])
        rows = _log_int(rng, 1, min(30000, 8192 * 4096 // channels // (2 if dtype == "f32" else 1)))
        post, gate = rng.random() < 0.5, rng.random() < 0.5
        case = _bn(op, "", rows, channels, post, gate, rng.random() < 0.8, rng.random() < 0.5,
                   not (post or gate) or rng.random() < 0.8, dtype, res)
    else:
        dk, dv = (8 * _log_int(rng, 3, 16) for _ in range(2))
        if rng.random() < 0.6:
            dk, dv = rng.choice([(64, 64), (128, 128), (64, 128), (128, 64)])
        heads = rng.choice([1, 2, 4, 6, 8, 12, 16, 32])
        qk = heads // rng.choice([d for d in (1, 1, 2, 3, 4) if heads % d == 0])
        norm = rng.random() < 0.7
        if op == "dr_step":
            rows = _log_int(rng, 1, 256)
            case = _step("", rows, rows + rng.randrange(20), heads, qk, dk, dv, dtype, norm)
        else:
            # 32-bit sequences and backward passes are shorter: their plain form and their arithmetic cost more
            budget = 32768 * 32 * 256 // (8 if dtype == "f32" else 4 if op == "dr_backward" else 1)
            most = max(64, min(16384 if op == "dr_forward" else 8192, budget // (heads * (dk + dv))))
            total = _log_int(rng, 1, most)
            packed = rng.random() < 0.4 and total >= 4
            n = _log_int(rng, 2, min(48, total)) if packed else _log_int(rng, 1, min(8, total))
            case = _dr(op, "", n, total if packed else max(1, total // n), heads, qk, dk, dv, dtype, packed,
                       rng.random() < 0.5, norm)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _lengths(case, seed):
    if not case["packed"]:
        return [case["tokens"]] * case["n"]
    r = random.Random(seed * 7919 + 29)
    n, total = case["n"], case["tokens"]
    # sequences of very different lengths, one of a single token
    cuts = sorted(r.randint(0, total - 1) for _ in range(n - 1)) if n > 1 else []
    if n > 2:
        cuts[0] = 1
        cuts.sort()
    cuts = [0] + cuts + [total]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 31)
    tt = _TYPES[case["dtype"]]

    def rand(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        out = torch.empty(*shape, dtype=dtype, device="cuda")
        out.normal_(generator=gen)
        if scale != 1.0:
            out.mul_(scale)
        if shift:
            out.add_(shift)
        return out

    s = {"case": dict(case), "op": case["op"]}
    if case["op"].startswith("bn"):
        rows, c, rt = case["rows"], case["channels"], _TYPES[case["res"]]
        s["x"] = rand(rows, c, dtype=tt, scale=1.5)
        s["z"] = rand(rows, c, dtype=tt) if case["gate"] else None
        s["post_weight"] = rand(c, scale=0.25, shift=1.0) if case["post"] else None
        s["branch_scale"] = rand(c, scale=0.1, shift=0.5) if case["scaled"] else None
        s["pre_weight"] = rand(c, scale=0.25, shift=1.0) if case["pre"] else None
        if case["op"] == "bn_forward":
            s["residual"] = rand(rows, c, dtype=rt, scale=2.0) if case["residual"] else None
        else:
            # what the forward pass kept: the stream behind the join, and 1 / rms of the block's output and of the stream
            s["h"] = rand(rows, c, dtype=rt, scale=2.0)
            s["dh"] = rand(rows, c, dtype=rt)
            s["dy"] = rand(rows, c, dtype=tt) if case["pre"] else None
            rms = lambda t: torch.cat([p.double().square().mean(1).add(_EPS).rsqrt().float() for p in t.split(4096)])  # noqa: E731
            s["rstd_post"] = rms(s["x"]) if case["post"] else None
            s["rstd_pre"] = rms(s["h"]) if case["pre"] else None
        if own:
            import mamba2_ssd_selective_gb300 as ssd

            s["runner"] = ssd.BlockNormRunner(rows, c, post_norm=case["post"], gate=case["gate"],
                                              residual=case["residual"], pre_norm=case["pre"], dtype=case["dtype"],
                                              residual_dtype=case["res"])
        return s
    h, qk, dk, dv = case["heads"], case["qk"], case["dk"], case["dv"]
    s["scale"] = 1.0 if case["norm"] else dk ** -0.5

    def tokens(total):
        # q, k and v are parts of a projection's output behind a SiLU, the two numbers of each head of another's: views
        # with its row stride
        qkv = rand(total, 2 * qk * dk + h * dv, dtype=tt)
        qkv.mul_(torch.sigmoid(qkv))
        s["q"], s["k"], s["v"] = qkv.split([qk * dk, qk * dk, h * dv], dim=1)
        s["log_decay"], s["beta"] = rand(total, 2 * h, dtype=tt).split([h, h], dim=1)
        if not case["norm"]:  # a model without the division keeps its keys short by other means
            s["k"].mul_(1.4 * dk ** -0.5)
        # log decays -A softplus(dt): A up to 16 over the heads, softplus(dt) from 0.001 to 0.1 about its bias
        big = torch.empty(h, device="cuda").uniform_(0.0, 16.0, generator=gen)
        bias = torch.exp(torch.empty(h, device="cuda").uniform_(math.log(1e-3), math.log(0.1), generator=gen))
        dt = torch.nn.functional.softplus(0.5 * s["log_decay"].float() + torch.log(torch.expm1(bias)))
        s["log_decay"].copy_(-big * dt)
        s["beta"].copy_(torch.sigmoid(s["beta"].float()))

    if case["op"] == "dr_step":
        rows, slots = case["rows"], case["slots"]
        tokens(rows)
        s["state"] = rand(slots, h, dk, dv, scale=0.3)
        s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:rows].to(torch.int32)
        if own:
            import mamba2_ssd_selective_gb300 as ssd

            s["runner"] = ssd.DeltaRuleRunner(rows, 1, h, dk, dv, nheads_qk=qk, qk_norm=case["norm"],
                                              dtype=case["dtype"])
        return s
    lens = _lengths(case, int(seed))
    n, total = len(lens), sum(lens)
    tokens(total)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["max_len"] = max(lens)
    s["init"] = rand(n, h, dk, dv, scale=0.3) if case["init"] else None
    if case["op"] == "dr_backward":
        s["do"] = rand(total, h * dv, dtype=tt)
        s["dfinal"] = rand(n, h, dk, dv) if case["init"] else None
    if own:
        import mamba2_ssd_selective_gb300 as ssd

        s["runner"] = ssd.DeltaRuleRunner(n, case["tokens"], h, dk, dv, nheads_qk=qk, qk_norm=case["norm"],
                                          dtype=case["dtype"], packed=case["packed"])
    return s


# ------------------------------------------------------------------ plain form

def _pad(x, s, heads):
    """(total, heads * d) rows -> (n, H, chunks, 64, d) in 32 bits, zeros past each sequence; heads are repeated up to H."""
    case, cu = s["case"], s["cu"].long()
    top = -(-s["max_len"] // _CHUNK) * _CHUNK
    rows = cu[:-1, None] + torch.arange(top, device="cuda")
    live = rows < cu[1:, None]
    x = x[rows.clamp(max=x.shape[0] - 1)].float() * live[..., None]
    x = x.view(*rows.shape, heads, -1).transpose(1, 2)
    x = x.repeat_interleave(case["heads"] // heads, dim=1)
    return x.reshape(*x.shape[:2], top // _CHUNK, _CHUNK, x.shape[-1])


def _unpad(x, s, heads, dtype):
    """(n, H, chunks, 64, d) -> (total, heads * d), summed over the states that share a head, rounded once."""
    cu, total = s["cu"].long(), s["q"].shape[0]
    tok = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu[1:], tok, right=True)
    n, h, nc, _, d = x.shape
    x = x.reshape(n, heads, h // heads, nc * _CHUNK, d).sum(2)
    return x[seq, :, tok - cu[seq]].reshape(total, heads * d).to(dtype)


def _short(x, s):
    """x / |x| and 1 / |x|, or x and 1."""
    if not s["case"]["norm"]:
        return x, torch.ones_like(x[..., :1])
    r = (x.square().sum(-1, keepdim=True) + _QK_EPS).rsqrt()
    return x * r, r


def _unit_inverse(low):
    """The inverse of I + low, low strictly lower triangular (.., 64, 64): inverses of diagonal blocks, doubled in size."""
    inv = torch.eye(_CHUNK, device="cuda").expand_as(low).contiguous()
    size = 1
    while size < _CHUNK:
        for at in range(0, _CHUNK, 2 * size):
            a, b = slice(at, at + size), slice(at + size, at + 2 * size)
            inv[..., b, a] = -(inv[..., b, b] @ low[..., b, a] @ inv[..., a, a])
        size *= 2
    return inv


def _chunks(s):
    """Everything of the chunks that does not depend on a state."""
    case = s["case"]
    c = {"beta": _pad(s["beta"], s, case["heads"]), "v": _pad(s["v"], s, case["heads"])}
    c["q"], c["rq"] = _short(_pad(s["q"], s, case["qk"]), s)
    c["k"], c["rk"] = _short(_pad(s["k"], s, case["qk"]), s)
    g = _pad(s["log_decay"], s, case["heads"]).double().cumsum(-2)
    gap = g - g.transpose(-1, -2)
    i = torch.arange(_CHUNK, device="cuda")
    c["with"] = torch.where(i[:, None] >= i, torch.exp(gap).float(), 0.0)  # decay from j to i, j <= i
    c["past"] = torch.where(i[:, None] > i, c["with"], 0.0)
    c["in"], c["out"], c["all"] = torch.exp(g).float(), torch.exp(g[..., -1:, :] - g).float(), torch.exp(g[..., -1:, :]).float()
    c["kk"] = c["k"] @ c["k"].transpose(-1, -2) * c["past"]
    c["qk"] = c["q"] @ c["k"].transpose(-1, -2) * c["with"] * s["scale"]
    return c


def _states(s, c):
    """States before each chunk and behind the last, (n, H, chunks + 1, dk, dv), and E: what each token adds, before beta."""
    case, nc = s["case"], c["k"].shape[2]
    inv = _unit_inverse(c["kk"] * c["beta"].transpose(-1, -2))
    w, e = inv @ (c["k"] * c["in"]), inv @ c["v"]
    kt = (c["k"] * c["out"] * c["beta"]).transpose(-1, -2)
    n, h = e.shape[:2]
    states = torch.empty(n, h, nc + 1, case["dk"], case["dv"], device="cuda")
    states[:, :, 0] = 0.0 if s["init"] is None else s["init"]
    for i in range(nc):
        e[:, :, i] -= w[:, :, i] @ states[:, :, i]
        states[:, :, i + 1] = states[:, :, i] * c["all"][:, :, i] + kt[:, :, i] @ e[:, :, i]
    return states, e


def _plain_forward(s):
    c = _chunks(s)
    states, e = _states(s, c)
    o = (c["q"] * c["in"] * s["scale"]) @ states[:, :, :-1] + c["qk"] @ (e * c["beta"])
    return {"o": _unpad(o, s, s["case"]["heads"], s["q"].dtype), "final_state": states[:, :, -1].contiguous()}


def _plain_backward(s):
    case, c = s["case"], _chunks(s)
    states, e = _states(s, c)
    beta, nc = c["beta"], e.shape[2]
    do = _pad(s["do"], s, case["heads"])
    d = e * beta
    # Z: the gradient of each token's addition, with what later tokens of its chunk take from it
    back = _unit_inverse(c["kk"] * beta).transpose(-1, -2)
    z = back @ (c["qk"].transpose(-1, -2) @ do)
    kz = back @ (c["k"] * c["out"])
    qt, kt = (c["q"] * c["in"] * s["scale"]).transpose(-1, -2), (c["k"] * c["in"] * beta).transpose(-1, -2)
    grads = torch.empty_like(states)  # of the state before each chunk and behind the last
    grads[:, :, nc] = 0.0 if s["dfinal"] is None else s["dfinal"]
    made = qt @ do
    for i in reversed(range(nc)):
        z[:, :, i] += kz[:, :, i] @ grads[:, :, i + 1]
        grads[:, :, i] = grads[:, :, i + 1] * c["all"][:, :, i] + made[:, :, i] - kt[:, :, i] @ z[:, :, i]
    dv = z * beta
    dqk = do @ d.transpose(-1, -2) * c["with"] * s["scale"]
    dkk = -(dv @ d.transpose(-1, -2)) * c["past"]
    dq = (do @ states[:, :, :-1].transpose(-1, -2)) * c["in"] * s["scale"] + dqk @ c["k"]
    dk = (d @ grads[:, :, 1:].transpose(-1, -2)) * c["out"] - (dv @ states[:, :, :-1].transpose(-1, -2)) * c["in"]
    dk = dk + dqk.transpose(-1, -2) @ c["q"] + dkk @ c["k"] + dkk.transpose(-1, -2) @ c["k"]
    # a log decay at token t: everything that passes from before t to t and later
    per = (c["q"] * dq).sum(-1, keepdim=True) - (c["v"] * dv).sum(-1, keepdim=True)
    end = (states[:, :, 1:] * grads[:, :, 1:]).sum((-1, -2))[..., None, None]
    dg = per.flip(-2).cumsum(-2).flip(-2) + end
    out = {"dv": _unpad(dv, s, case["heads"], s["q"].dtype), "dlog_decay": _unpad(dg, s, case["heads"], s["q"].dtype),
           "dbeta": _unpad((e * z).sum(-1, keepdim=True), s, case["heads"], s["q"].dtype)}
    if case["norm"]:
        dq = (dq - c["q"] * (c["q"] * dq).sum(-1, keepdim=True)) * c["rq"]
        dk = (dk - c["k"] * (c["k"] * dk).sum(-1, keepdim=True)) * c["rk"]
    out["dq"], out["dk"] = _unpad(dq, s, case["qk"], s["q"].dtype), _unpad(dk, s, case["qk"], s["q"].dtype)
    if s["init"] is not None:
        out["dinitial_state"] = grads[:, :, 0].contiguous()
    return out


def _plain_step(s):
    case, state, at = s["case"], s["state"], s["slots"].long()
    rows, h, qk = case["rows"], case["heads"], case["qk"]
    q, k = (_short(s[x].float().view(rows, qk, 1, -1).repeat_interleave(h // qk, dim=1), s)[0] for x in ("q", "k"))
    v, beta, g = s["v"].float().view(rows, h, 1, -1), s["beta"].float().view(rows, h, 1, 1), s["log_decay"].float().view(rows, h, 1, 1)
    old = state[at] * torch.exp(g)
    new = old + k.transpose(-1, -2) * (beta * (v - k @ old))
    state[at] = new
    return {"o": (q @ new * s["scale"]).to(s["q"].dtype).view(rows, -1), "state": state}


def _branch(s):
    """The block's output on its way to the stream, in 32 bits: (normed, gated, scaled)."""
    x = s["x"].float()
    if s["case"]["post"]:
        rstd = s["rstd_post"] if "rstd_post" in s else (x.square().mean(1) + _EPS).rsqrt()
        x = x * rstd[:, None] * s["post_weight"]
    gated = x if s["z"] is None else x * (s["z"].float() * torch.sigmoid(s["z"].float()))
    scaled = gated if s["branch_scale"] is None else gated * s["branch_scale"]
    return x, gated, scaled


def _plain_bn_forward(s):
    case = s["case"]
    h = _branch(s)[2]
    if s["residual"] is not None:
        h = h + s["residual"].float()
    out = {"h": h.to(_TYPES[case["res"]])}
    if case["post"]:
        out["rstd_post"] = (s["x"].float().square().mean(1) + _EPS).rsqrt()
    if case["pre"]:
        out["rstd_pre"] = (h.square().mean(1) + _EPS).rsqrt()
        out["y"] = (h * out["rstd_pre"][:, None] * s["pre_weight"]).to(s["x"].dtype)
    return out


def _norm_back(du, x, rstd):
    """Gradient of x through x rstd, du that of the normed value."""
    n = x * rstd[:, None]
    return (du - n * (du * n).mean(1, keepdim=True)) * rstd[:, None]


def _plain_bn_backward(s):
    case, out = s["case"], {}
    dh = s["dh"].float()
    if case["pre"]:
        h, dy = s["h"].float(), s["dy"].float()
        out["dpre_weight"] = (dy * h * s["rstd_pre"][:, None]).sum(0)
        dh = dh + _norm_back(dy * s["pre_weight"], h, s["rstd_pre"])
    if case["residual"]:
        out["dresidual"] = dh.to(s["dh"].dtype)
    normed, gated, _ = _branch(s)
    if case["scaled"]:
        out["dbranch_scale"] = (dh * gated).sum(0)
        dh = dh * s["branch_scale"]
    if case["gate"]:
        z = s["z"].float()
        p = torch.sigmoid(z)
        out["dz"] = (dh * normed * (p * (1 + z * (1 - p)))).to(s["x"].dtype)
        dh = dh * (z * p)
    if case["post"]:
        x = s["x"].float()
        out["dpost_weight"] = (dh * x * s["rstd_post"][:, None]).sum(0)
        dh = _norm_back(dh * s["post_weight"], x, s["rstd_post"])
    out["dx"] = dh.to(s["x"].dtype)
    return out


_PLAIN = {"dr_forward": _plain_forward, "dr_backward": _plain_backward, "dr_step": _plain_step,
          "bn_forward": _plain_bn_forward, "bn_backward": _plain_bn_backward}


# ------------------------------------------------------------------ one pass

def run(s):
    if not own:
        return _PLAIN[s["op"]](s)
    r, op = s["runner"], s["op"]
    if op == "dr_forward":
        o, final = r.forward(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], scale=s["scale"],
                             initial_state=s["init"], cu_seqlens=s["cu"] if s["case"]["packed"] else None)
        return {"o": o, "final_state": final}
    if op == "dr_backward":
        g = r.backward(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["do"], scale=s["scale"],
                       initial_state=s["init"], dfinal_state=s["dfinal"],
                       cu_seqlens=s["cu"] if s["case"]["packed"] else None)
    elif op == "dr_step":
        o = r.step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["state"], slot_idx=s["slots"],
                   scale=s["scale"])
        return {"o": o, "state": s["state"]}
    elif op == "bn_forward":
        g = r.forward(s["x"], residual=s["residual"], z=s["z"], post_weight=s["post_weight"],
                      branch_scale=s["branch_scale"], pre_weight=s["pre_weight"], eps=_EPS)
    else:
        g = r.backward(s["x"], s["h"], dh=s["dh"], dy=s["dy"], z=s["z"], post_weight=s["post_weight"],
                       branch_scale=s["branch_scale"], pre_weight=s["pre_weight"], rstd_post=s["rstd_post"],
                       rstd_pre=s["rstd_pre"])
    return {k: v for k, v in g.items() if v is not None}


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("bn"):
        size, rs = case["rows"] * case["channels"], 2 if case["res"] == "bf16" else 4
        post, gate, res, pre = (int(case[x]) for x in ("post", "gate", "residual", "pre"))
        if case["op"] == "bn_forward":
            return {"bytes": size * (es * (1 + gate + pre) + rs * (1 + res)), "flops": size * (4 + 4 * post + 5 * gate + 4 * pre)}
        # x is read for its norm, the gate or the scale; the stream for its norm
        reads_x = int(post or gate or case["scaled"])
        return {"bytes": size * (es * (reads_x + 1 + 2 * gate + pre) + rs * (1 + res + pre)),
                "flops": size * (6 + 12 * post + 12 * gate + 10 * pre)}
    h, qk, dk, dv = case["heads"], case["qk"], case["dk"], case["dv"]
    if case["op"] == "dr_step":
        one = h * dk * dv
        return {"bytes": case["rows"] * (8 * one + es * (2 * qk * dk + 2 * h * dv + 2 * h)), "flops": 7 * case["rows"] * one}
    total = case["tokens"] * (1 if case["packed"] else case["n"])
    states = 4 * case["n"] * h * dk * dv
    if case["op"] == "dr_forward":
        return {"bytes": total * es * (2 * qk * dk + 2 * h * dv + 2 * h) + states * (2 if case["init"] else 1),
                "flops": 7 * total * h * dk * dv}
    # q, k, v, the output's gradient, the heads' numbers, and a gradient of each but the output's
    return {"bytes": total * es * (4 * qk * dk + 3 * h * dv + 4 * h) + (3 * states if case["init"] else 0),
            "flops": 21 * total * h * dk * dv}


# ------------------------------------------------------------------ 64 bits

class _Tokens:
    """The tensors of all sequences token by token, in 64 bits, heads repeated."""

    def __init__(self, s, case):
        cu = s["cu"].tolist()
        self.s, self.case = s, case
        self.lens = [b - a for a, b in zip(cu, cu[1:])]
        self.n, self.total, self.top = len(self.lens), cu[-1], max(self.lens)
        self.len_t = torch.tensor(self.lens, device="cuda")
        self.first = torch.tensor(cu[:-1], device="cuda")
        self.length = {}
        if case["norm"]:
            for x in ("q", "k"):
                p = s[x].double().reshape(self.total, case["qk"], -1)
                self.length[x] = torch.sqrt((p * p).sum(-1) + _QK_EPS)

    def at(self, x, t, heads):
        rows = (self.first + t).clamp(max=self.total - 1)
        v = self.s[x][rows].double().view(self.n, heads, -1)
        if x in self.length:
            v = v / self.length[x][rows][..., None]
        return v.repeat_interleave(self.case["heads"] // heads, dim=1)

    def put(self, out, t, val):
        if min(self.lens) > t:
            out[self.first + t] = val
        else:
            ok = (t < self.len_t).nonzero()[:, 0]
            out[self.first[ok] + t] = val[ok]

    def step(self, state, t):
        """(decayed state, error of its prediction, state after token t); sequences that have ended keep theirs."""
        h = self.case["heads"]
        k, v = self.at("k", t, self.case["qk"]), self.at("v", t, h)
        low = torch.exp(self.at("log_decay", t, h))[..., None] * state
        err = v - torch.einsum("nhk,nhkv->nhv", k, low)
        new = low + torch.einsum("nhk,nhv->nhkv", self.at("beta", t, h) * k, err)
        return low, err, torch.where((t < self.len_t).view(-1, 1, 1, 1), new, state)


def _exact_forward(s, case):
    tk = _Tokens(s, case)
    state = (s["init"].double() if s["init"] is not None else
             torch.zeros(tk.n, case["heads"], case["dk"], case["dv"], dtype=torch.float64, device="cuda"))
    o = torch.zeros(tk.total, case["heads"], case["dv"], dtype=torch.float64, device="cuda")
    for t in range(tk.top):
        state = tk.step(state, t)[2]
        tk.put(o, t, float(s["scale"]) * torch.einsum("nhk,nhkv->nhv", tk.at("q", t, case["qk"]), state))
    return {"o": o.view(tk.total, -1), "final_state": state}


def _exact_backward(s, case):
    tk = _Tokens(s, case)
    h, qk, dk, dv, scale = case["heads"], case["qk"], case["dk"], case["dv"], float(s["scale"])
    zeros = lambda *d: torch.zeros(tk.total, h, *d, dtype=torch.float64, device="cuda")  # noqa: E731
    state = s["init"].double() if s["init"] is not None else torch.zeros(tk.n, h, dk, dv, dtype=torch.float64, device="cuda")
    grad = s["dfinal"].double() if s["dfinal"] is not None else torch.zeros_like(state)
    every, kept = 64, []
    for t in range(tk.top):
        if t % every == 0:
            kept.append(state)
        state = tk.step(state, t)[2]
    out = {"q": zeros(dk), "k": zeros(dk), "v": zeros(dv), "g": zeros(1), "b": zeros(1)}
    for block in reversed(range(len(kept))):
        states, t0 = [kept[block]], block * every
        t1 = min(tk.top, t0 + every)
        for t in range(t0, t1):
            states.append(tk.step(states[-1], t)[2])
        for t in reversed(range(t0, t1)):
            live = (t < tk.len_t).view(-1, 1, 1, 1)
            low, err, new = tk.step(states[t - t0], t)
            q, k, do, b = tk.at("q", t, qk), tk.at("k", t, qk), tk.at("do", t, h), tk.at("beta", t, h)
            tk.put(out["q"], t, scale * torch.einsum("nhkv,nhv->nhk", new, do))
            g = grad + scale * torch.einsum("nhk,nhv->nhkv", q, do)
            kg = torch.einsum("nhk,nhkv->nhv", k, g)
            tk.put(out["b"], t, (kg * err).sum(-1, keepdim=True))
            tk.put(out["v"], t, b * kg)
            tk.put(out["k"], t, b * (torch.einsum("nhkv,nhv->nhk", g, err) - torch.einsum("nhkv,nhv->nhk", low, kg)))
            g = g - torch.einsum("nhk,nhv->nhkv", k, b * kg)
            tk.put(out["g"], t, (g * low).sum((-1, -2))[..., None])
            grad = torch.where(live, torch.exp(tk.at("log_decay", t, h))[..., None] * g, grad)
    res = {"dv": out["v"].view(tk.total, -1), "dlog_decay": out["g"].view(tk.total, h), "dbeta": out["b"].view(tk.total, h)}
    for x in ("q", "k"):
        d = out[x].view(tk.total, qk, h // qk, dk).sum(2)
        if case["norm"]:  # x / |x|: what points along x is lost
            unit = s[x].double().reshape(tk.total, qk, dk) / tk.length[x][..., None]
            d = (d - unit * (unit * d).sum(-1, keepdim=True)) / tk.length[x][..., None]
        res["d" + x] = d.reshape(tk.total, -1)
    if s["init"] is not None:
        res["dinitial_state"] = grad
    return res


def _exact_step(s, case):
    rows, h, qk = case["rows"], case["heads"], case["qk"]
    of = torch.arange(h, device="cuda") // (h // qk)
    q, k = (s[x].double().reshape(rows, qk, -1) for x in ("q", "k"))
    if case["norm"]:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + _QK_EPS) for x in (q, k))
    q, k, v = q[:, of], k[:, of], s["v"].double().view(rows, h, -1)
    state, at = s["state"].double(), s["slots"].long()
    low = torch.exp(s["log_decay"].double())[..., None, None] * state[at]
    err = v - torch.einsum("rhk,rhkv->rhv", k, low)
    state[at] = low + torch.einsum("rhk,rhv->rhkv", s["beta"].double()[..., None] * k, err)
    return {"o": float(s["scale"]) * torch.einsum("rhk,rhkv->rhv", q, state[at]).reshape(rows, -1), "state": state}


def _exact_bn(s, case):
    x, out = s["x"].double(), {}
    one = torch.ones(case["channels"], dtype=torch.float64, device="cuda")
    pw, sc, w = (one if s[k] is None else s[k].double() for k in ("post_weight", "branch_scale", "pre_weight"))
    z = None if s["z"] is None else s["z"].double()
    gate = one if z is None else z / (1 + torch.exp(-z))
    forward = case["op"] == "bn_forward"
    rp = torch.ones_like(x[:, :1])
    if case["post"]:
        rp = 1 / torch.sqrt((x ** 2).sum(1, keepdim=True) / case["channels"] + _EPS) if forward else s["rstd_post"].double()[:, None]
    u = x * rp * (pw if case["post"] else 1.0)
    if forward:
        h = u * gate * sc + (0.0 if s["residual"] is None else s["residual"].double())
        out["h"] = h
        if case["post"]:
            out["rstd_post"] = rp[:, 0]
        if case["pre"]:
            r = 1 / torch.sqrt((h ** 2).sum(1, keepdim=True) / case["channels"] + _EPS)
            out["rstd_pre"], out["y"] = r[:, 0], h * r * w
        return out
    d = s["dh"].double()
    if case["pre"]:
        hn, dy = s["h"].double() * s["rstd_pre"].double()[:, None], s["dy"].double()
        out["dpre_weight"] = (dy * hn).sum(0)
        p = dy * w
        d = d + s["rstd_pre"].double()[:, None] * (p - hn * ((p * hn).sum(1, keepdim=True) / case["channels"]))
    if case["residual"]:
        out["dresidual"] = d
    if case["scaled"]:
        out["dbranch_scale"] = (d * u * gate).sum(0)
    d = d * sc
    if z is not None:
        ez = torch.exp(-z)
        out["dz"] = d * u * (1 + ez + z * ez) / (1 + ez) ** 2
    d = d * gate
    if case["post"]:
        xn = x * rp
        out["dpost_weight"] = (d * xn).sum(0)
        p = d * pw
        d = rp * (p - xn * ((p * xn).sum(1, keepdim=True) / case["channels"]))
    out["dx"] = d
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("bn"):
        return _exact_bn(s, case)
    return {"dr_forward": _exact_forward, "dr_backward": _exact_backward, "dr_step": _exact_step}[case["op"]](s, case)
