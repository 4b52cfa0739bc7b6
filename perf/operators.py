"""The retention operators as cases to measure: linear attention with a decay for
each head (prompt, gradients, single tokens) and group norm with an activation.

Each case runs in one of two forms on the same inputs: the plain form, in elementary
torch operations in 32 bits, and the framework's own entry points.

Notation: T tokens of n sequences, H query heads, K key/value heads, lam_h = exp(log_decay_h):
    S_t = lam S_(t-1) + k_t^T v_t,   o_t = scale q_t S_t          (S: dk x dv)
"""
import math
import random

import torch

own = False  # True: the framework's entry points; False: the plain form

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 128  # tokens per block of the plain form


# ------------------------------------------------------------------ cases

def _la(op, name, n, tokens, heads, kv, dk, dv, dtype="bf16", packed=False, init=False):
    """tokens: of each sequence, or of all sequences together when packed."""
    return {"name": name, "op": op, "n": n, "tokens": tokens, "heads": heads, "kv": kv, "dk": dk, "dv": dv,
            "dtype": dtype, "packed": packed, "init": init}


def _step(name, rows, slots, heads, kv, dk, dv, dtype="bf16"):
    return {"name": name, "op": "la_step", "rows": rows, "slots": slots, "heads": heads, "kv": kv, "dk": dk, "dv": dv,
            "dtype": dtype}


def _gn(op, name, n, m, channels, groups, act, dtype="bf16"):
    return {"name": name, "op": op, "n": n, "m": m, "channels": channels, "groups": groups, "act": act, "dtype": dtype}


def listed():
    return [
        # a short prompt of one user: latency
        _la("la_forward", "prompt_short", 1, 61, 8, 8, 64, 64),
        # one long document, few heads: the work has to be split along the sequence
        _la("la_forward", "prompt_long", 1, 31991, 16, 16, 128, 128),
        # a training batch's forward, the framework's benchmark length
        _la("la_forward", "prompt_batch", 4, 8192, 32, 32, 128, 128),
        # prompts of different lengths packed into one row, shared key/value heads, continued from cached states
        _la("la_forward", "prompt_packed", 24, 16384, 16, 4, 64, 128, packed=True, init=True),
        # a training step's backward
        _la("la_backward", "grad_batch", 2, 8192, 32, 32, 128, 128),
        # fine-tuning in 32 bits on packed samples
        _la("la_backward", "grad_packed_f32", 7, 5003, 12, 4, 64, 64, dtype="f32", packed=True, init=True),
        # one user's next token
        _step("token_one", 1, 4, 16, 16, 64, 64),
        # a serving batch's next token, states in a larger cache
        _step("token_batch", 256, 320, 32, 32, 128, 128),
        # norm of each head behind the training batch's mixer, with its gate
        _gn("gn_forward", "norm_heads", 32768, 1, 4096, 32, "gate"),
        # norm over whole feature maps, 32 bits, odd row count
        _gn("gn_forward", "norm_maps_f32", 6, 4099, 320, 32, "silu", dtype="f32"),
        # backward of the norm of each head
        _gn("gn_backward", "norm_heads_grad", 16384, 1, 4096, 32, "gate"),
        # backward of a norm over feature maps
        _gn("gn_backward", "norm_maps_grad", 8, 2048, 512, 32, "silu"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["la_forward", "la_forward", "la_backward", "la_step", "gn_forward", "gn_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("gn"):
        while True:
            groups = rng.choice([1, 2, 5, 8, 16, 32])
            channels = groups * rng.choice([3, 10, 16, 24, 64, 96, 128, 256])
            m = 1 if rng.random() < 0.5 else _log_int(rng, 2, 5000)
            n = _log_int(rng, 1, 30000) if m == 1 else _log_int(rng, 1, 64)
            if n * m * channels * (2 if dtype == "f32" else 1) <= 32768 * 4096 // 2:
                break
        case = _gn(op, "", n, m, channels, groups, rng.choice(["none", "silu", "gate"]), dtype)
    else:
        dk, dv = (8 * _log_int(rng, 3, 16) for _ in range(2))
        if rng.random() < 0.5:
            dk = dv = rng.choice([64, 128])
        heads = rng.choice([1, 2, 4, 6, 8, 12, 16, 32])
        kv = heads // rng.choice([d for d in (1, 1, 1, 2, 3, 4) if heads % d == 0])
        if op == "la_step":
            rows = _log_int(rng, 1, 300)
            case = _step("", rows, rows + rng.randrange(20), heads, kv, dk, dv, dtype)
        else:
            # 32-bit sequences and backward passes are shorter: their plain form and their arithmetic cost more
            budget = 32768 * 32 * 256 // (8 if dtype == "f32" else 4 if op == "la_backward" else 1)
            most = max(64, min(60000, budget // (heads * (dk + dv))))
            total = _log_int(rng, 1, most)
            packed = rng.random() < 0.4 and total >= 4
            n = _log_int(rng, 2, min(48, total)) if packed else _log_int(rng, 1, min(8, total))
            case = _la(op, "", n, total if packed else max(1, total // n), heads, kv, dk, dv, dtype, packed,
                       rng.random() < 0.5)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _lengths(case, seed):
    if not case["packed"]:
        return [case["tokens"]] * case["n"]
    r = random.Random(seed * 7919 + 13)
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
    gen.manual_seed(int(seed) * 1000003 + 17)
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
    if case["op"].startswith("gn"):
        n, m, c = case["n"], case["m"], case["channels"]
        s["x"] = rand(n, m, c, dtype=tt, scale=1.5, shift=0.25)
        s["weight"] = rand(c, scale=0.25, shift=1.0)
        s["bias"] = rand(c, scale=0.25)
        s["z"] = rand(n, m, c, dtype=tt) if case["act"] == "gate" else None
        s["eps"] = 1e-5
        if case["op"] == "gn_backward":
            s["dy"] = rand(n, m, c, dtype=tt)
            # what the forward pass kept: each group's mean and 1 / sqrt(var + eps), summed in 64 bits and stored in 32
            xg = s["x"].view(n, m, case["groups"], -1)
            step = max(1, (1 << 27) // (m * c))
            mean = torch.cat([p.double().mean((1, 3)) for p in xg.split(step)])
            var = torch.cat([p.double().var((1, 3), unbiased=False) for p in xg.split(step)])
            s["mean"], s["rstd"] = mean.float(), (var + s["eps"]).rsqrt().float()
        if own:
            import mamba2_ssd_selective_gb300 as ssd

            s["runner"] = ssd.GroupNormRunner(n, m, c, case["groups"], case["act"], case["dtype"])
        return s
    h, kv, dk, dv = case["heads"], case["kv"], case["dk"], case["dv"]
    # decays of 1 - 2^-e, e from 2 to 12 over the heads: half-lives from 3 to 3000 tokens
    e = 2.0 + 10.0 * torch.rand(h, generator=gen, device="cuda")
    s["log_decay"] = torch.log1p(-torch.exp2(-e.sort().values))
    s["scale"] = dk ** -0.5
    if case["op"] == "la_step":
        rows, slots = case["rows"], case["slots"]
        qkv = rand(rows, (h + kv) * dk + kv * dv, dtype=tt)
        s["q"], s["k"], s["v"] = qkv.split([h * dk, kv * dk, kv * dv], dim=1)
        s["state"] = rand(slots, h, dk, dv)
        s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:rows].to(torch.int32)
        if own:
            import mamba2_ssd_selective_gb300 as ssd

            s["runner"] = ssd.LinearAttnRunner(rows, 1, h, dk, dv, nheads_kv=kv, dtype=case["dtype"])
        return s
    lens = _lengths(case, int(seed))
    n, total = len(lens), sum(lens)
    # q, k and v are parts of the projection's output: views with its row stride
    qkv = rand(total, (h + kv) * dk + kv * dv, dtype=tt)
    s["q"], s["k"], s["v"] = qkv.split([h * dk, kv * dk, kv * dv], dim=1)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["max_len"] = max(lens)
    s["init"] = rand(n, h, dk, dv) if case["init"] else None
    if case["op"] == "la_backward":
        s["do"] = rand(total, h * dv, dtype=tt)
        s["dfinal"] = rand(n, h, dk, dv) if case["init"] else None
    if own:
        import mamba2_ssd_selective_gb300 as ssd

        s["runner"] = ssd.LinearAttnRunner(n, case["tokens"], h, dk, dv, nheads_kv=kv, dtype=case["dtype"],
                                           packed=case["packed"])
    return s


# ------------------------------------------------------------------ plain form

def _pad(x, s, heads):
    """(total, heads * d) rows -> (n, H, Lmax, d) in 32 bits, zeros past each sequence; heads are repeated up to H."""
    case, cu, top = s["case"], s["cu"].long(), s["max_len"]
    t = torch.arange(top, device="cuda")
    rows = cu[:-1, None] + t
    live = rows < cu[1:, None]
    x = x[rows.clamp(max=x.shape[0] - 1)].float() * live[..., None]
    x = x.view(*rows.shape, heads, -1).transpose(1, 2)
    return x.repeat_interleave(case["heads"] // heads, dim=1)


def _unpad(x, s, heads, dtype):
    """(n, H, Lmax, d) -> (total, heads * d), summed over the query heads that share a head, rounded once."""
    cu, total = s["cu"].long(), s["q"].shape[0]
    tok = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu[1:], tok, right=True)
    n, h, top, d = x.shape
    x = x.view(n, heads, h // heads, top, d).sum(2)
    return x[seq, :, tok - cu[seq]].reshape(total, heads * d).to(dtype)


def _power(log_decay, expo):
    """exp(log_decay_h * expo): (H, *expo.shape), or for expo (n, L) -> (n, H, L)."""
    return torch.exp(log_decay.view(-1, *([1] * expo.dim())) * expo)


def _mix(q, k, v, g):
    """sum_(j <= i) lam^(i - j) (q_i . k_j) v_j in blocks of tokens: products inside a block, states between blocks."""
    n, h, top, _ = q.shape
    dk, dv = k.shape[-1], v.shape[-1]
    pad = -top % _CHUNK
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(n, h, -1, _CHUNK, x.shape[-1]) for x in (q, k, v))
    nc = q.shape[2]
    i = torch.arange(_CHUNK, device="cuda", dtype=torch.float32)
    gap = i[:, None] - i
    inside = torch.where(gap >= 0, _power(g, gap.clamp(min=0)), 0.0)[:, None]
    out = (q @ k.transpose(-1, -2) * inside) @ v
    if nc > 1:
        made = (k * _power(g, _CHUNK - 1 - i)[:, None, :, None]).transpose(-1, -2) @ v
        c = torch.arange(nc, device="cuda", dtype=torch.float32)
        gap = c[:, None] - c - 1
        carry = torch.where(gap >= 0, _power(g, gap.clamp(min=0) * _CHUNK), 0.0)
        state = (carry @ made.view(n, h, nc, dk * dv)).view(n, h, nc, dk, dv)
        out = out + (q @ state) * _power(g, i + 1)[:, None, :, None]
    return out.reshape(n, h, top + pad, dv)[:, :, :top]


def _times(s):
    """Exponents of each padded position: from the sequence's start, and to its end (0 past it)."""
    lens = (s["cu"][1:] - s["cu"][:-1]).float()
    t = torch.arange(s["max_len"], device="cuda", dtype=torch.float32)
    left = lens[:, None] - 1 - t
    g = s["log_decay"].view(1, -1, 1)
    start = torch.exp(g * (t + 1))
    end = torch.where(left[:, None] >= 0, torch.exp(g * left.clamp(min=0)[:, None]), 0.0)
    whole = torch.exp(g[..., 0] * lens[:, None])
    return start[..., None], end[..., None], whole[..., None, None]


def _plain_forward(s):
    case, g, scale = s["case"], s["log_decay"], s["scale"]
    q, k, v = _pad(s["q"], s, case["heads"]), _pad(s["k"], s, case["kv"]), _pad(s["v"], s, case["kv"])
    start, end, whole = _times(s)
    o = _mix(q, k, v, g)
    final = (k * end).transpose(-1, -2) @ v
    if s["init"] is not None:
        o = o + (q @ s["init"]) * start
        final = final + whole * s["init"]
    return {"o": _unpad(o * scale, s, case["heads"], s["q"].dtype), "final_state": final}


def _plain_backward(s):
    case, g, scale = s["case"], s["log_decay"], s["scale"]
    q, k, v = _pad(s["q"], s, case["heads"]), _pad(s["k"], s, case["kv"]), _pad(s["v"], s, case["kv"])
    do = _pad(s["do"], s, case["heads"])
    start, end, whole = _times(s)
    dq = _mix(do, v, k, g)
    qb, kb, vb, dob = (x.flip(2) for x in (q, k, v, do))
    dk = _mix(vb, dob, qb, g).flip(2) * scale
    dv = _mix(kb, qb, dob, g).flip(2) * scale
    out = {}
    if s["init"] is not None:
        dq = dq + (do @ s["init"].transpose(-1, -2)) * start
        dk = dk + (v @ s["dfinal"].transpose(-1, -2)) * end
        dv = dv + (k @ s["dfinal"]) * end
        out["dinitial_state"] = (q * start).transpose(-1, -2) @ do * scale + whole * s["dfinal"]
    out["dq"] = _unpad(dq * scale, s, case["heads"], s["q"].dtype)
    out["dk"] = _unpad(dk, s, case["kv"], s["q"].dtype)
    out["dv"] = _unpad(dv, s, case["kv"], s["q"].dtype)
    return out


def _plain_step(s):
    case, state, at = s["case"], s["state"], s["slots"].long()
    rows, h, kv = case["rows"], case["heads"], case["kv"]
    q = s["q"].float().view(rows, h, 1, -1)
    k, v = (s[x].float().view(rows, kv, 1, -1).repeat_interleave(h // kv, dim=1) for x in ("k", "v"))
    new = state[at] * torch.exp(s["log_decay"]).view(1, h, 1, 1) + k.transpose(-1, -2) * v
    state[at] = new
    return {"o": (q @ new * s["scale"]).to(s["q"].dtype).view(rows, -1), "state": state}


def _gn_norm(s):
    """xhat, u and the statistics, in 32 bits."""
    case = s["case"]
    n, m, c, groups = case["n"], case["m"], case["channels"], case["groups"]
    x = s["x"].float().view(n, m, groups, c // groups)
    if "mean" in s:
        mean, rstd = s["mean"], s["rstd"]
    else:
        mean = x.mean((1, 3))
        rstd = ((x - mean[:, None, :, None]).square().mean((1, 3)) + s["eps"]).rsqrt()
    xhat = ((x - mean[:, None, :, None]) * rstd[:, None, :, None]).view(n, m, c)
    return xhat, xhat * s["weight"] + s["bias"], mean, rstd


def _plain_gn_forward(s):
    xhat, u, mean, rstd = _gn_norm(s)
    act = s["case"]["act"]
    if act == "silu":
        u = u * torch.sigmoid(u)
    elif act == "gate":
        z = s["z"].float()
        u = u * (z * torch.sigmoid(z))
    return {"y": u.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_gn_backward(s):
    case = s["case"]
    n, m, c, groups = case["n"], case["m"], case["channels"], case["groups"]
    xhat, u, _, rstd = _gn_norm(s)
    du, out = s["dy"].float(), {}
    if case["act"] == "silu":
        p = torch.sigmoid(u)
        du = du * (p * (1 + u * (1 - p)))
    elif case["act"] == "gate":
        z = s["z"].float()
        p = torch.sigmoid(z)
        out["dz"] = (du * u * (p * (1 + z * (1 - p)))).to(s["x"].dtype)
        du = du * (z * p)
    out["dweight"], out["dbias"] = (du * xhat).sum((0, 1)), du.sum((0, 1))
    dxhat = (du * s["weight"]).view(n, m, groups, -1)
    xg = xhat.view(n, m, groups, -1)
    a = dxhat.mean((1, 3), keepdim=True)
    b = (dxhat * xg).mean((1, 3), keepdim=True)
    out["dx"] = ((dxhat - a - xg * b) * rstd[:, None, :, None]).view(n, m, c).to(s["x"].dtype)
    return out


_PLAIN = {"la_forward": _plain_forward, "la_backward": _plain_backward, "la_step": _plain_step,
          "gn_forward": _plain_gn_forward, "gn_backward": _plain_gn_backward}


# ------------------------------------------------------------------ one pass

def run(s):
    if not own:
        return _PLAIN[s["op"]](s)
    r, op = s["runner"], s["op"]
    if op == "la_forward":
        o, final = r.forward(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], initial_state=s["init"],
                             cu_seqlens=s["cu"] if s["case"]["packed"] else None)
        return {"o": o, "final_state": final}
    if op == "la_backward":
        g = r.backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"], initial_state=s["init"],
                       dfinal_state=s["dfinal"], cu_seqlens=s["cu"] if s["case"]["packed"] else None)
        return {k: v for k, v in g.items() if v is not None}
    if op == "la_step":
        o = r.step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], slot_idx=s["slots"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if op == "gn_forward":
        y, mean, rstd = r.forward(s["x"], s["weight"], s["bias"], z=s["z"], eps=s["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    g = r.backward(s["dy"], s["x"], s["weight"], s["bias"], s["mean"], s["rstd"], z=s["z"])
    return {k: v for k, v in g.items() if v is not None}


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("gn"):
        size, gate = case["n"] * case["m"] * case["channels"], case["act"] == "gate"
        if case["op"] == "gn_forward":
            return {"bytes": size * es * (3 if gate else 2), "flops": size * (14 if gate else 10)}
        return {"bytes": size * es * (5 if gate else 3), "flops": size * (30 if gate else 20)}
    h, kv, dk, dv = case["heads"], case["kv"], case["dk"], case["dv"]
    if case["op"] == "la_step":
        one = h * dk * dv
        return {"bytes": case["rows"] * (8 * one + es * (h + kv) * (dk + dv)), "flops": 5 * case["rows"] * one}
    total = case["tokens"] * (1 if case["packed"] else case["n"])
    states = 4 * case["n"] * h * dk * dv
    if case["op"] == "la_forward":
        return {"bytes": total * es * (h + kv) * (dk + dv) + states * (2 if case["init"] else 1),
                "flops": 4 * total * h * dk * dv}
    moved = h * (2 * dk + dv) + 2 * kv * (dk + dv)  # q, dq, do; k, dk, v, dv
    return {"bytes": total * es * moved + (3 * states if case["init"] else 0), "flops": 10 * total * h * dk * dv}


# ------------------------------------------------------------------ 64 bits

def _exact_la(s, case):
    """The recurrence itself, token by token, for all sequences at once."""
    h, kv = case["heads"], case["kv"]
    cu = s["cu"].tolist()
    lens = [b - a for a, b in zip(cu, cu[1:])]
    n, total, top = len(lens), cu[-1], max(lens)
    lam = torch.exp(s["log_decay"].double()).view(1, h, 1, 1)
    scale = float(s["scale"])
    len_t = torch.tensor(lens, device="cuda")
    first = torch.tensor(cu[:-1], device="cuda")

    def at(x, t, heads):  # token t of every sequence, (n, H, d)
        rows = x[(first + t).clamp(max=total - 1)].double().view(n, heads, -1)
        return rows.repeat_interleave(h // heads, dim=1)

    def put(out, t, val):
        ok = (t < len_t).nonzero()[:, 0] if min(lens) <= t else slice(None)
        out[first[ok] + t] = val[ok]

    zeros = lambda d: torch.zeros(total, h, d, dtype=torch.float64, device="cuda")  # noqa: E731
    state = s["init"].double() if s["init"] is not None else torch.zeros(n, h, case["dk"], case["dv"],
                                                                         dtype=torch.float64, device="cuda")
    back = case["op"] == "la_backward"
    out = zeros(case["dk"] if back else case["dv"])
    for t in range(top):
        live = (t < len_t).view(n, 1, 1, 1)
        k, v = at(s["k"], t, kv), at(s["v"], t, kv)
        state = torch.where(live, lam * state + k[..., :, None] * v[..., None, :], state)
        if back:
            put(out, t, scale * torch.einsum("nhkv,nhv->nhk", state, at(s["do"], t, h)))
        else:
            put(out, t, scale * torch.einsum("nhkv,nhk->nhv", state, at(s["q"], t, h)))
    if not back:
        return {"o": out.view(total, -1), "final_state": state}
    dk, dv = zeros(case["dk"]), zeros(case["dv"])
    # the gradient of the state after token t
    grad = s["dfinal"].double() if s["dfinal"] is not None else torch.zeros_like(state)
    for t in reversed(range(top)):
        live = (t < len_t).view(n, 1, 1, 1)
        grad = torch.where(live, grad + scale * at(s["q"], t, h)[..., :, None] * at(s["do"], t, h)[..., None, :], grad)
        put(dk, t, torch.einsum("nhkv,nhv->nhk", grad, at(s["v"], t, kv)))
        put(dv, t, torch.einsum("nhkv,nhk->nhv", grad, at(s["k"], t, kv)))
        grad = torch.where(live, grad * lam, grad)
    res = {"dq": out.view(total, -1), "dk": dk.view(total, kv, h // kv, -1).sum(2).view(total, -1),
           "dv": dv.view(total, kv, h // kv, -1).sum(2).view(total, -1)}
    if s["init"] is not None:
        res["dinitial_state"] = grad
    return res


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("la_forward", "la_backward"):
        return _exact_la(s, case)
    if case["op"] == "la_step":
        h, kv, rows = case["heads"], case["kv"], case["rows"]
        heads = torch.arange(h, device="cuda") // (h // kv)
        q = s["q"].double().view(rows, h, -1)
        k, v = (s[x].double().view(rows, kv, -1)[:, heads] for x in ("k", "v"))
        state, at = s["state"].double(), s["slots"].long()
        lam = torch.exp(s["log_decay"].double())[None, :, None, None]
        state[at] = lam * state[at] + torch.einsum("rhk,rhv->rhkv", k, v)
        return {"o": float(s["scale"]) * torch.einsum("rhk,rhkv->rhv", q, state[at]).reshape(rows, -1), "state": state}
    n, m, c, groups = case["n"], case["m"], case["channels"], case["groups"]
    rep = c // groups
    x = s["x"].double()
    by = x.view(n, m, groups, rep)
    if case["op"] == "gn_forward":
        mean = by.sum((1, 3)) / (m * rep)
        var = (by ** 2).sum((1, 3)) / (m * rep) - mean ** 2
        rstd = 1 / torch.sqrt(var + s["eps"])
    else:
        mean, rstd = s["mean"].double(), s["rstd"].double()
    wide = lambda v: v.repeat_interleave(rep, dim=1)[:, None]  # noqa: E731
    w, b = s["weight"].double(), s["bias"].double()
    xhat = (x - wide(mean)) * wide(rstd)
    u = xhat * w + b
    gate = None if s["z"] is None else s["z"].double()
    if case["op"] == "gn_forward":
        if case["act"] == "silu":
            u = u / (1 + torch.exp(-u))
        elif gate is not None:
            u = u * gate / (1 + torch.exp(-gate))
        return {"y": u, "mean": mean, "rstd": rstd}
    dy, res = s["dy"].double(), {}
    if case["act"] == "silu":
        e = torch.exp(-u)
        dy = dy * (1 + e + u * e) / (1 + e) ** 2
    elif gate is not None:
        e = torch.exp(-gate)
        res["dz"] = dy * u * (1 + e + gate * e) / (1 + e) ** 2
        dy = dy * gate / (1 + e)
    res["dweight"], res["dbias"] = (dy * xhat).sum((0, 1)), dy.sum((0, 1))
    p = dy * w
    count = m * rep
    mean_p = wide(p.view(n, m, groups, rep).sum((1, 3)) / count)
    mean_px = wide((p * xhat).view(n, m, groups, rep).sum((1, 3)) / count)
    res["dx"] = wide(rstd) * (p - mean_p - xhat * mean_px)
    return res
