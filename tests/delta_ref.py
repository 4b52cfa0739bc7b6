"""64-bit reference of the gated delta rule and of the norms around a block: the recurrence token by token and the
formulas as they are defined, in float64 on the CPU; gradients through autograd."""
from __future__ import annotations

import torch


def delta_rule(q, k, v, g, b, scale, lens, init=None, eps=None):
    """q, k (T, K, dk), v (T, H, dv), g, b (T, H); lens: tokens of each sequence in order; eps: of qk_norm, or None.
    Returns o (T, H, dv) and the final states (n, H, dk, dv)."""
    H, dv = v.shape[1:]
    if eps is not None:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps) for x in (q, k))
    rep = H // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    o, final, t0 = [], [], 0
    for s, n in enumerate(lens):
        S = torch.zeros(H, q.shape[2], dv, dtype=torch.float64) if init is None else init[s]
        for t in range(t0, t0 + n):
            S = torch.exp(g[t])[:, None, None] * S
            err = v[t] - torch.einsum("hk,hkv->hv", k[t], S)
            S = S + torch.einsum("hk,hv->hkv", b[t][:, None] * k[t], err)
            o.append(scale * torch.einsum("hk,hkv->hv", q[t], S))
        final.append(S)
        t0 += n
    return torch.stack(o) if o else torch.zeros(0, H, dv, dtype=torch.float64), torch.stack(final)


def delta_rule_grads(q, k, v, g, b, scale, lens, do, init=None, dfinal=None, eps=None):
    """Gradients of <do, o> + <dfinal, final>: a dict of dq, dk, dv, dlog_decay, dbeta and dinitial_state."""
    n, H, dk, dv = len(lens), v.shape[1], q.shape[2], v.shape[2]
    x = {"dq": q, "dk": k, "dv": v, "dlog_decay": g, "dbeta": b,
         "dinitial_state": torch.zeros(n, H, dk, dv) if init is None else init}
    x = {name: t.detach().double().clone().requires_grad_() for name, t in x.items()}
    o, final = delta_rule(x["dq"], x["dk"], x["dv"], x["dlog_decay"], x["dbeta"], scale, lens, x["dinitial_state"], eps)
    loss = (o * do.double()).sum()
    if dfinal is not None:
        loss = loss + (final * dfinal.double()).sum()
    return dict(zip(x, torch.autograd.grad(loss, list(x.values()), allow_unused=True, materialize_grads=True)))


def decay_terms(q, v, g, grads, lens, rep):
    """(T, H): the root of the summed squares of what a token's dlog_decay is a sum of inside its chunk of 64 tokens,
    q.dq and v.dv of it and later tokens, or |dlog_decay| where that is more: what rounding errors are relative to."""
    # per head: the gradients of shared q are summed over heads, so each head's part is bounded by the whole's row norms
    dq = grads["dq"]
    qq = (q.double().norm(dim=-1) * dq.norm(dim=-1)).repeat_interleave(rep, 1) / q.shape[2] ** 0.5
    vv = v.double().norm(dim=-1) * grads["dv"].norm(dim=-1) / v.shape[2] ** 0.5
    out, t0 = torch.zeros_like(vv), 0
    for n in lens:
        for c in range(t0, t0 + n, 64):
            e = slice(c, min(t0 + n, c + 64))
            out[e] = (qq[e] ** 2 + vv[e] ** 2).flip(0).cumsum(0).flip(0).sqrt()
        t0 += n
    return torch.maximum(out, grads["dlog_decay"].abs())


def block_norm(x, residual=None, z=None, post_norm=False, pre_norm=True, pw=None, sc=None, w=None, eps=1e-6,
               constant_rms=False):
    """(h, y or None); constant_rms: gradients without the part that goes through the rms."""
    def rms(v):
        r = torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
        return r.detach() if constant_rms else r

    u = x
    if post_norm:
        u = u / rms(u)
        u = u if pw is None else u * pw
    if z is not None:
        u = u * z * torch.sigmoid(z)
    if sc is not None:
        u = u * sc
    h = u if residual is None else residual + u
    if not pre_norm:
        return h, None
    y = h / rms(h)
    return h, y if w is None else y * w
