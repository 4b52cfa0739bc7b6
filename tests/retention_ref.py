"""64-bit reference of the retention operators: the recurrences and formulas as
they are defined, token by token, in float64 on the CPU."""
from __future__ import annotations

import torch


def linear_attn(q, k, v, log_decay, scale, lens, init=None, do=None, dfinal=None):
    """q (T, H, dk), k (T, K, dk), v (T, K, dv); lens: tokens of each sequence in order.

    Returns o (T, H, dv) and final states, and with `do` also dq, dk, dv, dinit."""
    q, k, v = (x.double() for x in (q, k, v))
    T, H, dk = q.shape
    K, dv = k.shape[1], v.shape[2]
    rep = H // K
    kh, vh = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    lam = torch.exp(log_decay.double())[:, None, None]
    o = torch.zeros(T, H, dv, dtype=torch.float64)
    n = len(lens)
    fin = torch.zeros(n, H, dk, dv, dtype=torch.float64) if init is None else init.double().clone()
    dq, dkh, dvh = torch.zeros_like(q), torch.zeros_like(kh), torch.zeros_like(vh)
    dinit = torch.zeros(n, H, dk, dv, dtype=torch.float64) if dfinal is None else dfinal.double().clone()
    t0 = 0
    for s, L in enumerate(lens):
        S = fin[s]
        for t in range(t0, t0 + L):
            S = lam * S + kh[t][:, :, None] * vh[t][:, None, :]
            o[t] = scale * torch.einsum("hk,hkv->hv", q[t], S)
            if do is not None:
                dq[t] = scale * torch.einsum("hv,hkv->hk", do[t].double(), S)
        fin[s] = S
        if do is not None:
            R = dinit[s]
            for t in reversed(range(t0, t0 + L)):
                R = R + scale * q[t][:, :, None] * do[t].double()[:, None, :]
                dkh[t] = torch.einsum("hkv,hv->hk", R, vh[t])
                dvh[t] = torch.einsum("hkv,hk->hv", R, kh[t])
                R = lam * R
            dinit[s] = R
        t0 += L
    if do is None:
        return o, fin
    return (o, fin, dq, dkh.view(T, K, rep, dk).sum(2), dvh.view(T, K, rep, dv).sum(2), dinit)


def _silu(a):
    return a * torch.sigmoid(a)


def _dsilu(a):
    p = torch.sigmoid(a)
    return p * (1 + a * (1 - p))


def group_norm(x, groups, weight=None, bias=None, z=None, act="none", eps=1e-5, dy=None):
    """x (n, m, C).  Returns y, mean, rstd, and with `dy` also dx, dweight, dbias, dz."""
    x = x.double()
    n, m, C = x.shape
    w = torch.ones(C, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(C, dtype=torch.float64) if bias is None else bias.double()
    xg = x.view(n, m, groups, C // groups)
    mean = xg.mean((1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = 1 / torch.sqrt(var + eps)
    xh = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).view(n, m, C)
    u = xh * w + b
    y = u if act == "none" else _silu(u) if act == "silu" else u * _silu(z.double())
    if dy is None:
        return y, mean, rstd
    dy = dy.double()
    dz = None
    du = dy
    if act == "silu":
        du = dy * _dsilu(u)
    elif act == "gate":
        du = dy * _silu(z.double())
        dz = dy * u * _dsilu(z.double())
    dxh = (du * w).view(n, m, groups, -1)
    xhg = xh.view(n, m, groups, -1)
    dx = (dxh - dxh.mean((1, 3), keepdim=True) - xhg * (dxh * xhg).mean((1, 3), keepdim=True)) * rstd[:, None, :, None]
    return y, mean, rstd, dx.view(n, m, C), (du * xh).sum((0, 1)), du.sum((0, 1)), dz
