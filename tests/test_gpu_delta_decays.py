"""Gradients of log decays on the GPU, token by token, against the size of what passes the token: in heads that forget fast that
is little, and rounding errors of what no decay touches would show.

Tolerances.  A gradient is a sum of terms over a chunk's 64 tokens and its states, `passing` below: for a token t, A the sum
of the absolute values of the terms that pass it (those of a pair of tokens: a product q.k or k.k times each value of a sum over
v), B that of all terms that sums of rows less sums of columns take to it, pairs of tokens behind it among them, which cancel,
and with the absolute values of the products' own terms.
fp32: F32 of B.  Less than 200 roundings of 2^-24 follow one another in those sums, 1.2e-5 of B at most and, as they are of
both signs, far less; what the terms are made of (errors of prediction, states, their gradients) is within a quarter of F32 of
its norm, and a product of two such rows with both factors off by that is off by 2 * 5e-6 of the norms' product, for values of
both signs 1.6 times the sum of its terms' absolute values: 1.6e-5.
bf16: two factors of a term are rounded, and so is the result: (1 + 2^-8)^3 - 1 of A, beside F32 of B for the sums, which have
fp32 terms of which equal ones cancel exactly."""
from __future__ import annotations

import pytest
import torch

from tests import delta_ref as ref
from tests.test_gpu_delta import F32, Case, _built  # noqa: F401

pytestmark = pytest.mark.gpu

BF16_TERMS = (1 + 2 ** -8) ** 3 - 1


def passing(q, k, v, g, b, scale, lens, do, init, dfinal, eps):
    """(A, B), (T, H): token by token forward for the errors of prediction and the states before chunks, in reverse for the
    gradients of the errors and of the states behind chunks, then the terms of each chunk."""
    T, H = g.shape
    if eps is not None:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps) for x in (q, k))
    q, k = (x.repeat_interleave(H // q.shape[1], 1) for x in (q, k))
    outer = lambda x, y: torch.einsum("hk,hv->hkv", x, y)  # noqa: E731
    row = lambda x, S: torch.einsum("hk,hkv->hv", x, S)  # noqa: E731
    A, B, t0 = torch.zeros(T, H).double(), torch.zeros(T, H).double(), 0
    for s, n in enumerate(lens):
        S, before, E = init[s].double(), [], []
        for t in range(t0, t0 + n):
            if (t - t0) % 64 == 0:
                before.append(S)
            S = torch.exp(g[t])[:, None, None] * S
            E.append(v[t] - row(k[t], S))
            S = S + outer(b[t][:, None] * k[t], E[-1])
        G, behind, Z = dfinal[s].double(), [None] * len(before), [None] * n
        for t in reversed(range(t0, t0 + n)):
            if (t - t0) % 64 == 63 or t == t0 + n - 1:
                behind[(t - t0) // 64] = G
            G = G + scale * outer(q[t], do[t])
            Z[t - t0] = row(k[t], G)
            G = torch.exp(g[t])[:, None, None] * (G - outer(k[t], b[t][:, None] * Z[t - t0]))
        for c, S, D in zip(range(0, n, 64), before, behind):
            at = slice(t0 + c, min(t0 + n, t0 + c + 64))
            heads = lambda x: x[at].double().transpose(0, 1)  # noqa: E731
            qq, kk, oo, bb = heads(q).abs(), heads(k).abs(), heads(do).abs(), b[at].T
            ee, zz = (torch.stack(x[c:c + 64]).transpose(0, 1).abs() for x in (E, Z))
            S, D, G = S.abs(), D.abs(), g[at].T.cumsum(1)
            L = torch.exp(G[:, :, None] - G[:, None, :]).tril(-1)
            tt = lambda x: x.transpose(1, 2)  # noqa: E731
            pairs = lambda qk, k2: L * bb[:, None] * (scale * (oo @ tt(ee)) * qk + bb[..., None] * (zz @ tt(ee)) * k2)  # noqa: E731
            M, N = pairs((heads(q) @ tt(heads(k))).abs(), (heads(k) @ tt(heads(k))).abs()), pairs(qq @ tt(kk), kk @ tt(kk))
            read = torch.exp(G) * (scale * (qq * (oo @ tt(S))).sum(-1) + bb * (kk * (zz @ tt(S))).sum(-1))
            add = torch.exp(G[:, -1:] - G) * bb * (kk * (ee @ tt(D))).sum(-1)
            end = torch.exp(G[:, -1:]) * (S * D).sum((1, 2))[:, None]
            m = M.shape[1]
            for t in range(m):
                rest = read[:, t:].sum(1) + add[:, :t].sum(1) + end[:, 0]
                A[t0 + c + t] = rest + M[:, t:, :t].sum((1, 2))
                B[t0 + c + t] = rest + N[:, t:, :t].sum((1, 2)) + 2 * N[:, t:, t:].sum((1, 2))
        t0 += n
    return A, B


def check(c, lowest=None):
    """Our gradients and the reference's, (T, H) in 64 bits, ours held to the bound; lowest: what the reference takes for log
    decays below it."""
    got = c.backward()["dlog_decay"].double().cpu()
    inp = list(c.ref_inputs())
    if lowest is not None:
        inp[3] = inp[3].clamp(min=lowest)
    do = c.do.view(c.T, c.H, -1)
    want = ref.delta_rule_grads(*inp, do, c.init, c.dfinal, c.eps)["dlog_decay"]
    A, B = passing(*inp, do.double(), c.init, c.dfinal, c.eps)
    bound = F32 * B + (0.0 if c.dtype == "f32" else BF16_TERMS * A)
    over = (got - want).abs() / bound.clamp(min=1e-37)
    assert torch.isfinite(got).all() and over.max() <= 1, f"by heads, of the bound: {over.amax(0).tolist()}"
    return got, want


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 64, 64), ("f32", 128, 40), ("bf16", 64, 64), ("bf16", 128, 128), ("bf16", 136, 64)])
@pytest.mark.parametrize("norm", [True, False])
def test_heads_that_forget_fast(dtype, dk, dv, norm):
    rates = torch.tensor([-0.25, -1.0, -3.0, -5.0, -8.0, -12.0, -16.0, -30.0])
    check(Case([140, 77, 1], 8, 4, dk, dv, dtype, norm=norm, seed=71, decay=rates))


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 136)])
@pytest.mark.parametrize("decay", [float("-inf"), -1e30])
def test_nothing_passes_a_head_that_forgets_everything(decay, dtype, d):
    got, want = check(Case([150, 66], 2, 1, d, 64, dtype, seed=72, decay=torch.tensor([decay])), lowest=-300.0)
    assert want.abs().max() < 1e-30 and (got == 0).all()


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 136)])
def test_nothing_passes_a_reset(dtype, d):
    """Token 70 of 140 forgets everything: its gradient is what sums over its chunk's other pairs leave in fp32."""
    c = Case([140], 2, 2, d, 64, dtype, packed=False, seed=73)
    c.gates[70, :2] = float("-inf")
    got, want = check(c, lowest=-300.0)
    assert want[70].abs().max() < 1e-30 and (got[70].abs() <= F32 * want[64:128].norm(dim=0)).all()
