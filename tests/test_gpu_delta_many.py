"""Gradients of the gated delta rule where every block of the persistent kernels has many chunks and heads to go through: more
units (chunks x heads of q and k) than three times the SMs, full chunks and parts of one, heads shared.

A head's gradients do not depend on the others in a call, and all sums have a fixed order: a call on one head of q and k, whose
units are fewer than the SMs, gives the same bits.  Such a call is held to the 64-bit reference, by test_gpu_delta.py's bounds."""
from __future__ import annotations

import copy

import pytest
import torch

from tests.test_gpu_delta import Case, _built  # noqa: F401

pytestmark = pytest.mark.gpu

LENS = [700, 1, 0, 650, 64, 129, 333, 128, 200, 63, 500]  # 49 chunks


def part(c, k):
    """The k-th head of q and k, and its states, as a case."""
    x, n = copy.copy(c), c.H // c.K
    x.H, x.K = n, 1
    q, kk, v = c.qkv.split([c.K * c.dk] * 2 + [c.H * c.dv], 1)
    cols = lambda t, w, m=1: t[:, k * m * w:(k + 1) * m * w]  # noqa: E731
    x.qkv = torch.cat([cols(q, c.dk), cols(kk, c.dk), cols(v, c.dv, n)], 1)
    x.gates = torch.cat([cols(t, 1, n) for t in c.gates.split([c.H, c.H], 1)], 1)
    x.do = cols(c.do, c.dv, n).contiguous()
    x.init, x.dfinal = (t[:, k * n:(k + 1) * n].contiguous() for t in (c.init, c.dfinal))
    return x


@pytest.mark.parametrize("dtype,dk,dv,norm", [("bf16", 64, 64, True), ("bf16", 128, 128, True), ("bf16", 64, 128, False),
                                              ("bf16", 104, 40, True), ("f32", 64, 64, True), ("bf16", 136, 64, False)])
def test_many_units(dtype, dk, dv, norm):
    H, K = 24, 12
    c = Case(LENS, H, K, dk, dv, dtype, norm=norm, seed=81)
    g, n = c.backward(), H // K
    for k in range(K):
        got = part(c, k).backward()
        for name, w in (("dq", dk), ("dk", dk), ("dv", n * dv), ("dlog_decay", n), ("dbeta", n)):
            assert torch.equal(g[name][:, k * w:(k + 1) * w], got[name]), (name, k)
        assert torch.equal(g["dinitial_state"][:, k * n:(k + 1) * n], got["dinitial_state"]), k
    part(c, K - 1).check_backward()


def test_many_states_to_a_head():
    """Two heads of q and k for 24 states: a block's steps on one chunk."""
    c = Case([300, 77, 64], 24, 2, 64, 64, seed=82)
    c.check_backward()
