"""Linear attention where sequences are cut: chained segments, segments side by side, and their waits.

Tolerances are those of test_gpu_retention.py."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from tests.test_gpu_retention import Case, _built  # noqa: F401

pytestmark = pytest.mark.gpu

TIMEOUT = -9  # SSD_ERR_DEVICE_TIMEOUT


# at least as many items (sequences x heads, three times as many backward) as SMs, and rounds that segments fill
# better: (sequences' lengths, heads, key/value heads, packed, is forward cut, is backward)
CHAINED = [
    ([650] * 10, 16, 16, False, True, False),
    ([750] * 4, 16, 4, False, False, True),
    ([64 * 9 + 1] * 20, 8, 8, False, True, False),
    ([2300, 1, 0, 64, 5, 63, 2049, 0, 130, 17], 16, 4, True, False, True),
    ([2300, 1, 0, 64, 5, 63, 2049, 0, 130, 17] + [260] * 14, 32, 8, True, True, True),
]


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 72)])
@pytest.mark.parametrize("lens,H,K,packed,forward,backward", CHAINED)
def test_chained_segments(lens, H, K, packed, forward, backward, dk, dv):
    c = Case(lens, H, K, dk, dv, packed=packed, seed=sum(lens) + dv)
    # room for a state of each head that is handed over, so that this case takes the path it is meant for
    state, heads = H * dk * dv * 4, c.T * H * (dk + dv) * 4 if K < H else 0
    assert (ssd.ssd_linear_attn_workspace_size(c.runner().dims, False) > state) == forward
    assert (ssd.ssd_linear_attn_workspace_size(c.runner().dims, True) - heads > 3 * state) == backward
    c.check()


def test_chained_segments_without_states():
    Case([650] * 10, 16, 16, 64, 64, packed=False, seed=3).check(init=False)


def test_chained_decays():
    """Every kind of head in one queue of items: none, strong, and about where scores are weighed in another way."""
    decay = torch.tensor([0.0, -float("inf"), -30.0, -1.0, -1e-4, -0.4332, -0.4333, -0.2] * 2)
    Case([650] * 10, 16, 16, 64, 64, packed=False, seed=5, decay=decay).check()


def test_chained_repeats_give_equal_bits():
    c = Case([2300, 1, 700, 64, 5, 63, 2049, 0, 130, 17] + [260] * 14, 32, 8, 64, 64, seed=9)
    a, b = c.gpu(), c.gpu()
    for x, y in zip([a[0], a[1], *a[2].values()], [b[0], b[1], *b[2].values()]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 40), (8, 64)])
def test_side_by_side_states_of_both_reverse_passes(dk, dv, dtype):
    """dk and dv read one state, one of them transposed: widths that differ, shared heads, a last segment that is short."""
    long = 6000 if dtype == "bf16" else 901
    for c in (Case([long, 2, 0, 640], 4, 2, dk, dv, dtype, seed=dk), Case([long], 3, 3, dk, dv, dtype, packed=False, seed=dv)):
        heads = c.T * c.H * (dk + dv) * 4 if c.K < c.H else 0
        assert ssd.ssd_linear_attn_workspace_size(c.runner().dims, True) - heads > 6 * c.H * dk * dv * 4
        c.check(init=c.packed)


@pytest.mark.parametrize("lens,H,packed", [([200, 200], 4, False), ([1500], 2, False), ([650] * 10, 16, False),
                                           ([900, 0, 700], 3, True)])
def test_waits_that_give_up_are_reported_and_the_next_call_is_clean(lens, H, packed):
    """With the wait limit at 0 every wait that outlasts one parked poll gives up; the kernels drain what they started,
    return, and report it.  A hand-off inside a block is quicker than that, a wait for another segment's state is
    not.  A call that reports nothing is right, and afterwards the same call runs clean."""
    c = Case(lens, H, H, 64, 64, packed=packed, seed=41)
    r = c.runner()
    q, k, v = c.parts("cuda")
    kw = dict(initial_state=c.init.cuda(), cu_seqlens=c.cu.cuda() if packed else None)
    decay, do = c.decay.cuda(), c.do.cuda()

    def call():
        o, fin = r.forward(q, k, v, decay, **kw)
        st_f = ssd.ssd_device_status(r.workspace)
        g = r.backward(q, k, v, decay, do, **kw)
        st_b = ssd.ssd_device_status(r.workspace)
        return [o, fin, *g.values()], (st_f, st_b)

    first, st = call()
    assert st == (0, 0)
    prev = ssd.ssd_set_wait_limit_ns(0)
    try:
        hasty, st = call()
    finally:
        ssd.ssd_set_wait_limit_ns(prev)
    assert st[0] in (0, TIMEOUT) and st[1] in (0, TIMEOUT)
    if len(lens) * H >= 152:  # chained
        assert st[0] == TIMEOUT
    for x, y in zip(first[:2] * (st[0] == 0), hasty):
        assert torch.equal(x, y)
    for x, y in zip(first[2:] * (st[1] == 0), hasty[2:]):
        assert torch.equal(x, y)
    again, st = call()
    assert st == (0, 0)
    for x, y in zip(first, again):
        assert torch.equal(x, y)


def _operators(c, r, step, norm, cache):
    """One call of each operator; its outputs."""
    q, k, v = c.parts("cuda")
    decay = c.decay.cuda()
    slots = torch.tensor([3, 0, -1, 2], dtype=torch.int32, device="cuda")
    do, init, cu = c.do.cuda(), c.init.cuda(), c.cu.cuda()

    def call():
        o, fin = r.forward(q, k, v, decay, initial_state=init, cu_seqlens=cu)
        y, mean, rstd = norm.forward(o, None, None, z=do)
        n = norm.backward(do, o, None, None, mean, rstd, z=do)
        g = r.backward(q, k, v, decay, n["dx"], initial_state=init, cu_seqlens=cu)
        t = step.step(q[:4], k[:4], v[:4], decay, cache, slot_idx=slots)
        return [o, fin, y, t, *n.values(), *g.values()]

    return call


@pytest.mark.parametrize("how", ["graph", "stream"])
def test_captured_and_on_another_stream(how):
    c = Case([700, 3, 0, 900], 4, 2, 64, 64, seed=19)
    cache = torch.zeros(5, 4, 64, 64, device="cuda")
    call = _operators(c, c.runner(), ssd.LinearAttnRunner(4, 1, 4, 64, 64, nheads_kv=2), ssd.GroupNormRunner(c.T, 1, 256, 4, "gate"),
                      cache)
    want = [x.clone() for x in call()]
    state = cache.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            cache.zero_()
            got = call()
    torch.cuda.current_stream().wait_stream(side)
    if how == "graph":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        for _ in range(2):
            cache.zero_()
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache, state)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
