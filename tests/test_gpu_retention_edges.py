"""The retention operators at the edges of what they accept: bounds that are out of order, streams, long runs of tokens,
shapes that take kernels of their own.

Tolerances are those of test_gpu_retention.py."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from mamba2_ssd_selective_gb300.inputs import SsdShape, make_inputs
from tests.gpu_util import to_dev
from tests.test_gpu_retention import BF16, F32, Case, _built, close, gn_case, gn_check  # noqa: F401

pytestmark = pytest.mark.gpu


# (tokens, sequences, heads, dtype): segments side by side, chained, side by side on the CUDA cores
@pytest.mark.parametrize("T,n,H,dtype", [(8192, 3, 16, "bf16"), (9000, 23, 32, "bf16"), (1500, 5, 2, "f32")])
def test_sequences_that_overlap(T, n, H, dtype):
    """Sequences over all rows by turns with empty ones, so that their segments are more than there is room for where calls are
    cut: states are those of the whole row and the initial ones, and rows (equal for equal sequences) are right."""
    c = Case([T] + [0] * (n - 1), H, H, 64, 64, dtype, seed=n)
    r = c.runner()
    for backward in (False, True):  # cut in both directions: states of segments are in the workspace
        assert ssd.ssd_linear_attn_workspace_size(r.dims, backward) > n * H * 64 * 64 * 4
    one = Case([T], H, H, 64, 64, dtype, packed=False, seed=n)
    one.init, one.dfin, one.decay = c.init[:1], c.dfin[:1], c.decay
    c.init, c.dfin = c.init[:1].expand_as(c.init).contiguous(), c.dfin[:1].expand_as(c.dfin).contiguous()
    c.cu = torch.tensor([0, T] * (n // 2) + [0, T], dtype=torch.int32)
    o, fin, g = c.gpu(runner=r)
    want, wfin, wg = one.gpu()
    tol = 2 * (BF16 if dtype == "bf16" else F32)  # both sides are results
    close(o, want.cpu(), tol, "o")
    for name in ("dq", "dk", "dv"):
        close(g[name], wg[name].cpu(), tol, name)
    for got, whole, start in ((fin, wfin, c.init), (g["dinitial_state"], wg["dinitial_state"], c.dfin)):
        for s in range(n):
            if s % 2:
                assert torch.equal(got[s].cpu(), start[s])
            else:
                close(got[s], whole[0].cpu(), 2 * F32, f"state {s}")


@pytest.mark.parametrize("T,n,H,dtype", [(8192, 7, 4, "bf16"), (9000, 30, 16, "bf16"), (1500, 7, 2, "f32")])
def test_bounds_in_any_order(T, n, H, dtype):
    c = Case([T] + [0] * (n - 1), H, H, 64, 64, dtype, seed=n)
    gen = torch.Generator().manual_seed(n)
    for _ in range(4):
        c.cu = torch.randint(-T // 4, T + T // 4, (n + 1,), generator=gen, dtype=torch.int32)
        _, fin, g = c.gpu()
        assert torch.isfinite(fin).all() and torch.isfinite(g["dinitial_state"]).all()
        lens = (c.cu[1:].clamp(0, T) - c.cu[:-1].clamp(0, T)).clamp(min=0)
        for s in (lens == 0).nonzero()[:, 0].tolist():
            assert torch.equal(fin[s].cpu(), c.init[s]) and torch.equal(g["dinitial_state"][s].cpu(), c.dfin[s])


# whole, chained, side by side
@pytest.mark.parametrize("lens,H,packed,dtype", [([200, 70, 0], 2, True, "bf16"), ([650] * 10, 16, False, "bf16"), ([8000], 2, False, "bf16"),
                                                 ([3, 8000, 0, 257], 2, True, "bf16"), ([1500, 1500], 2, False, "f32"),
                                                 ([3, 1400, 0, 257], 2, True, "f32")])
def test_states_in_place(lens, H, packed, dtype):
    """final_states may be initial_states: the same bits, wherever sequences are cut."""
    c = Case(lens, H, H, 64, 64, dtype, packed=packed, seed=len(lens))
    r = c.runner()
    want_o, want, _ = c.gpu(backward=False, runner=r)
    q, k, v = c.parts("cuda")
    decay, cu = c.decay.cuda(), c.cu.cuda()
    for _ in range(10):
        states, o = c.init.cuda(), torch.empty_like(want_o)
        inputs = ssd.SsdLinearAttnInputs(q.data_ptr(), q.stride(0), k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0),
                                         decay.data_ptr(), states.data_ptr(), cu.data_ptr() if packed else None, c.scale)
        ssd.ssd_linear_attn_forward(r.dims, inputs, o, o.stride(0), states, r.workspace)
        assert ssd.ssd_device_status(r.workspace) == 0
        assert torch.equal(o, want_o) and torch.equal(states, want)


# ------------------------------------------------------------------ streams

def _calls():
    """(runner, a call of it on a given stream that returns its outputs) for each operator and direction.  (The step's
    rows have no slot, so that calls leave nothing behind.)"""
    c = Case([500], 4, 2, 64, 64, packed=False, seed=23)
    q, k, v = c.parts("cuda")
    decay, do, x = c.decay.cuda(), c.do.cuda(), torch.randn(500, 256, device="cuda").bfloat16()
    kw = dict(initial_state=c.init.cuda())
    r, tok, norm = c.runner(), ssd.LinearAttnRunner(500, 1, 4, 64, 64, nheads_kv=2), ssd.GroupNormRunner(500, 1, 256, 4)
    cache, slots = torch.zeros(1, 4, 64, 64, device="cuda"), torch.full((500,), -1, dtype=torch.int32, device="cuda")
    _, mean, rstd = norm.forward(x)
    torch.cuda.synchronize()
    return [(r, lambda s: list(r.forward(q, k, v, decay, **kw, stream=s))),
            (r, lambda s: list(r.backward(q, k, v, decay, do, **kw, stream=s).values())),
            (tok, lambda s: [tok.step(q, k, v, decay, cache, slot_idx=slots, stream=s)]),
            (norm, lambda s: list(norm.forward(x, stream=s))),
            (norm, lambda s: [t for t in norm.backward(x, x, None, None, mean, rstd, stream=s).values() if t is not None])]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("which", range(5))
def test_outputs_belong_to_the_given_stream(which, handle):
    """Outputs that are dropped while their stream has yet to write them are not what other tensors get."""
    _, call = _calls()[which]
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    for keep in range(len(want)):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)  # some 50 ms
        got = call(side.cuda_stream if handle else side)
        kept, dropped = got[keep], [(x.data_ptr(), x.shape, x.dtype) for i, x in enumerate(got) if i != keep]
        del got
        others = [torch.full(shape, 7.0, dtype=dtype, device="cuda") for _, shape, dtype in dropped for _ in range(2)]
        assert not {x.data_ptr() for x in others} & {p for p, _, _ in dropped}
        torch.cuda.synchronize()
        assert all((x == 7).all() for x in others)
        assert torch.equal(kept, want[keep])


@pytest.mark.parametrize("backward", [False, True])
def test_outputs_of_the_ssd_runner_belong_to_the_given_stream(backward):
    shape = SsdShape(1, 256, 2, 64, 64, 1, 64, 2)
    t = to_dev(make_inputs(shape, 5, "bf16"))
    r = ssd.SsdRunner(shape, "bf16")

    def call(stream):
        return list(r.backward(t, t["dy"], t["dfinal"], stream=stream).values()) if backward else list(r.forward(t, stream=stream))

    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = call(side)
    kept, dropped = got[0], [(x.data_ptr(), x.shape, x.dtype) for x in got[1:]]
    del got
    others = [torch.full(shape, 7.0, dtype=dtype, device="cuda") for _, shape, dtype in dropped for _ in range(2)]
    assert not {x.data_ptr() for x in others} & {p for p, _, _ in dropped}
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in others) and torch.equal(kept, want[0])


@pytest.mark.parametrize("which", [0, 1, 3, 4])
def test_workspaces_outlive_their_calls(which):
    """A runner that is dropped while another stream has yet to work in its workspace."""
    side = torch.cuda.Stream()
    for current in (False, True):  # stream= and torch.cuda.stream
        calls = _calls()
        r, call = calls[which]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
            if current:
                call(None)
        if not current:
            call(side)
        used, size = r.workspace.data_ptr(), r.workspace.numel()
        del calls, r, call
        others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert used not in {x.data_ptr() for x in others}
        torch.cuda.synchronize()


# ------------------------------------------------------------------ single tokens

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_states_of_many_steps(dtype):
    """6000 steps with decays that live about as long or longer, half a unit in the last place between two fp32 values: an
    error of lam itself would add up to 6000 * 2^-25 of what the state had at first."""
    L, H, d, rows = 6000, 3, 16, 2
    decay = torch.log1p(-torch.tensor([2.**-12 + 2.**-25, 2.**-16 + 2.**-25, 2.**-14 + 2.**-25], dtype=torch.float64)).float()
    c = Case([L] * rows, H, H, d, d, dtype, packed=False, seed=12, decay=decay)
    q, k, v = (x.reshape(rows, L, -1) for x in c.parts("cuda"))
    cache, g = c.init.cuda(), decay.cuda()
    tok = ssd.LinearAttnRunner(rows, 1, H, d, d, dtype=dtype)
    outs = [tok.step(q[:, t], k[:, t], v[:, t], g, cache) for t in range(L)]
    k64, v64 = (x.double().cpu().view(rows, L, H, d) for x in (k, v))
    left = torch.exp(decay.double() * torch.arange(L - 1, -1, -1, dtype=torch.float64)[:, None])  # (L, H)
    want = torch.einsum("rlhk,lh,rlhv->rhkv", k64, left, v64) + c.init.double() * torch.exp(decay.double() * L)[:, None, None]
    close(cache, want, F32, "state")
    o64 = torch.einsum("rhk,rhkv->rhv", q[:, -1].double().cpu().view(rows, H, d), want) * d ** -0.5
    close(outs[-1], o64.reshape(rows, -1), BF16 if dtype == "bf16" else F32, "last token")
    # and what one prompt of all tokens gives
    _, fin = c.runner().forward(*(x.reshape(rows * L, -1) for x in (q, k, v)), g, initial_state=c.init.cuda())
    close(cache, fin.cpu(), 2 * F32, "prompt")


# ------------------------------------------------------------------ group norm

@pytest.mark.parametrize("act", ["silu", "gate"])
@pytest.mark.parametrize("n,m,C,G", [(700, 1, 512, 8), (5, 60, 96, 2), (3, 4000, 96, 4), (2, 20000, 16, 2), (3, 1, 8192, 1)])
def test_group_norm_in_place(n, m, C, G, act):
    """y may be x or z: a team's groups, a cluster's, tiles, rows wider than a block."""
    x, _, w, b, z = (None if t is None else t.cuda() for t in gn_case(n, m, C, G, act, "bf16", 3))
    r = ssd.GroupNormRunner(n, m, C, G, act)
    want = r.forward(x, w, b, z=z)
    for over in ("x", "z") if act == "gate" else ("x",):
        t = {"x": x.clone(), "z": None if z is None else z.clone()}
        got = r.forward(t["x"], w, b, z=t["z"], out=t[over])
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0] is t[over]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,m,C,G", [(2, 5000, 512, 2), (3, 20000, 16, 2),  # tiles: more than 32 of a group, and fewer
                                     (50, 1, 48, 8), (37, 1, 320, 32), (41, 1, 104, 4), (33, 1, 200, 4),  # pairs: teams of 4 to 32
                                     (9, 5, 60, 6), (3, 90, 60, 6), (2, 4099, 20, 2),  # pairs: a warp, a block, a cluster
                                     (41, 1, 15, 5), (41, 1, 63, 3), (2, 3000, 9, 3)])  # single channels: teams, a cluster
def test_group_norm_kernels(n, m, C, G, dtype):
    gn_check(n, m, C, G, "gate", dtype, seed=n + C)


# ------------------------------------------------------------------ linear attention: batches of tokens, many sequences, scales

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv,H,K", [(64, 64, 4, 4), (128, 128, 4, 2), (40, 72, 6, 2), (128, 40, 8, 8), (256, 64, 4, 1)])
def test_steps_of_a_batch(dk, dv, H, K, dtype):
    """Rows enough for the kernels that take 64 columns of a state, in slots in no order, with a scale, into a view."""
    rows, L, scale = 40, 3, 0.3
    decay = torch.log1p(-torch.exp2(torch.linspace(-1, -12, H)))
    decay[0] = -float("inf")
    c = Case([L] * rows, H, K, dk, dv, dtype, packed=False, seed=dk + dv, decay=decay)
    c.scale = scale
    ro, rfin = c.ref()[:2]
    q, k, v = (x.reshape(rows, L, -1) for x in c.parts("cuda"))
    slots = torch.randperm(rows + 3, generator=torch.Generator().manual_seed(1))[:rows].to(torch.int32)
    cache = torch.full((rows + 3, H, dk, dv), 3.0, device="cuda")
    cache[slots.long().cuda()] = c.init.cuda()
    tok = ssd.LinearAttnRunner(rows, 1, H, dk, dv, nheads_kv=K, dtype=dtype)
    for t in range(L):
        buf = torch.full((rows, H * dv + 16), 7.0, dtype=c.qkv.dtype, device="cuda")
        o = tok.step(q[:, t], k[:, t], v[:, t], decay.cuda(), cache, slot_idx=slots.cuda(), scale=scale, out=buf[:, 8:-8])
        close(o, ro.view(rows, L, -1)[:, t], BF16 if dtype == "bf16" else F32, f"token {t}")
        assert (buf[:, :8] == 7).all() and (buf[:, -8:] == 7).all()
    close(cache[slots.long().cuda()], rfin, F32, "state")
    rest = sorted(set(range(rows + 3)) - set(slots.tolist()))
    assert (cache[rest] == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_sequences_than_are_cut(dtype):
    lens = torch.randint(0, 4, (1100,), generator=torch.Generator().manual_seed(2)).tolist()
    Case(lens, 2, 1, 32, 40, dtype, seed=2).check()


@pytest.mark.parametrize("scale", [0.3, -2.0, 0.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales(scale, dtype):
    c = Case([130, 0, 70], 4, 2, 64, 64, dtype, seed=6)
    c.scale = scale
    r = c.runner()
    x = [*c.parts("cuda"), c.decay.cuda()]
    kw = dict(scale=scale, initial_state=c.init.cuda(), cu_seqlens=c.cu.cuda())
    o, fin = r.forward(*x, **kw)
    g = r.backward(*x, c.do.cuda(), dfinal_state=c.dfin.cuda(), **kw)
    ro, rfin, rdq, rdk, rdv, rdinit = c.ref()
    tol = BF16 if dtype == "bf16" else F32
    flat = lambda t: t.reshape(c.T, -1)  # noqa: E731
    for got, want, t, name in ((o, flat(ro), tol, "o"), (fin, rfin, F32, "final state"), (g["dq"], flat(rdq), tol, "dq"),
                               (g["dk"], flat(rdk), tol, "dk"), (g["dv"], flat(rdv), tol, "dv"),
                               (g["dinitial_state"], rdinit, F32, "dinitial_state")):
        close(got, want, t, name)
