"""The gated delta rule and the block norm as programs use them: packed rows with gaps, streams, graphs, waits that give up, large
caches, values that are not numbers, and all parts of a block in a run.

Tolerances are those of test_gpu_delta.py unless a test says otherwise."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from tests import delta_ref as ref
from tests import retention_ref
from tests.test_gpu_delta import BF16, EPS, F32, GRAD, TYPES, Case, _built, close  # noqa: F401

pytestmark = pytest.mark.gpu

TIMEOUT = -9  # SSD_ERR_DEVICE_TIMEOUT


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_outside_the_sequences(dtype):
    """Rows before the first and behind the last sequence are neither read as data nor written."""
    c = Case([40, 70, 0, 90], 4, 2, 64, 64, dtype, seed=31)
    pad = 37
    total = c.T + 2 * pad

    def wide(x, fill):
        out = torch.full((total, x.shape[1]), fill, dtype=x.dtype, device="cuda")
        out[pad:pad + c.T] = x
        return out

    r = ssd.DeltaRuleRunner(c.n, total, 4, 64, 64, nheads_qk=2, qk_norm=True, dtype=dtype, packed=True)
    inputs = [wide(x, float("nan")) for x in c.inputs()]
    cu = (c.cu + pad).cuda()
    out = torch.full((total, 256), 3.0, dtype=TYPES[dtype], device="cuda")
    o, fin = r.forward(*inputs, scale=c.scale, initial_state=c.init.cuda(), cu_seqlens=cu, out=out)
    want, wfin = c.forward()
    close(o[pad:pad + c.T], want.cpu(), F32, "o")
    close(fin, wfin.cpu(), F32, "final")
    assert (o[:pad] == 3).all() and (o[pad + c.T:] == 3).all()
    g = {n: torch.full((total, w), 3.0, dtype=TYPES[dtype], device="cuda")
         for n, w in (("dq", 128), ("dk", 128), ("dv", 256), ("dlog_decay", 4), ("dbeta", 4))}
    di = torch.empty_like(c.init, device="cuda")
    do = wide(c.do.cuda(), float("nan"))
    r.backward(*inputs, do, scale=c.scale, initial_state=c.init.cuda(), cu_seqlens=cu)  # the workspace of backward passes
    init = c.init.cuda()
    args = r._inputs(*inputs, c.scale, init, cu)
    grads = ssd.SsdDeltaRuleGrads(g["dq"].data_ptr(), 128, g["dk"].data_ptr(), 128, g["dv"].data_ptr(), 256,
                                  g["dlog_decay"].data_ptr(), 4, g["dbeta"].data_ptr(), 4, di.data_ptr())
    df = c.dfinal.cuda()
    ssd.ssd_delta_rule_backward(r.dims, args, do, 256, df, grads, r.workspace)
    wg = c.backward()
    for n, x in g.items():
        close(x[pad:pad + c.T], wg[n].cpu(), F32, n)
        assert (x[:pad] == 3).all() and (x[pad + c.T:] == 3).all(), n
    close(di, wg["dinitial_state"].cpu(), F32, "dinitial_state")


@pytest.mark.parametrize("T,n,H,dtype", [(8192, 7, 2, "bf16"), (3000, 30, 4, "bf16"), (900, 7, 2, "f32")])
def test_bounds_in_any_order(T, n, H, dtype):
    """What sequences get is undefined then; empty ones keep their states, nothing hangs, and the next call is right."""
    c = Case([T] + [0] * (n - 1), H, H, 64, 64, dtype, seed=n)
    r, gen = c.runner(), torch.Generator().manual_seed(n)
    inputs, init, do, df = c.inputs(), c.init.cuda(), c.do.cuda(), c.dfinal.cuda()
    for _ in range(4):
        cu = torch.randint(-T // 4, T + T // 4, (n + 1,), generator=gen, dtype=torch.int32)
        _, fin = r.forward(*inputs, scale=c.scale, initial_state=init, cu_seqlens=cu.cuda())
        g = r.backward(*inputs, do, scale=c.scale, initial_state=init, dfinal_state=df, cu_seqlens=cu.cuda())
        assert ssd.ssd_device_status(r.workspace) == 0
        lens = cu[1:].clamp(0, T) - cu[:-1].clamp(0, T)
        for s in (lens <= 0).nonzero()[:, 0].tolist():
            assert torch.equal(fin[s].cpu(), c.init[s]) and torch.equal(g["dinitial_state"][s].cpu(), c.dfinal[s])
    o, fin = r.forward(*inputs, scale=c.scale, initial_state=init, cu_seqlens=c.cu.cuda())
    want, wfin = c.forward()
    assert torch.equal(o, want) and torch.equal(fin, wfin)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["q", "k", "v", "log_decay", "beta"])
def test_a_bad_token_stays_with_its_sequence(what, dtype):
    """A NaN in token 100 of the second sequence: other sequences keep their bits, that sequence's tokens before its chunk too."""
    c = Case([90, 150, 80], 2, 1, 64, 64, dtype, seed=33)
    o, fin = c.forward()
    g = c.backward()
    at = 90 + 100
    col = {"q": 3, "k": 64 + 5, "v": 128 + 7}
    if what in col:
        c.qkv[at, col[what]] = float("nan")
    else:
        c.gates[at, 0 if what == "log_decay" else 2] = float("nan")
    bo, bfin = c.forward()
    bg = c.backward()
    for x, y in [(o, bo)] + [(g[n], bg[n]) for n in ("dq", "dk", "dv", "dlog_decay", "dbeta")]:
        assert torch.equal(x[:90], y[:90]) and torch.equal(x[240:], y[240:])
    assert torch.equal(o[90:90 + 64], bo[90:90 + 64])
    assert torch.isnan(bo[at]).any()
    for x, y in ((fin, bfin), (g["dinitial_state"], bg["dinitial_state"])):
        assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2])
    if what != "q":
        assert torch.isnan(bfin[1]).any()


def test_equal_bits():
    for c in (Case([300, 0, 65, 1, 129], 4, 2, 64, 128, seed=34), Case([4200], 2, 2, 64, 64, packed=False, seed=35)):
        a, b = c.forward(), c.forward()
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        a, b = c.backward(), c.backward()
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_a_cache_of_more_than_2_31_elements():
    slots, H = 4200, 32
    cache = torch.empty(slots, H, 128, 128, device="cuda")
    c = Case([1] * 48, H, H, 128, 128, packed=False, seed=36)
    at = torch.arange(slots - 48, slots, dtype=torch.int32, device="cuda")
    cache[slots - 48:] = c.init.cuda()
    small = c.init.cuda()
    for n in (48, 3):  # the kernel of whole states, and the other
        r = ssd.DeltaRuleRunner(n, 1, H, 128, 128, qk_norm=True)
        inputs = [x[:n] for x in c.inputs()]
        o = r.step(*inputs, cache, slot_idx=at[:n].contiguous(), scale=c.scale)
        want = r.step(*inputs, small, scale=c.scale)
        assert torch.equal(o, want) and torch.equal(cache[slots - 48:], small)


def test_rows_of_more_than_2_31_elements():
    """q, k, v in a tensor whose last rows are beyond 32 bits."""
    c = Case([70], 1, 1, 64, 64, packed=False, seed=37)
    stride = 2 ** 25
    wide = torch.empty(70 * stride, dtype=torch.bfloat16, device="cuda").view(70, stride)
    inputs = list(c.inputs())
    for i, at in ((0, 0), (1, 64), (2, stride - 64)):
        wide[:, at:at + 64] = inputs[i]
        inputs[i] = wide[:, at:at + 64]
    r = c.runner()
    kw = dict(scale=c.scale, initial_state=c.init.cuda())
    want, got = c.forward(), r.forward(*inputs, **kw)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    want, got = c.backward(), r.backward(*inputs, c.do.cuda(), dfinal_state=c.dfinal.cuda(), **kw)
    assert all(torch.equal(want[n], got[n]) for n in want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_outputs_and_batches(dtype):
    """(sequences, tokens, channels) tensors, and an output with a row stride of its own."""
    c = Case([70, 70], 2, 2, 64, 72, dtype, packed=False, seed=38)
    want, _ = c.forward()
    inputs = [x.reshape(2, 70, -1) for x in c.inputs()]
    wide = torch.full((2, 70, 144 + 16), 5.0, dtype=TYPES[dtype], device="cuda")
    o, _ = c.runner().forward(*inputs, scale=c.scale, initial_state=c.init.cuda(), out=wide[..., :144])
    assert torch.equal(o.reshape(140, 144), want) and (wide[..., 144:] == 5).all()


@pytest.mark.parametrize("lens,H,packed", [([200, 200], 4, False), ([4200], 2, False), ([650] * 10, 16, False),
                                           ([900, 0, 700], 3, True)])
def test_waits_that_give_up_are_reported_and_the_next_call_is_clean(lens, H, packed):
    """With the wait limit at 0 every wait that outlasts one parked poll gives up; the kernels drain what they started, return,
    and report it.  A call that reports nothing is right, and afterwards the same call runs clean."""
    c = Case(lens, H, H, 64, 64, packed=packed, seed=41)
    r, inputs, do, init = c.runner(), c.inputs(), c.do.cuda(), c.init.cuda()
    kw = dict(initial_state=init, cu_seqlens=c.cu.cuda() if packed else None, scale=c.scale)

    def call():
        o, fin = r.forward(*inputs, **kw)
        st_f = ssd.ssd_device_status(r.workspace)
        g = r.backward(*inputs, do, **kw)
        return [o, fin, *g.values()], (st_f, ssd.ssd_device_status(r.workspace))

    first, st = call()
    assert st == (0, 0)
    prev = ssd.ssd_set_wait_limit_ns(0)
    try:
        hasty, st = call()
    finally:
        ssd.ssd_set_wait_limit_ns(prev)
    assert st[0] in (0, TIMEOUT) and st[1] in (0, TIMEOUT)
    for x, y in zip(first[:2] * (st[0] == 0), hasty):
        assert torch.equal(x, y)
    for x, y in zip(first[2:] * (st[1] == 0), hasty[2:]):
        assert torch.equal(x, y)
    again, st = call()
    assert st == (0, 0)
    for x, y in zip(first, again):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ streams and graphs

def _operators():
    """(runner, a call of it on a given stream that returns its outputs) for each operator and direction."""
    c = Case([500], 4, 2, 64, 64, packed=False, seed=23)
    inputs, do, init = c.inputs(), c.do.cuda(), c.init.cuda()
    kw = dict(initial_state=init, scale=c.scale)
    r, tok = c.runner(), ssd.DeltaRuleRunner(500, 1, 4, 64, 64, nheads_qk=2, qk_norm=True)
    cache, slots = torch.zeros(1, 4, 64, 64, device="cuda"), torch.full((500,), -1, dtype=torch.int32, device="cuda")
    norm = ssd.BlockNormRunner(500, 256, post_norm=True, gate=True)
    x, z, res, w = (torch.randn(500, 256, device="cuda").bfloat16() for _ in range(4))
    out = norm.forward(x, residual=res, z=z)
    stats = dict(rstd_post=out["rstd_post"], rstd_pre=out["rstd_pre"])
    torch.cuda.synchronize()
    return [(r, lambda s=None: list(r.forward(*inputs, **kw, stream=s))),
            (r, lambda s=None: list(r.backward(*inputs, do, **kw, stream=s).values())),
            (tok, lambda s=None: [tok.step(*inputs, cache, slot_idx=slots, stream=s)]),
            (norm, lambda s=None: [t for t in norm.forward(x, residual=res, z=z, stream=s).values()]),
            (norm, lambda s=None: [t for t in norm.backward(x, out["h"], dy=w, dh=res, z=z, stream=s, **stats).values() if t is not None])]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("which", range(5))
def test_outputs_belong_to_the_given_stream(which, handle):
    """Outputs that are dropped while their stream has yet to write them are not what other tensors get."""
    _, call = _operators()[which]
    want = [x.clone() for x in call()]
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


@pytest.mark.parametrize("which", range(5))
def test_captured(which):
    _, call = _operators()[which]
    want = [x.clone() for x in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        for x in got:
            x.fill_(9)
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_captured_calls_that_share_a_workspace():
    """A prompt and its gradient captured from one runner, replayed in turn, with other inputs at the same places."""
    a, b = (Case([300, 0, 77], 4, 2, 64, 128, packed=True, seed=s) for s in (51, 52))
    r = a.runner()
    held, do, init = [x.clone() for x in a.inputs()], a.do.cuda(), a.init.cuda()
    kw = dict(scale=a.scale, initial_state=init, cu_seqlens=a.cu.cuda())
    calls = (lambda: list(r.forward(*held, **kw)), lambda: list(r.backward(*held, do, **kw).values()))
    graphs = []
    for call in calls:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        graphs.append((graph, got))
    for c in (a, b, a):
        for x, y in zip((*held, do, init), (*c.inputs(), c.do.cuda(), c.init.cuda())):
            x.copy_(y)
        for graph, got in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (graph, got), call in zip(graphs, calls):
            for x, y in zip(got, call()):
                assert torch.equal(x, y)


def test_two_runners_at_once():
    """Each its own workspace: prompts, gradients and norms on two streams side by side give what they give alone."""
    cases = [Case([900, 40], 4, 2, 128, 64, packed=True, seed=s) for s in (61, 62)]
    runners = [c.runner() for c in cases]
    norms = [ssd.BlockNormRunner(700, 512, post_norm=True) for _ in cases]
    x = [torch.randn(700, 512, device="cuda").bfloat16() for _ in cases]
    args = [(c.inputs(), c.do.cuda(), dict(scale=c.scale, initial_state=c.init.cuda(), cu_seqlens=c.cu.cuda())) for c in cases]

    def call(i, stream=None):
        inputs, do, kw = args[i]
        n = norms[i].forward(x[i], residual=x[i], stream=stream)
        g = norms[i].backward(x[i], n["h"], dy=x[i], rstd_post=n["rstd_post"], rstd_pre=n["rstd_pre"], stream=stream)
        return [*runners[i].forward(*inputs, stream=stream, **kw), *runners[i].backward(*inputs, do, stream=stream, **kw).values(),
                n["h"], n["y"], g["dx"], g["dresidual"]]

    want = [call(0), call(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[call(i, s) for i, s in enumerate(streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for both in got:
        for xs, ys in zip(both, want):
            for g, w in zip(xs, ys):
                assert torch.equal(g, w)


def test_a_prompt_of_one_token():
    """A runner of single tokens takes one as a prompt too, and its gradient."""
    c = Case([1, 1, 1], 2, 2, 64, 64, packed=False, seed=42)
    r = c.runner()
    states = c.init.cuda()
    o = r.step(*c.inputs(), states, scale=c.scale)
    p, fin = r.forward(*c.inputs(), scale=c.scale, initial_state=c.init.cuda())
    close(p, o.cpu(), 2 * BF16, "o")
    close(fin, states.cpu(), F32, "states")
    c.check_backward()


# ------------------------------------------------------------------ a block

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_block(dtype):
    """The stream joined and normed, the delta rule, the norm of each head with its gate, the projection's output normed, scaled
    and joined: outputs and gradients against 64 bits.

    fp32: six operators and five products, each within F32 of its inputs' result, and gradients as many again: 22 * 2e-5, as
    random errors sqrt(22) * 2e-5 = 1e-4; 2e-4 leaves the same for what the rule itself makes of errors of its inputs.
    bf16: some 12 roundings forward, 18 more backward, of 2.26e-3 each: sqrt(30) * 2.26e-3 = 1.3e-2 and, for the same reason,
    2.6e-2."""
    lens, H, K, d, C = [100, 30], 4, 2, 64, 256
    T, tt, tol = sum(lens), TYPES[dtype], 2e-4 if dtype == "f32" else 2.6e-2
    g = torch.Generator().manual_seed(50)
    R = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, res = R(T, C).to(tt), R(T, C)
    wq, wk, wv, wz = (R(C, n * d).div(C ** 0.5).to(tt) for n in (K, K, H, H))
    wg, wo = R(C, 2 * H).div(C ** 0.5).to(tt), R(H * d, C).div((H * d) ** 0.5).to(tt)
    w1, w2, w3, sc, wn = 1 + 0.2 * R(C), 1 + 0.2 * R(C), 1 + 0.2 * R(C), 0.5 + 0.1 * R(C), 1 + 0.2 * R(H * d)
    dh, dy = R(T, C), R(T, C).to(tt)

    # 64 bits
    leaf = [t.double().clone().requires_grad_() for t in (x, res, w1, sc)]
    h1, y1 = ref.block_norm(leaf[0], leaf[1], w=leaf[2])
    q, k, v, z, gates = (y1 @ w.double() for w in (wq, wk, wv, wz, wg))
    ld, b = -torch.nn.functional.softplus(gates[:, :H]), torch.sigmoid(gates[:, H:])
    o, _ = ref.delta_rule(q.view(T, K, d), k.view(T, K, d), v.view(T, H, d), ld, b, 1.0, lens, eps=EPS)
    n = retention_ref.group_norm(o.reshape(T, 1, H * d), H, wn, z=z.view(T, 1, -1), act="gate")[0].view(T, -1)
    h2, y2 = ref.block_norm(n @ wo.double(), h1, post_norm=True, pw=w2.double(), sc=leaf[3], w=w3.double())
    want = torch.autograd.grad((h2 * dh.double()).sum() + (y2 * dy.double()).sum(), leaf)

    cu = lambda t: t.cuda()  # noqa: E731
    x, res, wq, wk, wv, wz, wg, wo, w1, w2, w3, sc, wn, dh, dy = map(cu, (x, res, wq, wk, wv, wz, wg, wo, w1, w2, w3, sc, wn, dh, dy))
    join1 = ssd.BlockNormRunner(T, C, dtype=dtype, residual_dtype="f32")
    join2 = ssd.BlockNormRunner(T, C, post_norm=True, dtype=dtype, residual_dtype="f32")
    rule = ssd.DeltaRuleRunner(2, T, H, d, d, nheads_qk=K, qk_norm=True, dtype=dtype, packed=True)
    heads = ssd.GroupNormRunner(T, 1, H * d, H, "gate", dtype)
    bounds = torch.tensor([0, 100, 130], dtype=torch.int32, device="cuda")
    j1 = join1.forward(x, residual=res, pre_weight=w1)
    y1 = j1["y"]
    q, k, v, z = y1 @ wq, y1 @ wk, y1 @ wv, y1 @ wz
    raw = (y1 @ wg).float()
    ld, b = (-torch.nn.functional.softplus(raw[:, :H])).to(tt), torch.sigmoid(raw[:, H:]).to(tt)
    o, _ = rule.forward(q, k, v, ld, b, scale=1.0, cu_seqlens=bounds, final_state=False)
    n, mean, rstd = heads.forward(o, wn, z=z)
    out = n @ wo
    j2 = join2.forward(out, residual=j1["h"], post_weight=w2, branch_scale=sc, pre_weight=w3)
    close(j2["h"], h2.detach(), tol, "h")
    close(j2["y"], y2.detach(), tol, "y")
    g2 = join2.backward(out, j2["h"], dh=dh, dy=dy, post_weight=w2, branch_scale=sc, pre_weight=w3, rstd_post=j2["rstd_post"],
                        rstd_pre=j2["rstd_pre"])
    gn = heads.backward(g2["dx"] @ wo.T, o, wn, None, mean, rstd, z=z)
    gr = rule.backward(q, k, v, ld, b, gn["dx"], scale=1.0, cu_seqlens=bounds)
    draw = torch.cat([-gr["dlog_decay"].float() * torch.sigmoid(raw[:, :H]),
                      gr["dbeta"].float() * torch.sigmoid(raw[:, H:]) * (1 - torch.sigmoid(raw[:, H:]))], 1).to(tt)
    dy1 = gr["dq"] @ wq.T + gr["dk"] @ wk.T + gr["dv"] @ wv.T + gn["dz"] @ wz.T + draw @ wg.T
    g1 = join1.backward(x, j1["h"], dh=g2["dresidual"], dy=dy1, pre_weight=w1, rstd_pre=j1["rstd_pre"])
    for got, w, name in ((g1["dx"], want[0], "dx"), (g1["dresidual"], want[1], "dresidual"), (g1["dpre_weight"], want[2], "dw1"),
                         (g2["dbranch_scale"], want[3], "dscale")):
        close(got, w, tol, name)
