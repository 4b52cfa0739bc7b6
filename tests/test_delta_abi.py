"""Host-side checks of the gated delta rule and of the block norm (no GPU): workspace sizes, refusals before anything
is launched, the runners' argument checks, and the 64-bit reference's gradients against differences."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from mamba2_ssd_selective_gb300.build import build
from tests import delta_ref as ref

INVALID, NULL, ALIGN, DTYPE, WORKSPACE, UNSUPPORTED = -1, -3, -4, -5, -6, -7
A, B, C, D, E, F = (4096 * i for i in range(1, 7))  # addresses that are never read


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    ssd.load()


def dr_dims(**kw):
    d = dict(nseq=2, seqlen=100, total_tokens=0, packed=0, nheads=4, nheads_qk=2, headdim_k=64, headdim_v=64, dtype=0,
             qk_norm=1)
    d.update(kw)
    return ssd.SsdDeltaRuleDims(**d)


def dr_inputs(**kw):
    d = dict(q=A, q_tok_stride=128, k=B, k_tok_stride=128, v=C, v_tok_stride=256, log_decay=D, log_decay_tok_stride=4,
             beta=E, beta_tok_stride=4, initial_states=None, cu_seqlens=None, scale=0.125, norm_eps=1e-6)
    d.update(kw)
    return ssd.SsdDeltaRuleInputs(**d)


def refused(status, call, *args):
    with pytest.raises(ssd.SsdError) as e:
        call(*args, stream=0)
    assert e.value.status == status


def test_delta_rule_workspace():
    small = ssd.ssd_delta_rule_workspace_size(dr_dims(), False)
    assert 0 < small < ssd.ssd_delta_rule_workspace_size(dr_dims(), True)
    # packed: a place more for each sequence than the rows would fill
    packed = [ssd.ssd_delta_rule_workspace_size(dr_dims(packed=1, total_tokens=640, nseq=n), False) for n in (1, 11)]
    assert packed[1] > packed[0]
    for bad in (dict(nseq=0), dict(seqlen=0), dict(nheads=3), dict(nheads_qk=0), dict(nheads_qk=3), dict(headdim_k=0),
                dict(headdim_v=12), dict(headdim_k=264), dict(dtype=2), dict(packed=2), dict(qk_norm=2),
                dict(packed=1, total_tokens=0), dict(total_tokens=199), dict(nheads=2048, nheads_qk=2048),
                dict(nseq=2 ** 20, seqlen=2 ** 11)):
        assert ssd.ssd_delta_rule_workspace_size(dr_dims(**bad), False) == 0, bad


# (dims, inputs, o, o stride, final, status)
DR_REFUSALS = [
    (dict(nheads=3), {}, F, 256, None, INVALID),
    (dict(headdim_k=20), {}, F, 256, None, UNSUPPORTED),
    (dict(headdim_v=264), {}, F, 256, None, UNSUPPORTED),
    (dict(dtype=7), {}, F, 256, None, DTYPE),
    ({}, dict(q=None), F, 256, None, NULL),
    ({}, dict(log_decay=None), F, 256, None, NULL),
    ({}, dict(beta=None), F, 256, None, NULL),
    ({}, dict(k=B + 8), F, 256, None, ALIGN),
    ({}, dict(beta=E + 1), F, 256, None, ALIGN),
    ({}, dict(v_tok_stride=260), F, 256, None, ALIGN),
    ({}, dict(k_tok_stride=64), F, 256, None, INVALID),
    ({}, dict(log_decay_tok_stride=3), F, 256, None, INVALID),
    ({}, dict(cu_seqlens=4096), F, 256, None, INVALID),
    (dict(packed=1, total_tokens=9), {}, F, 256, None, NULL),
    ({}, dict(scale=float("nan")), F, 256, None, INVALID),
    ({}, dict(norm_eps=-1.0), F, 256, None, INVALID),
    ({}, dict(initial_states=4100), F, 256, None, ALIGN),
    ({}, {}, None, 256, None, NULL),
    ({}, {}, F, 128, None, INVALID),
    ({}, {}, F, 256, 4100, ALIGN),
    ({}, {}, F, 256, None, WORKSPACE),
]


@pytest.mark.parametrize("case", range(len(DR_REFUSALS)))
def test_delta_rule_forward_refuses(case):
    dims, inputs, o, stride, fin, status = DR_REFUSALS[case]
    refused(status, ssd.ssd_delta_rule_forward, dr_dims(**dims), dr_inputs(**inputs), o, stride, fin, None, 0)


def big(dims, backward):
    return 1 << 20, ssd.ssd_delta_rule_workspace_size(dims, backward)


@pytest.mark.parametrize("o", [A, B, C, D, E])
def test_delta_rule_outputs_that_start_where_an_input_does(o):
    d = dr_dims()
    refused(INVALID, ssd.ssd_delta_rule_forward, d, dr_inputs(), o, 256, None, *big(d, False))


def test_delta_rule_backward_refuses():
    def grads(**kw):
        d = dict(dq=A + (1 << 16), dq_tok_stride=128, dk=B + (1 << 16), dk_tok_stride=128, dv=C + (1 << 16),
                 dv_tok_stride=256, dlog_decay=D + (1 << 16), dlog_decay_tok_stride=4, dbeta=E + (1 << 16),
                 dbeta_tok_stride=4, dinitial_states=None)
        d.update(kw)
        return ssd.SsdDeltaRuleGrads(**d)

    call, d = ssd.ssd_delta_rule_backward, dr_dims()
    args = lambda g, dout=F, dfin=None, ws=(None, 0), dims=d: (dims, dr_inputs(), dout, 256, dfin, g, *ws)  # noqa: E731
    for name in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
        refused(NULL, call, *args(grads(**{name: None})))
    refused(NULL, call, *args(grads(), dout=None))
    refused(INVALID, call, *args(grads(dv_tok_stride=128)))
    refused(INVALID, call, *args(grads(dbeta_tok_stride=2)))
    refused(ALIGN, call, *args(grads(dq=A + 8)))
    refused(ALIGN, call, *args(grads(dinitial_states=4100)))
    refused(ALIGN, call, *args(grads(), dfin=4100))
    refused(WORKSPACE, call, *args(grads()))
    ws = big(d, True)
    refused(WORKSPACE, call, *args(grads(), ws=(ws[0], ws[1] - 1)))
    refused(ALIGN, call, *args(grads(), ws=(ws[0] + 16, ws[1])))
    for name, at in (("dq", A), ("dk", C), ("dv", F), ("dlog_decay", D), ("dbeta", E)):
        refused(INVALID, call, *args(grads(**{name: at}), ws=ws))
    refused(INVALID, call, *args(grads(dinitial_states=1 << 18), dfin=1 << 18, ws=ws))


def test_delta_rule_step_refuses():
    d, call = dr_dims(seqlen=1), ssd.ssd_delta_rule_step
    refused(INVALID, call, dr_dims(), dr_inputs(), 1 << 18, 2, None, F, 256)
    refused(INVALID, call, dr_dims(packed=1, total_tokens=1), dr_inputs(cu_seqlens=A), 1 << 18, 2, None, F, 256)
    refused(INVALID, call, d, dr_inputs(initial_states=A), 1 << 18, 2, None, F, 256)
    refused(NULL, call, d, dr_inputs(), None, 2, None, F, 256)
    refused(INVALID, call, d, dr_inputs(), 1 << 18, 0, None, F, 256)
    refused(ALIGN, call, d, dr_inputs(), (1 << 18) + 4, 2, None, F, 256)
    refused(ALIGN, call, d, dr_inputs(), 1 << 18, 2, 4098, F, 256)
    refused(INVALID, call, d, dr_inputs(), 1 << 18, 2, None, B, 256)


@pytest.mark.parametrize("seed", range(20))
def test_places_of_packed_chunks(seed):
    """Chunk c of sequence s has place start / 64 + s + c: no two share one, and all are inside what is allocated."""
    g = torch.Generator().manual_seed(seed)
    n = int(torch.randint(1, 40, (1,), generator=g))
    lens = torch.randint(0, [3, 70, 300][seed % 3], (n,), generator=g).tolist()
    total = max(1, sum(lens))
    seen, a = set(), 0
    for s, x in enumerate(lens):
        for c in range(-(-x // 64)):
            place = a // 64 + s + c
            assert place not in seen and place < total // 64 + n
            seen.add(place)
        a += x


@pytest.mark.parametrize("seed", range(20))
def test_places_of_packed_segments(seed):
    """The same for segments of n rows: start / n + s."""
    g = torch.Generator().manual_seed(seed)
    nseq, n = int(torch.randint(1, 20, (1,), generator=g)), 64 * int(torch.randint(1, 5, (1,), generator=g))
    lens = torch.randint(0, 900, (nseq,), generator=g).tolist()
    seen, a = set(), 0
    for s, x in enumerate(lens):
        for k in range(-(-x // n)):
            place = a // n + s + k
            assert place not in seen and place < sum(lens) // n + nseq
            seen.add(place)
        a += x


def test_few_long_sequences_are_cut():
    """States of segments are in the workspace exactly where cutting pays."""
    def extra(**kw):
        d = dr_dims(**kw)
        chunks = d.nseq * -(-d.seqlen // 64) * d.nheads
        return ssd.ssd_delta_rule_workspace_size(d, False) / chunks

    whole = extra(nseq=40, seqlen=8192, nheads=4)
    assert extra(nseq=1, seqlen=8192, nheads=4) > 1.05 * whole
    assert abs(extra(nseq=1, seqlen=300, nheads=4) - whole) < 0.05 * whole


# ---------------------------------------------------------------- block norm

def bn_dims(**kw):
    d = dict(rows=10, channels=64, dtype=0, residual_dtype=0, post_norm=1, gate=1, residual=1, pre_norm=1)
    d.update(kw)
    return ssd.SsdBlockNormDims(**d)


def bn_inputs(**kw):
    d = dict(x=A, x_row_stride=64, z=B, z_row_stride=64, residual=C, residual_row_stride=64, post_weight=D,
             branch_scale=D, pre_weight=D, eps=1e-6)
    d.update(kw)
    return ssd.SsdBlockNormInputs(**d)


def test_block_norm_workspace():
    assert ssd.ssd_block_norm_workspace_size(bn_dims()) >= 3 * 64 * 4
    for bad in (dict(rows=0), dict(channels=0), dict(gate=2), dict(post_norm=-1), dict(residual=3), dict(pre_norm=2),
                dict(dtype=2), dict(dtype=1, residual_dtype=0), dict(channels=16385)):
        assert ssd.ssd_block_norm_workspace_size(bn_dims(**bad)) == 0, bad


# (dims, inputs, h, h stride, y, status)
BN_REFUSALS = [
    (dict(rows=0), {}, E, 64, F, INVALID),
    (dict(dtype=3), {}, E, 64, F, DTYPE),
    (dict(dtype=1, residual_dtype=0), {}, E, 64, F, DTYPE),
    (dict(channels=20000), {}, E, 64, F, UNSUPPORTED),
    ({}, dict(x=None), E, 64, F, NULL),
    ({}, dict(z=None), E, 64, F, NULL),
    ({}, dict(residual=None), E, 64, F, NULL),
    (dict(gate=0), {}, E, 64, F, INVALID),
    (dict(residual=0), {}, E, 64, F, INVALID),
    (dict(post_norm=0), {}, E, 64, F, INVALID),
    (dict(pre_norm=0), {}, E, 64, F, INVALID),
    (dict(pre_norm=0), dict(pre_weight=None), E, 64, F, INVALID),
    (dict(pre_norm=0), dict(pre_weight=None), None, 64, None, NULL),
    ({}, dict(x_row_stride=63), E, 64, F, INVALID),
    ({}, dict(x_row_stride=2 ** 31), E, 64, F, UNSUPPORTED),
    ({}, dict(x=A + 1), E, 64, F, ALIGN),
    ({}, dict(branch_scale=D + 2), E, 64, F, ALIGN),
    ({}, dict(eps=float("nan")), E, 64, F, INVALID),
    ({}, dict(eps=-1.0), E, 64, F, INVALID),
    ({}, {}, E, 63, F, INVALID),
    ({}, {}, E, 64, None, NULL),
    ({}, {}, A, 64, F, INVALID),
    ({}, {}, E, 64, B, INVALID),
    ({}, {}, E, 64, C, INVALID),
    ({}, {}, E, 64, E, INVALID),
    ({}, {}, C, 72, F, INVALID),
]


@pytest.mark.parametrize("case", range(len(BN_REFUSALS)))
def test_block_norm_forward_refuses(case):
    dims, inputs, h, hs, y, status = BN_REFUSALS[case]
    d = bn_dims(**dims)
    refused(status, ssd.ssd_block_norm_forward, d, bn_inputs(**inputs), h, hs, y, 64, 1 << 17 if d.post_norm else None,
            1 << 18 if d.pre_norm else None)


def test_block_norm_backward_refuses():
    def saved(**kw):
        d = dict(h=C, h_row_stride=64, dh=D, dh_row_stride=64, dy=E, dy_row_stride=64, rstd_post=F, rstd_pre=F)
        d.update(kw)
        return ssd.SsdBlockNormSaved(**d)

    def grads(**kw):
        d = dict(dx=1 << 16, dx_row_stride=64, dz=1 << 17, dz_row_stride=64, dresidual=1 << 18, dresidual_row_stride=64,
                 dpost_weight=1 << 19, dbranch_scale=1 << 19, dpre_weight=1 << 19)
        d.update(kw)
        return ssd.SsdBlockNormGrads(**d)

    call = ssd.ssd_block_norm_backward
    inputs = bn_inputs(residual=None)
    args = lambda s, g, i=inputs, d=bn_dims(), ws=(None, 0): (d, i, s, g, *ws)  # noqa: E731
    refused(INVALID, call, *args(saved(), grads(), bn_inputs()))  # the residual is not read
    refused(NULL, call, *args(saved(h=None), grads()))
    refused(NULL, call, *args(saved(dy=None), grads()))
    refused(NULL, call, *args(saved(rstd_post=None), grads()))
    refused(NULL, call, *args(saved(rstd_pre=None), grads()))
    refused(NULL, call, *args(saved(), grads(dx=None)))
    refused(NULL, call, *args(saved(), grads(dz=None)))
    refused(NULL, call, *args(saved(), grads(dresidual=None)))
    refused(INVALID, call, *args(saved(), grads(), d=bn_dims(residual=0)))
    refused(ALIGN, call, *args(saved(), grads(dpre_weight=(1 << 19) + 2)))
    refused(WORKSPACE, call, *args(saved(), grads()))
    ws = (1 << 20, ssd.ssd_block_norm_workspace_size(bn_dims()))
    refused(WORKSPACE, call, *args(saved(), grads(), ws=(ws[0], ws[1] - 1)))
    refused(ALIGN, call, *args(saved(), grads(), ws=(ws[0] + 8, ws[1])))
    for name, at in (("dx", A), ("dx", E), ("dz", B), ("dx", C), ("dresidual", C), ("dx", D)):
        refused(INVALID, call, *args(saved(), grads(**{name: at}), ws=ws))
    refused(INVALID, call, *args(saved(), grads(dresidual=D, dresidual_row_stride=72), ws=ws))


# ---------------------------------------------------------------- runners

def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _calls():
    """A runner and a call on it for each operator and direction, with tensors of the CPU."""
    rule, tok = (ssd.DeltaRuleRunner(2, t, 2, 16, 16, device="cpu") for t in (3, 1))
    norm = ssd.BlockNormRunner(6, 32, device="cpu")
    x, n, stat = bf(6, 32), bf(6, 2), torch.zeros(6)
    return [(rule, lambda **kw: rule.forward(x, x, x, n, n, **kw)),
            (rule, lambda **kw: rule.backward(x, x, x, n, n, x, **kw)),
            (tok, lambda **kw: tok.step(x[:2], x[:2], x[:2], n[:2], n[:2], torch.zeros(2, 2, 16, 16), **kw)),
            (norm, lambda **kw: norm.forward(x, residual=x, **kw)),
            (norm, lambda **kw: norm.backward(x, x, dy=x, rstd_pre=stat, **kw))]


@pytest.mark.parametrize("which", range(5))
def test_calls_enter_the_runners_device(which, monkeypatch):
    """A runner of the second GPU makes it the current one, wherever it is called from."""
    runner, call = _calls()[which]
    runner.device = torch.device("cuda", 1)
    current, entered = [0], []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)
            current.append(self.device.index)

        def __exit__(self, *exc):
            current.pop()

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    with pytest.raises(ValueError, match="on cuda:1, got"):  # the tensors are the CPU's: refused, but on the right device
        call()
    assert entered == [torch.device("cuda", 1)] and current == [0]


@pytest.mark.parametrize("which", range(5))
def test_streams_of_another_device_are_refused(which):
    class Stream:
        device = torch.device("cuda", 1)

    runner, call = _calls()[which]
    runner.device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="stream: expected one of cuda:0"):
        call(stream=Stream())


def test_runners_refuse():
    with pytest.raises(ValueError, match="invalid dims"):
        ssd.DeltaRuleRunner(1, 8, 3, 64, 64, nheads_qk=2, device="cpu")
    with pytest.raises(ValueError, match="invalid dims"):
        ssd.BlockNormRunner(4, 32, dtype="f32", residual_dtype="bf16", device="cpu")
    rule = ssd.DeltaRuleRunner(2, 3, 4, 16, 24, nheads_qk=2, device="cpu")
    q, v, n = bf(6, 32), bf(6, 96), bf(6, 4)
    for bad, match in ((dict(q=bf(6, 64)), "q: expected 6 rows of 32"), (dict(v=bf(5, 96)), "v: expected 6 rows"),
                       (dict(k=q.float()), "k: expected torch.bfloat16"), (dict(beta=bf(6, 2)), "beta: expected 6 rows of 4"),
                       (dict(log_decay=n.float()), "log_decay: expected"),
                       (dict(q=bf(6, 64)[:, ::2]), "q: channels must be contiguous"),
                       (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), "cu_seqlens goes with packed"),
                       (dict(initial_state=torch.zeros(2, 4, 24, 16)), "initial_state: expected")):
        kw = {**dict(q=q, k=q, v=v, log_decay=n, beta=n), **bad}
        with pytest.raises(ValueError, match=match):
            rule.forward(**kw)
    norm = ssd.BlockNormRunner(4, 32, gate=True, device="cpu")
    x = bf(4, 32)
    for kw, match in ((dict(residual=x), "z: needed"), (dict(z=x), "residual: needed"),
                      (dict(residual=x, z=x, post_weight=torch.ones(32)), "post_weight goes with"),
                      (dict(residual=x, z=x, pre_weight=torch.ones(31)), "pre_weight: expected")):
        with pytest.raises(ValueError, match=match):
            norm.forward(x, **kw)
    with pytest.raises(ValueError, match="rstd_post goes with"):
        norm.backward(x, x, dy=x, z=x, rstd_pre=torch.ones(4), rstd_post=torch.ones(4))
    with pytest.raises(ValueError, match="dy: needed"):
        norm.backward(x, x, z=x, rstd_pre=torch.ones(4))


# ---------------------------------------------------------------- the reference itself

@pytest.mark.parametrize("eps", [None, 1e-6])
def test_reference_gradients_against_differences(eps):
    g = torch.Generator().manual_seed(3)
    R = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    lens, K, H, dk, dv = [3, 0, 2], 1, 2, 3, 2
    x = [R(5, K, dk), 0.5 * R(5, K, dk), R(5, H, dv), -R(5, H).abs(), torch.sigmoid(R(5, H)), R(3, H, dk, dv)]
    do, df = R(5, H, dv), R(3, H, dk, dv)

    def loss(a):
        o, fin = ref.delta_rule(*a[:5], 0.7, lens, a[5], eps)
        return float((o * do).sum() + (fin * df).sum())

    grads = list(ref.delta_rule_grads(*x[:5], 0.7, lens, do, x[5], df, eps).values())
    for i, t in enumerate(x):
        want = torch.zeros_like(t)
        for j in range(t.numel()):
            d = torch.zeros(t.numel(), dtype=torch.float64)
            d[j] = 1e-6
            up, down = ([y + s * d.view(t.shape) if n == i else y for n, y in enumerate(x)] for s in (1, -1))
            want.view(-1)[j] = (loss(up) - loss(down)) / 2e-6
        assert torch.allclose(grads[i], want, atol=1e-7, rtol=1e-6), i
