"""Host-side checks of the retention entry points (no GPU): workspace sizes and
refusals before anything is launched, the runners' argument checks, and the 64-bit
reference's own gradients against differences of its forward."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from mamba2_ssd_selective_gb300.build import build
from tests import retention_ref as ref

INVALID, NULL, ALIGN, DTYPE, WORKSPACE, UNSUPPORTED = -1, -3, -4, -5, -6, -7


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    ssd.load()


def la_dims(**kw):
    d = dict(nseq=2, seqlen=100, total_tokens=0, packed=0, nheads=4, nheads_kv=2, headdim_k=64, headdim_v=64, dtype=0)
    d.update(kw)
    return ssd.SsdLinearAttnDims(**d)


def la_inputs(**kw):  # addresses are never read: every call below is refused on the host
    d = dict(q=4096, q_tok_stride=256, k=4096, k_tok_stride=128, v=4096, v_tok_stride=128, log_decay=4096,
             initial_states=None, cu_seqlens=None, scale=0.125)
    d.update(kw)
    return ssd.SsdLinearAttnInputs(**d)


def refused(status, call, *args):
    with pytest.raises(ssd.SsdError) as e:
        call(*args, stream=0)
    assert e.value.status == status


def test_linear_attn_workspace():
    assert ssd.ssd_linear_attn_workspace_size(la_dims(), False) > 0
    # shared key/value heads: the per-head gradients go through the workspace
    assert ssd.ssd_linear_attn_workspace_size(la_dims(), True) > 200 * 4 * 64 * 4
    for bad in (dict(nseq=0), dict(seqlen=0), dict(nheads=3), dict(nheads_kv=0), dict(headdim_k=0), dict(headdim_v=12),
                dict(headdim_k=264), dict(dtype=2), dict(packed=2), dict(packed=1, total_tokens=0),
                dict(total_tokens=199), dict(nheads=2048, nheads_kv=2048), dict(nseq=2 ** 20, seqlen=2 ** 11)):
        assert ssd.ssd_linear_attn_workspace_size(la_dims(**bad), False) == 0, bad


# (dims, inputs, o, o stride, final, workspace address, bytes, status)
LA_REFUSALS = [
    (dict(nheads=3), {}, 4096, 256, None, INVALID),
    (dict(headdim_k=20), {}, 4096, 256, None, UNSUPPORTED),
    (dict(dtype=7), {}, 4096, 256, None, DTYPE),
    ({}, dict(q=None), 4096, 256, None, NULL),
    ({}, dict(log_decay=None), 4096, 256, None, NULL),
    ({}, dict(k=4104), 4096, 256, None, ALIGN),
    ({}, dict(v_tok_stride=132), 4096, 256, None, ALIGN),
    ({}, dict(k_tok_stride=64), 4096, 256, None, INVALID),
    ({}, dict(cu_seqlens=4096), 4096, 256, None, INVALID),
    (dict(packed=1, total_tokens=9), {}, 4096, 256, None, NULL),
    ({}, dict(scale=float("nan")), 4096, 256, None, INVALID),
    ({}, dict(initial_states=4100), 4096, 256, None, ALIGN),
    ({}, {}, None, 256, None, NULL),
    ({}, {}, 4096, 128, None, INVALID),
    ({}, {}, 4096, 256, 4100, ALIGN),
    ({}, {}, 4096, 256, None, WORKSPACE),
]


@pytest.mark.parametrize("case", range(len(LA_REFUSALS)))
def test_linear_attn_forward_refuses(case):
    dims, inputs, o, stride, fin, status = LA_REFUSALS[case]
    refused(status, ssd.ssd_linear_attn_forward, la_dims(**dims), la_inputs(**inputs), o, stride, fin, None, 0)


def test_linear_attn_backward_refuses():
    def grads(**kw):
        d = dict(dq=4096, dq_tok_stride=256, dk=4096, dk_tok_stride=128, dv=4096, dv_tok_stride=128,
                 dinitial_states=None)
        d.update(kw)
        return ssd.SsdLinearAttnGrads(**d)

    def call(status, dout=4096, stride=256, dfin=None, g=grads()):
        refused(status, ssd.ssd_linear_attn_backward, la_dims(), la_inputs(), dout, stride, dfin, g, None, 0)

    call(NULL, dout=None)
    call(INVALID, stride=248)
    call(ALIGN, dfin=4104)
    call(NULL, g=grads(dk=None))
    call(ALIGN, g=grads(dv=4098))
    call(INVALID, g=grads(dq_tok_stride=128))
    call(ALIGN, g=grads(dinitial_states=4104))
    call(WORKSPACE)


def test_linear_attn_step_refuses():
    def call(status, dims={}, inputs={}, states=4096, nslots=4, idx=None, o=4096, stride=256):
        refused(status, ssd.ssd_linear_attn_step, la_dims(**{"seqlen": 1, **dims}), la_inputs(**inputs), states, nslots,
                idx, o, stride)

    call(INVALID, dims=dict(seqlen=2))
    call(INVALID, dims=dict(packed=1, total_tokens=2))
    call(INVALID, inputs=dict(initial_states=4096))
    call(NULL, states=None)
    call(ALIGN, states=4100)
    call(INVALID, nslots=0)
    call(ALIGN, idx=4098)
    call(NULL, o=None)


def gn_dims(**kw):
    d = dict(nsamples=2, nrows=5, channels=48, groups=3, dtype=0, activation=0)
    d.update(kw)
    return ssd.SsdGroupNormDims(**d)


def gn_inputs(**kw):
    d = dict(x=4096, x_row_stride=48, z=None, z_row_stride=0, weight=None, bias=None, eps=1e-5)
    d.update(kw)
    return ssd.SsdGroupNormInputs(**d)


def test_group_norm_refuses():
    fwd = ssd.ssd_group_norm_forward

    def call(status, dims={}, inputs={}, y=4096, stride=48, mean=None, rstd=None):
        refused(status, fwd, gn_dims(**dims), gn_inputs(**inputs), y, stride, mean, rstd, None, 0)

    for bad in (dict(nsamples=0), dict(nrows=0), dict(groups=5), dict(activation=3), dict(dtype=2),
                dict(channels=131072, groups=2), dict(nsamples=2 ** 20, nrows=2 ** 11)):
        assert ssd.ssd_group_norm_workspace_size(gn_dims(**bad), True) == 0, bad
    call(INVALID, dims=dict(groups=5))
    call(DTYPE, dims=dict(dtype=3))
    call(NULL, inputs=dict(x=None))
    call(ALIGN, inputs=dict(x=4097))
    call(INVALID, inputs=dict(x_row_stride=47))
    call(INVALID, inputs=dict(z=4096, z_row_stride=48))
    call(NULL, dims=dict(activation=2))
    call(ALIGN, inputs=dict(weight=4098))
    call(INVALID, inputs=dict(eps=-1.0))
    call(INVALID, inputs=dict(eps=float("nan")))
    call(NULL, y=None)
    call(ALIGN, mean=4097)
    call(WORKSPACE)
    bwd = ssd.ssd_group_norm_backward
    grads = ssd.SsdGroupNormGrads(4096, 48, None, 0, None, None)
    refused(NULL, bwd, gn_dims(), gn_inputs(), None, 48, 4096, 4096, grads, None, 0)
    refused(NULL, bwd, gn_dims(), gn_inputs(), 4096, 48, None, 4096, grads, None, 0)
    refused(INVALID, bwd, gn_dims(), gn_inputs(), 4096, 48, 4096, 4096,
            ssd.SsdGroupNormGrads(4096, 48, 4096, 48, None, None), None, 0)
    refused(NULL, bwd, gn_dims(activation=2), gn_inputs(z=4096, z_row_stride=48), 4096, 48, 4096, 4096, grads, None, 0)
    refused(WORKSPACE, bwd, gn_dims(), gn_inputs(), 4096, 48, 4096, 4096, grads, None, 0)


def test_runners_check_tensors():
    r = ssd.LinearAttnRunner(2, 3, 4, 16, 8, nheads_kv=2, device="cpu")
    q, k, v, g = (torch.zeros(6, n, dtype=torch.bfloat16) for n in (64, 32, 16, 1))
    decay = torch.zeros(4)
    with pytest.raises(ValueError, match="q: expected"):
        r.forward(q.float(), k, v, decay)
    with pytest.raises(ValueError, match="k: expected"):
        r.forward(q, k[:5], v, decay)
    with pytest.raises(ValueError, match="v: channels"):
        r.forward(q, k, torch.zeros(16, 6, dtype=torch.bfloat16).t(), decay)
    with pytest.raises(ValueError, match="q: rows must be evenly spaced"):
        r.forward(torch.zeros(2, 4, 64, dtype=torch.bfloat16)[:, :3], k, v, decay)
    with pytest.raises(ValueError, match="log_decay"):
        r.forward(q, k, v, decay.double())
    with pytest.raises(ValueError, match="initial_state"):
        r.forward(q, k, v, decay, initial_state=torch.zeros(2, 4, 8, 16))
    with pytest.raises(ValueError, match="cu_seqlens"):
        r.forward(q, k, v, decay, cu_seqlens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="invalid dims"):
        ssd.LinearAttnRunner(2, 3, 4, 12, 8, device="cpu")
    n = ssd.GroupNormRunner(2, 3, 8, 2, "gate", device="cpu")
    x = torch.zeros(2, 3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="z goes with"):
        n.forward(x)
    with pytest.raises(ValueError, match="weight"):
        n.forward(x, torch.ones(7), z=x)


def test_reference_gradients_against_differences():
    """The references' gradients against central differences of their forwards.  The linear attention is linear in
    each of q, k, v and the state, so that any step is exact; the norm's third derivatives leave h^2 ~ 1e-8."""
    gen = torch.Generator().manual_seed(3)
    R = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    lens, H, K, dk, dv = [5, 0, 1, 7], 4, 2, 3, 2
    T, n = sum(lens), len(lens)
    q, k, v, do = R(T, H, dk), R(T, K, dk), R(T, K, dv), R(T, H, dv)
    init, dfin, decay = R(n, H, dk, dv), R(n, H, dk, dv), -torch.rand(H, generator=gen, dtype=torch.float64)
    grads = ref.linear_attn(q, k, v, decay, 0.7, lens, init, do, dfin)[2:]
    for i, x in enumerate((q, k, v, init)):
        e = R(*x.shape)

        def loss(sign):
            a = [q, k, v, init]
            a[i] = x + sign * e
            o, fin = ref.linear_attn(*a[:3], decay, 0.7, lens, a[3])
            return (o * do).sum() + (fin * dfin).sum()

        assert torch.allclose((loss(1) - loss(-1)) / 2, (grads[i] * e).sum(), rtol=1e-10, atol=1e-10)
    x, w, b, z, dy = R(2, 3, 12), R(12), R(12), R(2, 3, 12), R(2, 3, 12)
    for act in ("none", "silu", "gate"):
        got = ref.group_norm(x, 4, w, b, z if act == "gate" else None, act, 1e-5, dy)[3:]
        for i, (t, name) in enumerate(((x, "x"), (w, "w"), (b, "b"), (z, "z"))):
            if name == "z" and act != "gate":
                continue
            e, h = R(*t.shape), 1e-4

            def loss(sign):
                a = {"x": x, "w": w, "b": b, "z": z}
                a[name] = t + sign * h * e
                return (ref.group_norm(a["x"], 4, a["w"], a["b"], a["z"], act)[0] * dy).sum()

            assert torch.allclose((loss(1) - loss(-1)) / (2 * h), (got[i] * e).sum(), rtol=1e-5, atol=1e-6), (act, name)
