"""Calls of the gated delta rule and the block norm that the documentation allows and runners do not make: outputs left out,
gradients with strides of their own, gates at odd places, calls without a token."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from tests import delta_ref as ref
from tests.test_gpu_block_norm import Case as Norm
from tests.test_gpu_delta import BF16, F32, TYPES, Case, _built, close  # noqa: F401

pytestmark = pytest.mark.gpu


def c_inputs(r, c, init=None, cu=None):
    keep = [x.contiguous() for x in c.inputs()]
    return keep, r._inputs(*keep, c.scale, init, cu)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_with_strides_of_their_own(dtype):
    """Each gradient is a part of a wider tensor, whose other channels stay; one of the initial state without one given."""
    c = Case([130, 0, 64, 77], 4, 2, 64, 72, dtype, seed=91)
    want = c.backward(init=False)
    c0 = Case([130, 0, 64, 77], 4, 2, 64, 72, dtype, seed=91)
    c0.init = torch.zeros_like(c.init)
    dinit = c0.backward()["dinitial_state"]  # that of an initial state of zeros
    r, cu, do, df = c.runner(), c.cu.cuda(), c.do.cuda(), c.dfinal.cuda()
    keep, inputs = c_inputs(r, c, None, cu)
    ws = torch.empty(ssd.ssd_delta_rule_workspace_size(r.dims, True), dtype=torch.uint8, device="cuda")
    names = ("dq", "dk", "dv", "dlog_decay", "dbeta")
    wide = {n: torch.full((c.T, want[n].shape[1] + p), 3.0, dtype=TYPES[dtype], device="cuda")
            for n, p in zip(names, (8, 16, 24, 3, 5))}
    di = torch.empty_like(dinit)
    g = ssd.SsdDeltaRuleGrads(*(x for n in names for x in (wide[n].data_ptr(), wide[n].shape[1])), di.data_ptr())
    ssd.ssd_delta_rule_backward(r.dims, inputs, do, do.shape[1], df, g, ws)
    for n in names:
        w = want[n].shape[1]
        assert torch.equal(wide[n][:, :w], want[n]) and (wide[n][:, w:] == 3).all(), n
    assert torch.equal(di, dinit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_at_odd_places(dtype):
    """log_decay and beta are aligned to an element, with odd strides."""
    c = Case([100, 65], 3, 3, 64, 64, dtype, seed=92)
    wide = torch.full((c.T, 9), float("nan"), dtype=TYPES[dtype], device="cuda")
    wide[:, 1:4], wide[:, 5:8] = c.gates[:, :3].cuda(), c.gates[:, 3:].cuda()
    q, k, v = c.inputs()[:3]
    gates = wide[:, 1:4], wide[:, 5:8]
    kw = dict(scale=c.scale, initial_state=c.init.cuda(), cu_seqlens=c.cu.cuda())
    for x, y in zip(c.runner().forward(q, k, v, *gates, **kw), c.forward()):
        assert torch.equal(x, y)
    got, want = c.runner().backward(q, k, v, *gates, c.do.cuda(), dfinal_state=c.dfinal.cuda(), **kw), c.backward()
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("lens,H", [([5000], 2), ([70, 0, 6000, 1], 1), ([90, 40], 2)])
def test_without_a_final_state(lens, H):
    """Cut and whole sequences; o a part of a wider tensor."""
    c = Case(lens, H, 1, 64, 64, seed=93)
    want, _ = c.forward()
    wide = torch.full((c.T, 64 * H + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    o, fin = c.forward(final_state=False, out=wide[:, 8:8 + 64 * H])
    assert fin is None and torch.equal(o, want) and (wide[:, :8] == 3).all() and (wide[:, 8 + 64 * H:] == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_sequence_has_a_token(dtype):
    """Rows that belong to nobody: outputs stay, states pass through."""
    c = Case([50, 20], 2, 1, 64, 64, dtype, seed=94)
    r, cu, init, df = c.runner(), torch.full((3,), 40, dtype=torch.int32, device="cuda"), c.init.cuda(), c.dfinal.cuda()
    out = torch.full((c.T, 128), 3.0, dtype=TYPES[dtype], device="cuda")
    _, fin = r.forward(*c.inputs(), scale=c.scale, initial_state=init, cu_seqlens=cu, out=out)
    assert (out == 3).all() and torch.equal(fin, init)
    g = r.backward(*c.inputs(), c.do.cuda(), scale=c.scale, initial_state=init, dfinal_state=df, cu_seqlens=cu)
    assert torch.equal(g["dinitial_state"], df) and ssd.ssd_device_status(r.workspace) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -2.5])
def test_scales(scale, dtype):
    c = Case([100], 2, 1, 64, 64, dtype, packed=False, seed=95)
    c.scale = scale
    if scale:
        c.check_forward()
        c.check_backward()
    else:
        o, fin = c.forward()
        _, wfin = ref.delta_rule(*c.ref_inputs(), c.init.double(), c.eps)
        close(fin, wfin, F32, "final_state")
        g = c.backward()
        assert (o == 0).all() and (g["dq"] == 0).all()


def test_a_step_into_a_part_of_a_tensor():
    for n, H in ((5, 4), (320, 4)):  # both kernels
        c = Case([1] * n, H, 2, 64, 128, packed=False, seed=96)
        states, again = c.init.cuda(), c.init.cuda()
        want = c.runner().step(*c.inputs(), states, scale=c.scale)
        wide = torch.full((n, H * 128 + 16), 3.0, dtype=torch.bfloat16, device="cuda")
        c.runner().step(*c.inputs(), again, scale=c.scale, out=wide[:, 8:8 + H * 128])
        assert torch.equal(wide[:, 8:8 + H * 128], want) and torch.equal(states, again)
        assert (wide[:, :8] == 3).all() and (wide[:, 8 + H * 128:] == 3).all()


@pytest.mark.parametrize("rows,C", [(9, 200), (9, 1003), (2450, 512)])
def test_a_norm_without_its_stream_or_statistics(rows, C):
    """h, rstd_post and rstd_pre may be NULL."""
    c = Norm(rows, C, res="f32", seed=97)
    weights, z, x, res = c.weights(), c.cuda(c.z), c.cuda(c.x), c.cuda(c.r)
    want = c.runner.forward(x, residual=res, z=z, **weights)
    inputs = c.runner._inputs(x, z, res, True, weights["post_weight"], weights["branch_scale"], weights["pre_weight"], 1e-6)
    y = torch.empty_like(x)
    ssd.ssd_block_norm_forward(c.runner.dims, inputs, None, 0, y, C, None, None)
    assert torch.equal(y, want["y"])


@pytest.mark.parametrize("rows,C", [(40, 512), (2450, 512), (33, 1003)])
def test_a_gradient_of_a_weight_in_the_weights_place(rows, C):
    c = Norm(rows, C, seed=98)
    weights, z, x, h = c.weights(), c.cuda(c.z), c.cuda(c.x), c.cuda(c.r)
    stats = [torch.ones(rows, device="cuda") for _ in range(2)]
    dy = c.cuda(c.dy)
    want = c.runner.backward(x, h, dy=dy, z=z, rstd_post=stats[0], rstd_pre=stats[1], **weights)
    inputs = c.runner._inputs(x, z, None, False, weights["post_weight"], weights["branch_scale"], weights["pre_weight"], 0.0)
    saved = ssd.SsdBlockNormSaved(h.data_ptr(), C, None, 0, dy.data_ptr(), C, stats[0].data_ptr(), stats[1].data_ptr())
    dx, dz, dres = (torch.empty_like(x) for _ in range(3))
    grads = ssd.SsdBlockNormGrads(dx.data_ptr(), C, dz.data_ptr(), C, dres.data_ptr(), C,
                                  *(weights[w].data_ptr() for w in ("post_weight", "branch_scale", "pre_weight")))
    ssd.ssd_block_norm_backward(c.runner.dims, inputs, saved, grads, c.runner.workspace)
    assert torch.equal(dx, want["dx"]) and torch.equal(dz, want["dz"]) and torch.equal(dres, want["dresidual"])
    for w in ("post_weight", "branch_scale", "pre_weight"):
        assert torch.equal(weights[w], want["d" + w]), w
