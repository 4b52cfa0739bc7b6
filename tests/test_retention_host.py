"""What the retention entry points decide on the host (no GPU)."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from mamba2_ssd_selective_gb300.build import build
from mamba2_ssd_selective_gb300.inputs import SsdShape


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    ssd.load()


def _calls():
    """A runner and a call on it for each operator and direction, with tensors of the CPU."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    attn, tok = (ssd.LinearAttnRunner(2, t, 2, 16, 16, device="cpu") for t in (3, 1))
    norm = ssd.GroupNormRunner(6, 1, 32, 2, device="cpu")
    x, decay, stat = bf(6, 32), torch.zeros(2), torch.zeros(6, 2)
    return [(attn, lambda **kw: attn.forward(x, x, x, decay, **kw)),
            (attn, lambda **kw: attn.backward(x, x, x, decay, x, **kw)),
            (tok, lambda **kw: tok.step(x[:2], x[:2], x[:2], decay, torch.zeros(2, 2, 16, 16), **kw)),
            (norm, lambda **kw: norm.forward(x, **kw)),
            (norm, lambda **kw: norm.backward(x, x, None, None, stat, stat, **kw))]


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


@pytest.mark.parametrize("call", [lambda r: r.forward({}), lambda r: r.forward_varlen({}), lambda r: r.backward({}, None)])
def test_calls_of_the_ssd_runner_enter_its_device(call, monkeypatch):
    class Entered(Exception):
        pass

    def guard(device):
        raise Entered(str(device))

    runner = ssd.SsdRunner(SsdShape(1, 256, 2, 64, 64, 1, 64, 2), "bf16", device="cpu")
    runner.device = torch.device("cuda", 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", guard)
    with pytest.raises(Entered, match="cuda:1"):
        call(runner)


# ------------------------------------------------------------------ outputs on inputs (addresses are never read)

def _refused(call, *args):
    """Status of a call that has all that it needs but for the place of an output."""
    with pytest.raises(ssd.SsdError) as e:
        call(*args, stream=0)
    return e.value.status


INVALID, WS = -1, (4096 * 100, 1 << 40)


def test_linear_attn_outputs_on_inputs_are_refused():
    dims = ssd.SsdLinearAttnDims(2, 100, 0, 0, 4, 4, 64, 64, 0)
    q, k, v, do, s0, s1 = (4096 * i for i in range(1, 7))
    inputs = ssd.SsdLinearAttnInputs(q, 256, k, 256, v, 256, 4096 * 9, s0, None, 0.1)
    for out in (q, k, v):
        assert _refused(ssd.ssd_linear_attn_forward, dims, inputs, out, 256, None, *WS) == INVALID

    def backward(dq=4096 * 10, dk=4096 * 11, dv=4096 * 12, dinit=4096 * 13):
        return _refused(ssd.ssd_linear_attn_backward, dims, inputs, do, 256, s1,
                        ssd.SsdLinearAttnGrads(dq, 256, dk, 256, dv, 256, dinit), *WS)

    for x in (q, k, v, do):
        assert backward(dq=x) == backward(dk=x) == backward(dv=x) == INVALID
    assert backward(dinit=s0) == backward(dinit=s1) == INVALID
    one = ssd.SsdLinearAttnDims(2, 1, 0, 0, 4, 4, 64, 64, 0)
    inputs.initial_states = None
    for out in (q, k, v):
        assert _refused(ssd.ssd_linear_attn_step, one, inputs, s0, 2, None, out, 256) == INVALID


def test_group_norm_outputs_on_inputs_are_refused():
    dims = ssd.SsdGroupNormDims(2, 5, 48, 3, 0, ssd.SSD_ACT_GATE)
    x, z, dy, m, r, dx, dz = (4096 * i for i in range(1, 8))
    inputs = ssd.SsdGroupNormInputs(x, 48, z, 64, None, None, 1e-5)
    for y, stride in ((x, 48), (z, 64)):  # in place only at the same places
        assert _refused(ssd.ssd_group_norm_forward, dims, inputs, y, stride + 8, m, r, *WS) == INVALID
    for bad in [dict(dx=t) for t in (x, z, dy, dz)] + [dict(dz=t) for t in (x, z, dy)]:
        p = {"dx": dx, "dz": dz, **bad}
        grads = ssd.SsdGroupNormGrads(p["dx"], 48, p["dz"], 48, None, None)
        assert _refused(ssd.ssd_group_norm_backward, dims, inputs, dy, 48, m, r, grads, *WS) == INVALID
