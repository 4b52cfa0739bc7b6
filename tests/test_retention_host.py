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
