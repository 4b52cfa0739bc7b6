"""The gated delta rule on the GPU against the 64-bit reference.

Tolerances, as relative L2 errors.  fp32 tensors and fp32 states: 2e-5 (F32), by the count of test_gpu_retention.py: sums
of less than 2^17 products, roundings of 2^-24 that add like a random walk, sums in blocks.  A rounding to bf16 is off
by at most 2^-8 of the value and anywhere below: 2^-8 / sqrt(3) = 2.26e-3 of the norm, or less.  bf16 outputs: the output,
the products inside a chunk, the state and the additions as operands are each rounded once: sqrt(4) * 2.26e-3, so
4.6e-3 (BF16).  Gradients have one rounding more, of their weights: sqrt(5) * 2.26e-3, so 5.1e-3 (GRAD).
dlog_decay is a sum of terms of both signs, its error is measured against the
root of its terms' squares (ref.decay_terms).  States of bf16 inputs keep fp32 precision: F32."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from tests import delta_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16, GRAD = 2e-5, 4.6e-3, 5.1e-3
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssd_selective_gb300.build import build

    build()
    ssd.load()


def close(got, want, tol, what="", relative_to=None):
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    err = (got - want).norm() / (want if relative_to is None else relative_to).norm().clamp(min=1e-30)
    assert err <= tol, f"{what}: {err:.2e} > {tol:.2e}"


class Case:
    """Random inputs of one shape: q, k, v are views of one projection's output, log_decay and beta of another's."""

    def __init__(self, lens, H, K, dk, dv, dtype="bf16", packed=True, norm=True, seed=0, decay=None, beta=None):
        g = torch.Generator().manual_seed(seed)
        R = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.lens, self.H, self.K, self.dk, self.dv, self.dtype, self.packed = lens, H, K, dk, dv, dtype, packed
        self.T, self.n, self.norm = sum(lens), len(lens), norm
        tt = TYPES[dtype]
        qkv = R(self.T, 2 * K * dk + H * dv)
        qkv = qkv * torch.sigmoid(qkv)
        if not norm:
            qkv[:, K * dk:2 * K * dk] *= 1.4 * dk ** -0.5
        self.qkv = qkv.to(tt)
        rate = torch.exp(R(H) * 2 - 3)
        ld = -rate * torch.nn.functional.softplus(R(self.T, H)) if decay is None else decay.expand(self.T, H)
        b = torch.sigmoid(R(self.T, H)) if beta is None else torch.as_tensor(beta).expand(self.T, H)
        self.gates = torch.cat([ld, b.float()], 1).to(tt)
        self.do = R(self.T, H * dv).to(tt)
        self.init, self.dfinal = 0.3 * R(self.n, H, dk, dv), R(self.n, H, dk, dv)
        self.scale = 0.8 if norm else dk ** -0.5
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        self.cu = torch.tensor(cu, dtype=torch.int32) if packed else None

    def runner(self, **kw):
        return ssd.DeltaRuleRunner(self.n, self.T if self.packed else self.lens[0], self.H, self.dk, self.dv,
                                   nheads_qk=self.K, qk_norm=self.norm, dtype=self.dtype, packed=self.packed, **kw)

    def inputs(self, device="cuda"):
        """q, k, v, log_decay, beta as a user has them."""
        qkv, gates = self.qkv.to(device), self.gates.to(device)
        return (*qkv.split([self.K * self.dk] * 2 + [self.H * self.dv], 1), *gates.split([self.H, self.H], 1))

    def ref_inputs(self):
        q, k, v, g, b = (x.double() for x in self.inputs("cpu"))
        return (q.view(self.T, self.K, -1), k.view(self.T, self.K, -1), v.view(self.T, self.H, -1), g, b, self.scale,
                self.lens)

    @property
    def eps(self):
        return EPS if self.norm else None

    def forward(self, init=True, **kw):
        return self.runner().forward(*self.inputs(), scale=self.scale, initial_state=self.init.cuda() if init else None,
                                     cu_seqlens=None if self.cu is None else self.cu.cuda(), **kw)

    def backward(self, init=True, dfinal=True, **kw):
        return self.runner().backward(*self.inputs(), self.do.cuda(), scale=self.scale,
                                      initial_state=self.init.cuda() if init else None,
                                      dfinal_state=self.dfinal.cuda() if dfinal else None,
                                      cu_seqlens=None if self.cu is None else self.cu.cuda(), **kw)

    def check_forward(self, init=True):
        o, fin = self.forward(init)
        want, wfin = ref.delta_rule(*self.ref_inputs(), self.init.double() if init else None, self.eps)
        close(o, want.reshape(self.T, -1), F32 if self.dtype == "f32" else BF16, "o")
        close(fin, wfin, F32, "final_state")

    def check_backward(self, init=True, dfinal=True):
        g = self.backward(init, dfinal)
        inp = self.ref_inputs()
        want = ref.delta_rule_grads(*inp, self.do.view(self.T, self.H, -1), self.init if init else None,
                                    self.dfinal if dfinal else None, self.eps)
        tol = F32 if self.dtype == "f32" else GRAD
        for name in ("dq", "dk", "dv", "dbeta"):
            close(g[name], want[name].reshape(self.T, -1), tol, name)
        terms = ref.decay_terms(inp[0], inp[2], inp[3], want, self.lens, self.H // self.K)
        close(g["dlog_decay"], want["dlog_decay"], tol, "dlog_decay", relative_to=terms)
        if init:
            close(g["dinitial_state"], want["dinitial_state"], F32, "dinitial_state")
        else:
            assert g["dinitial_state"] is None


SHAPES = [
    # lens, H, K, dk, dv, packed
    ([1], 1, 1, 64, 64, False),
    ([1, 1, 1], 2, 2, 64, 64, True),
    ([63], 2, 2, 64, 64, False),
    ([64], 2, 1, 64, 64, False),
    ([65, 65], 2, 1, 64, 128, False),
    ([200], 2, 2, 128, 64, False),
    ([130, 1, 0, 64, 77], 4, 2, 128, 128, True),
    ([0, 0, 150, 3], 3, 1, 24, 40, True),
    ([97], 2, 2, 8, 8, False),
    ([70, 70], 4, 4, 72, 120, False),
    ([90, 40], 2, 1, 136, 64, True),
    ([90], 1, 1, 256, 256, False),
    ([75], 2, 2, 104, 200, False),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_forward(shape, norm, dtype):
    lens, H, K, dk, dv, packed = SHAPES[shape]
    Case(lens, H, K, dk, dv, dtype, packed, norm, seed=shape).check_forward(init=shape % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_backward(shape, norm, dtype):
    lens, H, K, dk, dv, packed = SHAPES[shape]
    Case(lens, H, K, dk, dv, dtype, packed, norm, seed=100 + shape).check_backward(init=shape % 3 != 1, dfinal=shape % 3 != 2)


DECAYS = {
    "none": torch.tensor([0.0]),                       # nothing is ever forgotten
    "slow": torch.tensor([-1e-4]),
    "fast": torch.tensor([-3.0]),
    "all": torch.tensor([float("-inf")]),              # every token starts anew
    "far": torch.tensor([-1e30]),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", list(DECAYS))
def test_decays(decay, dtype):
    # no gradient of the decays themselves where they are infinite: the reference has 0 * inf there
    c = Case([150, 66], 2, 1, 64, 64, dtype, seed=7, decay=DECAYS[decay])
    c.check_forward()
    if decay not in ("all", "far"):
        c.check_backward()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_reset_in_the_middle(dtype):
    """Token 70 forgets everything: what follows is as of a new sequence, to fp32's last bits."""
    c = Case([140], 2, 2, 64, 64, dtype, packed=False, seed=8)
    c.gates[70, :2] = float("-inf")
    o, fin = c.forward()
    want, wfin = ref.delta_rule(*c.ref_inputs(), c.init.double(), EPS)
    close(o, want.reshape(140, -1), F32 if dtype == "f32" else BF16, "o")
    close(fin, wfin, F32, "final")
    g = c.backward()
    inp = list(c.ref_inputs())
    inp[3] = inp[3].clamp(min=-300.0)
    want = ref.delta_rule_grads(*inp, c.do.view(140, 2, -1), c.init, c.dfinal, EPS)
    tol = F32 if dtype == "f32" else GRAD
    for name in ("dq", "dk", "dv", "dbeta"):
        close(g[name], want[name].reshape(140, -1), tol, name)
    close(g["dinitial_state"], want["dinitial_state"], F32, "dinitial_state")


@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0])
def test_strengths(beta):
    """beta 0 writes nothing, 1 replaces, 2 reflects (states keep their size)."""
    for dtype in ("f32", "bf16"):
        c = Case([130], 2, 2, 64, 64, dtype, packed=False, seed=9, beta=beta, decay=torch.tensor([-0.02]))
        c.check_forward()
        c.check_backward()


def test_equal_keys():
    """Every key the same, beta 1: each token replaces what the last one wrote; the inverse has entries of both signs."""
    c = Case([100], 1, 1, 64, 64, "f32", packed=False, seed=10, beta=1.0, decay=torch.tensor([0.0]))
    c.qkv[:, 64:128] = c.qkv[:1, 64:128]
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("lens,H,K,dk,dv,packed", [([4500], 2, 1, 64, 64, False), ([4097, 4097], 1, 1, 40, 128, False),
                                                    ([4700], 1, 1, 128, 72, False), ([70, 0, 6000, 1], 1, 1, 64, 64, True)])
@pytest.mark.parametrize("init", [True, False])
def test_cut_sequences(lens, H, K, dk, dv, packed, init):
    """Few long sequences: segments side by side."""
    Case(lens, H, K, dk, dv, "bf16", packed, seed=13).check_forward(init)


def test_cut_sequences_in_place():
    """The states of cut sequences updated in place."""
    c = Case([5000], 2, 2, 64, 64, packed=False, seed=14)
    want, fin = c.forward()
    r, states, o = c.runner(), c.init.cuda(), torch.empty_like(want)
    inputs = r._inputs(*c.inputs(), c.scale, states, None)
    keep = c.inputs()
    for name, x in zip(("q", "k", "v", "log_decay", "beta"), keep):
        setattr(inputs, name, x.data_ptr())
    ssd.ssd_delta_rule_forward(r.dims, inputs, o, 128, states, r.workspace)
    assert torch.equal(o, want) and torch.equal(states, fin)


def test_long_memory_keeps_its_precision():
    """6000 tokens, decays of 1 - 1e-5 that are equal for all tokens: their rounding errors would add up."""
    c = Case([6000], 1, 1, 64, 64, "bf16", packed=False, seed=11, decay=torch.tensor([-1e-5]), beta=0.05)
    c.check_forward()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_continues_a_prompt(dtype):
    """A prompt, then tokens against a cache of states, is the whole sequence as one."""
    tail, lens = 5, [70, 3, 129]
    c = Case([x + tail for x in lens], 4, 2, 64, 128, dtype, seed=12)
    want, wfin = ref.delta_rule(*c.ref_inputs(), c.init.double(), EPS)
    inp, cu = c.inputs(), c.cu.tolist()
    head = torch.cat([torch.arange(cu[s], cu[s] + n) for s, n in enumerate(lens)]).cuda()
    r = ssd.DeltaRuleRunner(3, len(head), 4, 64, 128, nheads_qk=2, qk_norm=True, dtype=dtype, packed=True)
    hcu = torch.tensor([0, 70, 73, 202], dtype=torch.int32, device="cuda")
    o, fin = r.forward(*(x[head].contiguous() for x in inp), scale=c.scale, initial_state=c.init.cuda(), cu_seqlens=hcu)
    close(o, want[head.cpu()].reshape(len(head), -1), F32 if dtype == "f32" else BF16, "prompt")
    cache = torch.full((7, 4, 64, 128), 7.0, device="cuda")
    idx = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    cache[idx.long()] = fin
    tok = ssd.DeltaRuleRunner(3, 1, 4, 64, 128, nheads_qk=2, qk_norm=True, dtype=dtype)
    for t in range(tail):
        rows = torch.tensor([cu[s] + n + t for s, n in enumerate(lens)])
        o = tok.step(*(x[rows.cuda()] for x in inp), cache, slot_idx=idx, scale=c.scale)
        # a step's only rounding is the output's
        close(o, want[rows].reshape(3, -1), F32 if dtype == "f32" else 2 ** -8, f"token {t}")
    close(cache[idx.long()], wfin, F32, "states")
    rest = torch.ones(7, dtype=torch.bool)
    rest[idx.cpu().long()] = False
    assert (cache[rest.cuda()] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 64), (3, 4, 2, 8, 8), (2, 2, 1, 128, 40), (5, 3, 3, 256, 256),
                                   (160, 2, 1, 64, 128), (80, 2, 2, 128, 128), (2, 1, 1, 24, 72),
                                   (310, 4, 2, 128, 128), (700, 2, 1, 40, 64)])
@pytest.mark.parametrize("norm", [True, False])
def test_step(shape, norm, dtype):
    n, H, K, dk, dv = shape
    c = Case([1] * n, H, K, dk, dv, dtype, packed=False, norm=norm, seed=20)
    want, wfin = ref.delta_rule(*c.ref_inputs(), c.init.double(), c.eps)
    states = c.init.cuda()
    o = c.runner().step(*c.inputs(), states, scale=c.scale)
    close(o, want.reshape(n, -1), F32 if dtype == "f32" else 2 ** -8, "o")
    close(states, wfin, F32, "states")


def test_step_without_a_slot():
    c = Case([1] * 4, 2, 2, 64, 64, packed=False, seed=21)
    states = torch.ones(3, 2, 64, 64, device="cuda")
    out = torch.full((4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    c.runner().step(*c.inputs(), states, slot_idx=torch.tensor([-1, 3, 1, 2 ** 30], dtype=torch.int32, device="cuda"), out=out)
    assert (out[[0, 1, 3]] == 0).all() and (out[2] != 0).any()
    assert (states[0] == 1).all() and (states[2] == 1).all() and (states[1] != 1).any()


@pytest.mark.parametrize("dv", [64, 128])
def test_step_without_a_slot_among_many(dv):
    """The kernel of whole states: rows without a slot leave the cache alone, states of others are not touched."""
    n, H, dk = 330, 4, 48
    c = Case([1] * n, H, H, dk, dv, "f32", packed=False, seed=22)
    g = torch.Generator().manual_seed(1)
    slots = torch.randperm(400, generator=g)[:n].to(torch.int32)
    slots[::7] = -1
    slots[3::50] = 400
    cache = torch.randn(400, H, dk, dv, generator=g)
    states = cache.cuda()
    o = c.runner().step(*c.inputs(), states, slot_idx=slots.cuda(), scale=c.scale)
    live = (slots >= 0) & (slots < 400)
    want, wfin = ref.delta_rule(*c.ref_inputs(), cache.double()[slots.long().clamp(0, 399)], EPS)
    close(o[live.cuda()], want.reshape(n, -1)[live], F32, "o")
    assert (o[~live.cuda()] == 0).all()
    at = slots[live].long()
    close(states[at.cuda()], wfin[live], F32, "states")
    rest = torch.ones(400, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(states[rest.cuda()].cpu(), cache[rest])


def test_step_many_tokens_of_a_long_memory():
    """3000 steps with equal decays of 1 - 2^-11: a decay that is off by its rounding would show in the state."""
    H = 2
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(3000, 1, H * 64, generator=g).bfloat16() for _ in range(3))
    ld = torch.full((1, H), -2.0 ** -11).bfloat16()
    b = torch.full((1, H), 2.0 ** -7).bfloat16()
    r = ssd.DeltaRuleRunner(1, 1, H, 64, 64, qk_norm=True)
    states = torch.zeros(1, H, 64, 64, device="cuda")
    qc, kc, vc, lc, bc = q.cuda(), k.cuda(), v.cuda(), ld.cuda(), b.cuda()
    for t in range(3000):
        r.step(qc[t], kc[t], vc[t], lc, bc, states)
    wide = lambda x: x.double().view(3000, H, 64)  # noqa: E731
    _, want = ref.delta_rule(wide(q), wide(k), wide(v), ld.double().expand(3000, H), b.double().expand(3000, H), 1.0, [3000], eps=EPS)
    close(states, want, F32, "states")
