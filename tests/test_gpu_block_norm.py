"""The norms around a block on the GPU against the 64-bit formulas.

Tolerances, relative to the norm of the result.  fp32: sums over a row of less than 2^14 values or over less than 2^14 rows, in
blocks, roundings of 2^-24 that add like a random walk: below 2^-24 * 2^7, and a few more of the values themselves, so 1e-5
(F32).  bf16 outputs are rounded once: 2^-8 / sqrt(3) = 2.26e-3 where the values are many, 2^-8 = 3.9e-3 at most (BF16).
A gradient through a norm is a difference, du - n mean(n du) times 1 / rms, which for a row of one channel leaves only
eps / x^2 of du: there a relative bound would ask for more digits than du has.  So an error of 2^-22 of what is
subtracted from (two roundings of each of the two, in fp32) is added to the bound."""
from __future__ import annotations

import itertools

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from tests import delta_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = 1e-5, 2 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssd_selective_gb300.build import build

    build()
    ssd.load()


def close(got, want, what, subtracted=0.0):
    tol = BF16 if got.dtype == torch.bfloat16 else F32
    got, want = got.detach().double().cpu(), want.detach().double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    err, most = float((got - want).norm()), tol * float(want.norm()) + 2 ** -22 * subtracted
    assert err <= most, f"{what}: {err:.2e} > {most:.2e}"


class Case:
    def __init__(self, rows, C, post=True, gate=True, residual=True, pre=True, dtype="bf16", res=None, weights=True, seed=0,
                 pad=0):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.C, self.pad = rows, C, pad
        tt, rt = TYPES[dtype], TYPES[res or dtype]
        # rows with a gap behind each, as in a part of a wider tensor
        R = lambda t: torch.randn(rows, C + pad, generator=g).to(t)[:, :C]  # noqa: E731
        W = lambda on: 1 + 0.25 * torch.randn(C, generator=g) if on and weights else None  # noqa: E731
        self.x, self.z, self.r = R(tt), R(tt) if gate else None, R(rt) if residual else None
        self.pw, self.sc, self.w = W(post), W(True), W(pre)
        self.dh, self.dy = R(rt), R(tt) if pre else None
        self.parts = dict(post_norm=post, gate=gate, residual=residual, pre_norm=pre)
        self.runner = ssd.BlockNormRunner(rows, C, dtype=dtype, residual_dtype=res, **self.parts)

    def cuda(self, t):
        if t is None or t.dim() == 1:
            return None if t is None else t.cuda()
        wide = torch.full((self.rows, self.C + self.pad), 9.0, dtype=t.dtype, device="cuda")
        wide[:, :self.C] = t.cuda()
        return wide[:, :self.C]

    def weights(self):
        return dict(post_weight=self.cuda(self.pw), branch_scale=self.cuda(self.sc), pre_weight=self.cuda(self.w))

    def check(self):
        names = ("x", "r", "z", "pw", "sc", "w")
        leaf = {n: None if getattr(self, n) is None else getattr(self, n).double().clone().requires_grad_() for n in names}
        wh, wy = ref.block_norm(leaf["x"], leaf["r"], leaf["z"], self.parts["post_norm"], self.parts["pre_norm"],
                                leaf["pw"], leaf["sc"], leaf["w"], EPS)
        out = self.runner.forward(self.cuda(self.x), residual=self.cuda(self.r), z=self.cuda(self.z), eps=EPS, **self.weights())
        close(out["h"], wh, "h")
        assert (out["y"] is None) == (wy is None)
        if wy is not None:
            close(out["y"], wy, "y")
        # backward reads the h it is given: gradients at the same point, so h is taken wide enough to be that point
        h = wh.detach().to(self.runner.rdtype)
        loss, part = self.backward_loss(leaf, h), self.backward_loss(leaf, h, True)
        got = self.runner.backward(self.cuda(self.x), self.cuda(h), dh=self.cuda(self.dh), dy=self.cuda(self.dy),
                                   z=self.cuda(self.z), rstd_post=out["rstd_post"],
                                   rstd_pre=None if wy is None else (h.double().square().mean(1) + EPS).rsqrt().float().cuda(),
                                   **self.weights())
        have = {n: t for n, t in leaf.items() if t is not None}
        want = dict(zip(have, torch.autograd.grad(loss, list(have.values()))))
        before = dict(zip(have, torch.autograd.grad(part, list(have.values()))))
        for ours, theirs in (("dx", "x"), ("dz", "z"), ("dresidual", "r"), ("dpost_weight", "pw"), ("dbranch_scale", "sc"),
                             ("dpre_weight", "w")):
            assert (got[ours] is None) == (theirs not in want), ours
            if theirs in want:
                close(got[ours], want[theirs], ours, float(before[theirs].norm()) if theirs in "xr" else 0.0)

    def backward_loss(self, leaf, h, constant_rms=False):
        """<dh, h> + <dy, y> with y taken at the given h, whose difference from the exact one is a constant."""
        wh, _ = ref.block_norm(leaf["x"], leaf["r"], leaf["z"], self.parts["post_norm"], False, leaf["pw"], leaf["sc"], eps=EPS,
                               constant_rms=constant_rms)
        at = wh + (h.double() - wh).detach()
        loss = (wh * self.dh.double()).sum()
        if self.dy is not None:
            rms = torch.sqrt((at * at).mean(-1, keepdim=True) + EPS)
            y = at / (rms.detach() if constant_rms else rms)
            loss = loss + ((y if leaf["w"] is None else y * leaf["w"]) * self.dy.double()).sum()
        return loss


@pytest.mark.parametrize("parts", list(itertools.product([False, True], repeat=4)))
def test_parts(parts):
    post, gate, residual, pre = parts
    for dtype, res in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")):
        Case(37, 136, post, gate, residual, pre, dtype, res, seed=sum(parts)).check()


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,C", [(1, 1), (3, 2), (9, 7), (5, 250), (8, 256), (17, 264), (4, 509), (700, 512), (33, 1000), (7, 1023),
                                    (2, 1026), (650, 2048), (3, 4088), (311, 4096), (2, 4099), (5, 8192), (3, 8200), (2, 16384),
                                    (1, 16383)])
def test_sizes(rows, C, dtype, res):
    Case(rows, C, dtype=dtype, res=res, seed=rows + C).check()


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,C", [(2450, 512), (2433, 264), (1300, 1000), (620, 1502), (350, 1003), (305, 2047), (2500, 248)])
def test_blocks_that_go_through_many_rows(rows, C, dtype, res):
    Case(rows, C, dtype=dtype, res=res, seed=rows + C).check()


@pytest.mark.parametrize("pad", [1, 2, 6, 8])
def test_strided_rows(pad):
    for dtype in ("bf16", "f32"):
        Case(19, 512, dtype=dtype, seed=pad, pad=pad).check()
        Case(5, 2000, dtype=dtype, seed=pad, pad=pad).check()


def test_without_weights():
    for dtype in ("bf16", "f32"):
        Case(21, 768, dtype=dtype, weights=False, seed=4).check()


def test_the_stream_updated_in_place():
    c = Case(200, 1024, res="f32", seed=5)
    args = dict(z=c.cuda(c.z), eps=EPS, **c.weights())
    want = c.runner.forward(c.cuda(c.x), residual=c.cuda(c.r), **args)
    r = c.cuda(c.r)
    got = c.runner.forward(c.cuda(c.x), residual=r, h_out=r, **args)
    assert got["h"] is r and torch.equal(r, want["h"]) and torch.equal(got["y"], want["y"])


def test_gradient_of_the_stream_in_place():
    c = Case(40, 1024, seed=6)
    h = c.cuda(c.r)
    stats = dict(rstd_post=torch.ones(40, device="cuda"), rstd_pre=torch.ones(40, device="cuda"))
    kw = dict(dy=c.cuda(c.dy), z=c.cuda(c.z), **stats, **c.weights())
    dh = c.cuda(c.dh)
    want = c.runner.backward(c.cuda(c.x), h, dh=dh, **kw)
    r, s = c.runner, 1024
    inputs = r._inputs(c.cuda(c.x), kw["z"], None, False, kw["post_weight"], kw["branch_scale"], kw["pre_weight"], 0.0)
    x, dx, dz = c.cuda(c.x), torch.empty_like(dh), torch.empty_like(dh)
    inputs.x = x.data_ptr()
    saved = ssd.SsdBlockNormSaved(h.data_ptr(), s, dh.data_ptr(), s, kw["dy"].data_ptr(), s, stats["rstd_post"].data_ptr(),
                                  stats["rstd_pre"].data_ptr())
    grads = ssd.SsdBlockNormGrads(dx.data_ptr(), s, dz.data_ptr(), s, dh.data_ptr(), s, None, None, None)
    ssd.ssd_block_norm_backward(r.dims, inputs, saved, grads, r.workspace)
    assert torch.equal(dh, want["dresidual"]) and torch.equal(dx, want["dx"]) and torch.equal(dz, want["dz"])


def test_no_gradient_from_elsewhere():
    c = Case(40, 512, seed=7)
    kw = dict(dy=c.cuda(c.dy), z=c.cuda(c.z), rstd_post=torch.ones(40, device="cuda"), rstd_pre=torch.ones(40, device="cuda"),
              **c.weights())
    h = c.cuda(c.r)
    want = c.runner.backward(c.cuda(c.x), h, dh=torch.zeros_like(h), **kw)
    got = c.runner.backward(c.cuda(c.x), h, **kw)
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_a_bad_row_stays_a_row():
    """NaN and infinities of a row reach its own outputs only."""
    c = Case(64, 1024, seed=8)
    good = c.runner.forward(c.cuda(c.x), residual=c.cuda(c.r), z=c.cuda(c.z), eps=EPS, **c.weights())
    c.x[3, 5], c.x[40, 1000] = float("nan"), float("inf")
    bad = c.runner.forward(c.cuda(c.x), residual=c.cuda(c.r), z=c.cuda(c.z), eps=EPS, **c.weights())
    rest = [i for i in range(64) if i not in (3, 40)]
    assert torch.equal(bad["y"][rest], good["y"][rest]) and torch.equal(bad["h"][rest], good["h"][rest])
    assert torch.isnan(bad["y"][3]).all() and torch.isnan(bad["y"][40]).any()


def test_rows_of_zeros():
    c = Case(4, 256, dtype="f32", seed=9)
    for t in (c.x, c.r):
        t.zero_()
    c.check()
