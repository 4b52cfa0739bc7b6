"""The block norm's parts in each of its kernels (a row to a block, and blocks that go through rows in a ring in shared memory),
wide rows among many, rows with gaps and tensors updated in place where the ring has them on their way.  Bounds are
test_gpu_block_norm.py's."""
from __future__ import annotations

import itertools

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from tests.test_gpu_block_norm import EPS, Case, _built  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("rows,C", [(37, 1024), (2450, 512), (37, 1003)])
@pytest.mark.parametrize("parts", list(itertools.product([False, True], repeat=4)))
def test_parts(parts, rows, C, weights):
    for dtype, res in KINDS:
        Case(rows, C, *parts, dtype, res, weights=weights, seed=sum(parts)).check()


@pytest.mark.parametrize("dtype,res", KINDS)
@pytest.mark.parametrize("rows,C", [(320, 4104), (330, 5120), (311, 6144), (305, 8192), (310, 8200), (304, 16384), (200, 5001)])
def test_many_wide_rows(rows, C, dtype, res):
    Case(rows, C, dtype=dtype, res=res, seed=rows + C).check()


@pytest.mark.parametrize("dtype,res", KINDS)
@pytest.mark.parametrize("parts", [(True, True, True, True), (False, False, True, True), (False, True, True, False)])
def test_many_wide_rows_of_some_parts(parts, dtype, res):
    Case(320, 6144, *parts, dtype, res, seed=7).check()


@pytest.mark.parametrize("rows,C,pad", [(2450, 512, 8), (1300, 1000, 16), (320, 5120, 8)])
def test_many_rows_with_gaps(rows, C, pad):
    for dtype, res in KINDS:
        Case(rows, C, dtype=dtype, res=res, seed=pad, pad=pad).check()


@pytest.mark.parametrize("rows,C", [(2450, 512), (650, 4096), (320, 5120)])
@pytest.mark.parametrize("dtype,res", KINDS)
def test_the_stream_in_place_among_many_rows(rows, C, dtype, res):
    c = Case(rows, C, dtype=dtype, res=res, seed=C)
    args = dict(z=c.cuda(c.z), eps=EPS, **c.weights())
    x, r = c.cuda(c.x), c.cuda(c.r)
    want = c.runner.forward(x, residual=r, **args)
    got = c.runner.forward(x, residual=r, h_out=r, **args)
    assert got["h"] is r and torch.equal(r, want["h"]) and torch.equal(got["y"], want["y"])
    # and its gradient
    dh, dy = c.cuda(c.dh), c.cuda(c.dy)
    saved = dict(rstd_post=want["rstd_post"], rstd_pre=want["rstd_pre"])
    weights, z = c.weights(), args["z"]
    want = c.runner.backward(x, r, dh=dh, dy=dy, z=z, **saved, **weights)
    inputs = c.runner._inputs(x, z, None, False, weights["post_weight"], weights["branch_scale"], weights["pre_weight"], 0.0)
    dx, dz = torch.empty_like(x), torch.empty_like(x)
    keep = ssd.SsdBlockNormSaved(r.data_ptr(), C, dh.data_ptr(), C, dy.data_ptr(), C, saved["rstd_post"].data_ptr(),
                                 saved["rstd_pre"].data_ptr())
    grads = ssd.SsdBlockNormGrads(dx.data_ptr(), C, dz.data_ptr(), C, dh.data_ptr(), C, None, None, None)
    ssd.ssd_block_norm_backward(c.runner.dims, inputs, keep, grads, c.runner.workspace)
    assert torch.equal(dh, want["dresidual"]) and torch.equal(dx, want["dx"]) and torch.equal(dz, want["dz"])
