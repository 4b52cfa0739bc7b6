"""The retention operators at the edges of what they accept: bounds that are out of order, streams, long runs of tokens,
shapes that take kernels of their own.

Tolerances are those of test_gpu_retention.py."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from tests.test_gpu_retention import BF16, F32, Case, _built, close  # noqa: F401

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
