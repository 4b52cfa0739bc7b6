"""The gated delta rule with keys that are nearly the same: each token takes back what the ones before it wrote, so that outputs
and states are sums of a chunk's additions that cancel, and errors of the additions add up.

Tolerances, relative L2 errors.  bf16: an addition is the sum of two bf16 terms, off by 2^-17 of its size at most, which is up to
twice that of a value; 64 of them add up like a random walk: sqrt(64) * 2 * 2^-17 = 1.2e-4 (STATE) of a state's or an output's
values.  The weights of outputs have two terms as well: twice that, and one rounding of the output, 2^-8 / sqrt(3) = 2.26e-3 of
the norm: 2.5e-3 (OUT).  fp32: F32, by the same count with 2^-24 far below it."""
from __future__ import annotations

import pytest
import torch

from tests import delta_ref as ref
from tests.test_gpu_delta import F32, Case, _built, close  # noqa: F401

pytestmark = pytest.mark.gpu

STATE, OUT = 1.2e-4, 2.5e-3


@pytest.mark.parametrize("dtype,lens,dk,dv,packed", [("bf16", [400], 64, 64, False), ("bf16", [130, 0, 64, 77], 128, 128, True),
                                                     ("bf16", [200, 200], 128, 64, False), ("bf16", [150], 40, 104, False),
                                                     ("bf16", [4500], 64, 64, False), ("bf16", [90], 136, 64, False),
                                                     ("f32", [400], 64, 64, False)])
@pytest.mark.parametrize("noise", [0.0, 0.1, 0.5])
@pytest.mark.parametrize("beta,decay", [(0.5, 0.0), (0.5, -0.02), (1.0, 0.0), (1.0, -0.02)])
def test_keys_that_are_nearly_equal(dtype, lens, dk, dv, packed, noise, beta, decay):
    c = Case(lens, 2, 1, dk, dv, dtype, packed=packed, seed=5, beta=beta, decay=torch.tensor([decay]))
    k = c.qkv[:, dk:2 * dk].float()
    c.qkv[:, dk:2 * dk] = (k[:1] + noise * k).to(c.qkv.dtype)
    o, fin = c.forward()
    want, wfin = ref.delta_rule(*c.ref_inputs(), c.init.double(), c.eps)
    f32 = dtype == "f32"
    close(o, want.reshape(c.T, -1), F32 if f32 else OUT, "o")
    close(fin, wfin, F32 if f32 else STATE, "final_state")
