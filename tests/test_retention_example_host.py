"""The retention example's autograd function, with runners of the CPU that stand for the kernels."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import retention as example  # noqa: E402


def kernel(f):
    """Outputs without a graph, as kernels write them."""
    return torch.no_grad()(f)


class Attn:
    """o = q k v, token by token."""

    @kernel
    def forward(self, q, k, v, log_decay, final_state=True):
        return q * k * v, None

    @kernel
    def backward(self, q, k, v, log_decay, do):
        return {"dq": do * k * v, "dk": do * q * v, "dv": do * q * k}


class Norm:
    """y = o weight z."""

    @kernel
    def forward(self, o, weight, z):
        return o * weight * z, None, None

    @kernel
    def backward(self, dy, o, weight, bias, mean, rstd, z):
        return {"dx": dy * weight * z, "dz": dy * o * weight, "dweight": (dy * o * z).sum(0)}


def test_second_derivatives_are_refused():
    """A loss with a penalty on its own gradient: the kernels' gradients are no graph, and the penalty's part would be left
    out without a word."""
    gen = torch.Generator().manual_seed(0)
    q, k, v, z = (torch.randn(3, 4, generator=gen, requires_grad=True) for _ in range(4))
    weight = torch.randn(4, generator=gen, requires_grad=True)
    y = example._Mix.apply(q, k, v, z, weight, torch.zeros(1), Attn(), Norm())
    grads = torch.autograd.grad(y.square().sum(), (q, k, v, z, weight), create_graph=True)
    plain = torch.autograd.grad((q * k * v * weight * z).square().sum(), (q, k, v, z, weight))
    for got, want in zip(grads, plain):
        assert torch.allclose(got, want)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (y.sum() + sum(g.square().sum() for g in grads)).backward()
