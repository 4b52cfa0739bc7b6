"""The retention example: serving and training with the operators together."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import retention as example  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [(5, 130, 1, 64), (3,), (700, 2)])
def test_tokens_continue_prompts(lengths):
    mixer = example.RetentionMixer(256, 4, 64, 128)
    diff, largest = example.serve(mixer, lengths)
    # Both sides round q, k, v, z, o and y to bf16 (2^-9 each) from the same values, o from different orders of
    # sums: what differs is o's rounding, P's and S's as operands of the whole sequences, and y's
    # after them, 4 x 2^-9 of values that a norm keeps near 1, then averaged by the last product.
    assert diff <= 8 * 2.**-9 * max(1., largest)


def test_training_learns():
    mixer, teacher = example.RetentionMixer(256, 4, 64, 128), example.RetentionMixer(256, 4, 64, 128, seed=7)
    losses = example.train(mixer, teacher)
    assert losses[-1] < 0.7 * losses[0]


def plain_loss(mixer, x, goal, nseq, w_in, w_out, norm_weight):
    """The mixer's training loss in 64 bits, from the definitions."""
    rows, h, dk, dv = x.shape[0], mixer.nheads, mixer.headdim_k, mixer.headdim_v
    q, k, v, z = (x @ w_in).split(mixer.splits, dim=1)
    q, k, v = (t.view(nseq, rows // nseq, h, -1).transpose(1, 2) for t in (q, k, v))
    t = torch.arange(rows // nseq)
    ago = (t[:, None] - t[None]).double()
    decay = torch.exp(mixer.log_decay.cpu().double()[:, None, None] * ago.clamp(min=0)) * (ago >= 0)
    o = (((q @ k.transpose(-1, -2)) * decay * dk**-0.5) @ v).transpose(1, 2)
    u = (o - o.mean(-1, keepdim=True)) / torch.sqrt(o.var(-1, unbiased=False, keepdim=True) + 1e-5)
    y = u.reshape(rows, h * dv) * norm_weight * z * torch.sigmoid(z)
    return ((y @ w_out) - goal).square().mean()


def test_gradients_of_the_mixer():
    mixer = example.RetentionMixer(256, 4, 64, 128)
    gen = torch.Generator().manual_seed(3)
    x, goal = torch.randn(2 * 96, 256, generator=gen), torch.randn(2 * 96, 256, generator=gen)
    for p in mixer.parameters():
        p.requires_grad_(True)
    out = mixer(x.cuda(), mixer.attn_runner(2, 96), mixer.norm_runner(2 * 96))
    got = torch.autograd.grad((out - goal.cuda()).square().mean(), mixer.parameters())
    exact = [p.detach().cpu().double().requires_grad_(True) for p in mixer.parameters()]
    want = torch.autograd.grad(plain_loss(mixer, x.double(), goal.double(), 2, *exact), exact)
    # A gradient goes through bf16 about eight times (x, a weight, the projection, o, y, dy, dx of the norm, dq, dk, dv or
    # dz), each time with an independent relative error of at most 2^-9.
    for g, w in zip(got, want):
        assert (g.cpu().double() - w).norm() <= 8 * 2.**-9 * w.norm()
