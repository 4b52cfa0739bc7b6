"""A retention mixer served and trained with libssd's operators.

    python examples/retention.py

Serving: prompts of different lengths, packed into one row, give the states of their last tokens, which go into a
cache; then each sequence takes one token at a time.  Training: the same mixer learns what another one does, with
gradients through linear attention and the gated norm of each head.  Projections are plain matrix products.
"""
from __future__ import annotations

import math
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba2_ssd_selective_gb300 as ssd  # noqa: E402


class _Mix(torch.autograd.Function):
    """Linear attention, then the norm of each head times silu of a gate.  Its gradients have no derivatives of their own."""

    @staticmethod
    def forward(ctx, q, k, v, z, weight, log_decay, attn, norm):
        o, _ = attn.forward(q, k, v, log_decay, final_state=False)
        y, mean, rstd = norm.forward(o, weight, z=z)
        ctx.save_for_backward(q, k, v, z, weight, log_decay, o, mean, rstd)
        ctx.runners = attn, norm
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        q, k, v, z, weight, log_decay, o, mean, rstd = ctx.saved_tensors
        attn, norm = ctx.runners
        n = norm.backward(dy.contiguous(), o, weight, None, mean, rstd, z=z)
        a = attn.backward(q, k, v, log_decay, n["dx"])
        return a["dq"], a["dk"], a["dv"], n["dz"], n["dweight"], None, None, None


class RetentionMixer:
    """x -> out of one layer: q, k, v and the gate are projections of x, heads decay at fixed rates."""

    def __init__(self, width: int, nheads: int, headdim_k: int, headdim_v: int, seed: int = 0, device="cuda"):
        gen = torch.Generator(device="cpu").manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen) / math.sqrt(rows)).to(device)

        self.nheads, self.headdim_k, self.headdim_v, self.device = nheads, headdim_k, headdim_v, device
        self.splits = [nheads * headdim_k, nheads * headdim_k, nheads * headdim_v, nheads * headdim_v]
        self.w_in, self.w_out = weight(width, sum(self.splits)), weight(nheads * headdim_v, width)
        self.norm_weight = torch.ones(nheads * headdim_v, device=device)
        # head h forgets half in 2^(h + 3) tokens
        self.log_decay = -math.log(2.) / 2. ** torch.arange(3, 3 + nheads, dtype=torch.float32, device=device)

    def parameters(self):
        return [self.w_in, self.w_out, self.norm_weight]

    def attn_runner(self, nseq: int, tokens: int, packed: bool = False):
        return ssd.LinearAttnRunner(nseq, tokens, self.nheads, self.headdim_k, self.headdim_v, packed=packed)

    def norm_runner(self, rows: int):
        return ssd.GroupNormRunner(rows, 1, self.nheads * self.headdim_v, self.nheads, "gate")

    def project(self, x):
        """q, k, v and the gate: views of one projection of x (rows, width)."""
        return (x.bfloat16() @ self.w_in.bfloat16()).split(self.splits, dim=1)

    def __call__(self, x, attn, norm):
        """Training: x (nseq * tokens, width) in fp32, the runners of that shape."""
        q, k, v, z = self.project(x)
        y = _Mix.apply(q, k, v, z, self.norm_weight, self.log_decay, attn, norm)
        return (y @ self.w_out.bfloat16()).float()

    @torch.no_grad()
    def prompt(self, x, cu_seqlens):
        """Packed prompts x (rows, width): outputs, and the states (sequences, heads, headdim_k, headdim_v)."""
        q, k, v, z = self.project(x)
        attn = self.attn_runner(cu_seqlens.numel() - 1, x.shape[0], packed=True)
        o, states = attn.forward(q, k, v, self.log_decay, cu_seqlens=cu_seqlens)
        y, _, _ = self.norm_runner(x.shape[0]).forward(o, self.norm_weight, z=z)
        return (y @ self.w_out.bfloat16()).float(), states

    @torch.no_grad()
    def token(self, x, cache, slots, attn, norm):
        """One token of each row of x, its state in cache[slots]; the runners are those of x's rows."""
        q, k, v, z = self.project(x)
        o = attn.step(q, k, v, self.log_decay, cache, slot_idx=slots)
        y, _, _ = norm.forward(o, self.norm_weight, z=z)
        return (y @ self.w_out.bfloat16()).float()


def serve(mixer: RetentionMixer, lengths=(5, 130, 1, 64), new_tokens: int = 8, width: int = 256):
    """Largest difference between tokens that continue packed prompts one at a time and the same sequences given
    whole, and the largest output."""
    gen = torch.Generator(device="cpu").manual_seed(1)
    whole = [torch.randn(n + new_tokens, width, generator=gen).to(mixer.device) for n in lengths]
    n = len(lengths)

    def bounds(ls):
        return torch.tensor([0, *torch.tensor(ls).cumsum(0).tolist()], dtype=torch.int32, device=mixer.device)

    _, states = mixer.prompt(torch.cat([x[:m] for x, m in zip(whole, lengths)]), bounds(lengths))
    # a cache with room for more sequences, these ones anywhere in it
    slots = torch.arange(2 * n - 1, 0, -2, dtype=torch.int32, device=mixer.device)
    cache = torch.zeros((2 * n,) + states.shape[1:], device=mixer.device)
    cache[slots.long()] = states
    attn, norm = mixer.attn_runner(n, 1), mixer.norm_runner(n)
    got = [mixer.token(torch.stack([x[m + i] for x, m in zip(whole, lengths)]), cache, slots, attn, norm)
           for i in range(new_tokens)]
    want, _ = mixer.prompt(torch.cat(whole), bounds([m + new_tokens for m in lengths]))
    want = torch.stack([w[-new_tokens:] for w in want.split([m + new_tokens for m in lengths])], dim=1)
    return (torch.stack(got) - want).abs().max().item(), want.abs().max().item()


def train(mixer: RetentionMixer, teacher: RetentionMixer, steps: int = 30, nseq: int = 4, tokens: int = 256,
          width: int = 256, rate: float = 2e-3):
    """Losses of `steps` steps of Adam towards the teacher's outputs."""
    gen = torch.Generator(device="cpu").manual_seed(2)
    x = torch.randn(nseq * tokens, width, generator=gen).to(mixer.device)
    attn, norm = mixer.attn_runner(nseq, tokens), mixer.norm_runner(nseq * tokens)
    with torch.no_grad():
        target = teacher(x, attn, norm)
    for p in mixer.parameters():
        p.requires_grad_(True)
    opt = torch.optim.Adam(mixer.parameters(), lr=rate)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (mixer(x, attn, norm) - target).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    for p in mixer.parameters():
        p.requires_grad_(False)
    return [v.item() for v in losses]


def main() -> None:
    mixer, teacher = RetentionMixer(256, 4, 64, 128), RetentionMixer(256, 4, 64, 128, seed=7)
    diff, largest = serve(mixer)
    print(f"tokens one at a time against whole sequences: largest difference {diff:.4f} of outputs up to {largest:.2f}")
    losses = train(mixer, teacher)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")


if __name__ == "__main__":
    main()
