"""A small stack of SSM blocks served with this library: packed prompts of
differing lengths, single tokens, and a speculative round with rollback.

    python examples/mixer_block.py

A block is: input projection -> [z | x B C | dt] -> short causal convolution ->
recurrence -> gated norm -> output projection -> residual add and norm.  The
projections are plain matrix products; everything between them is this
library.  The weights are random; the run checks that a prompt taken at once
and the same tokens taken one by one (or as accepted drafts) end in the same
hidden states, up to the rounding of the bf16 activations between the parts.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import state_space_recurrence_amd as rs  # noqa: E402


class Block:
    """One layer for a pool of ``slots`` sequences."""

    def __init__(self, slots: int, dim: int, heads: int, groups: int, *, max_draft: int, seed: int):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.inner, self.heads, self.groups = heads * 64, heads, groups
        channels = self.inner + 2 * groups * 128
        self.split = (self.inner, channels, heads)                       # z | x B C | dt
        self.w_in = (rand(sum(self.split), dim) / math.sqrt(dim)).bfloat16()
        self.w_out = (rand(dim, self.inner) / math.sqrt(self.inner)).bfloat16()
        self.conv = rs.ConvState(slots, heads, groups, rand(channels, 4) / 2, 0.1 * rand(channels), rand(heads) - 2,
                                 max_draft=max_draft)
        rate = torch.rand(heads, generator=g, device="cuda") * math.log(16.0)
        self.ssm = rs.LayerState(slots, heads, groups, -torch.exp(rate), rand(heads), max_draft=max_draft)
        self.w_gate = torch.ones(self.inner, device="cuda")
        self.w_next = torch.ones(dim, device="cuda")

    def _rows(self, hidden):
        return (hidden @ self.w_in.t()).split(self.split, -1)            # views of one row per token

    def _out(self, y, z, residual):
        o = rs.gated_norm(y, z, self.w_gate, groups=self.groups)
        return rs.add_norm(o @ self.w_out.t(), residual, self.w_next, residual_out=residual)[0]

    def prompts(self, hidden, residual, cu, slots, fresh):
        """Packed prompts: hidden, residual [tokens, dim], cu [rows+1] offsets."""
        z, u, dt = self._rows(hidden)
        x, B, C, d = rs.conv_prefill(self.conv, u, dt, cu, fresh=fresh, slots=slots)
        y = rs.prefill_packed(self.ssm, x, B, C, d, cu, fresh=fresh, y_dtype=torch.bfloat16, slots=slots)
        return self._out(y, z, residual)

    def token(self, hidden, residual, slots):
        """One token per row."""
        z, u, dt = self._rows(hidden)
        y = rs.step(self.ssm, *rs.conv_step(self.conv, u, dt, slots=slots), slots=slots)
        return self._out(y, z, residual)

    def drafts(self, hidden, residual, slots):
        """T draft positions per row: hidden, residual [rows, T, dim]; nothing is kept before ``accept``."""
        n, T, dim = hidden.shape
        z, u, dt = self._rows(hidden)
        y = rs.verify(self.ssm, *rs.conv_verify(self.conv, u, dt, slots=slots), slots=slots)
        out = self._out(y.view(n * T, self.heads, 64), z.reshape(n * T, -1), residual.view(n * T, dim))
        return out.view(n, T, dim)

    def accept(self, keep, T, slots):
        rs.conv_accept(self.conv, keep, T, slots=slots)
        rs.accept(self.ssm, keep, T, slots=slots)


class Stack:
    def __init__(self, slots=6, dim=256, heads=8, groups=2, layers=2, max_draft=4):
        self.blocks = [Block(slots, dim, heads, groups, max_draft=max_draft, seed=i) for i in range(layers)]
        self.first = torch.ones(dim, device="cuda")

    def _start(self, embeddings):
        """Residual stream (fp32) and the first block's normed input."""
        e = embeddings.reshape(-1, embeddings.shape[-1]).bfloat16()
        hidden, residual = rs.add_norm(e, torch.zeros_like(e, dtype=torch.float32), self.first)
        return hidden.view(embeddings.shape), residual.view(embeddings.shape)

    def prompts(self, embeddings, cu, slots, fresh=None):
        hidden, residual = self._start(embeddings)
        for b in self.blocks:
            hidden = b.prompts(hidden, residual, cu, slots, fresh)
        return hidden

    def token(self, embeddings, slots):
        hidden, residual = self._start(embeddings)
        for b in self.blocks:
            hidden = b.token(hidden, residual, slots)
        return hidden

    def round(self, embeddings, keep, slots):
        """A speculative round: verify T drafts per row, keep the first keep[row] of them."""
        hidden, residual = self._start(embeddings)
        for b in self.blocks:
            hidden = b.drafts(hidden, residual, slots)
        for b in self.blocks:
            b.accept(keep, embeddings.shape[1], slots)
        return hidden


def main(lengths=(37, 1, 150, 5), tokens=18, dim=256, seed=0, verbose=True):
    """Greatest difference of the hidden states between the two ways, relative to their size."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = len(lengths)
    slots = torch.randperm(n + 2, generator=g, device="cuda")[:n].to(torch.int32)
    seqs = [torch.randn(length + tokens + 4, dim, generator=g, device="cuda") for length in lengths]
    at = lambda t: torch.stack([s[length + t] for s, length in zip(seqs, lengths)])  # noqa: E731

    # prompts at once, then tokens, then a round of four drafts of which some are kept
    a = Stack(n + 2, dim)
    cu = torch.tensor([0, *lengths]).cumsum(0).to(torch.int32).cuda()
    fresh = torch.ones(n, dtype=torch.int32, device="cuda")
    prompt = a.prompts(torch.cat([s[:length] for s, length in zip(seqs, lengths)]), cu, slots, fresh)
    steps = [a.token(at(t), slots) for t in range(tokens)]
    keep = torch.tensor([4, 0, 2, 3, 1, 4][:n], dtype=torch.int32, device="cuda")
    drafts = a.round(torch.stack([at(tokens + t) for t in range(4)], 1), keep, slots)

    # the same tokens one by one
    b = Stack(n + 2, dim)
    worst = 0.0

    def far(u, v):
        return float((u.float() - v.float()).norm() / v.float().norm())

    for r, (s, length) in enumerate(zip(seqs, lengths)):
        one = slots[r:r + 1]
        out = torch.cat([b.token(s[t:t + 1], one) for t in range(length + tokens + 4)])
        worst = max(worst, far(prompt[cu[r]:cu[r + 1]], out[:length]),
                    far(torch.stack([h[r] for h in steps]), out[length:length + tokens]),
                    far(drafts[r], out[length + tokens:]))
    for blk in a.blocks + b.blocks:
        blk.conv.check_device_errors()
        rs.check_device_errors(blk.ssm)
    if verbose:
        print(f"{n} sequences of {lengths} tokens, {tokens} tokens and a round of 4 drafts: "
              f"hidden states differ by {worst:.2e}")
    return worst


if __name__ == "__main__":
    main()
