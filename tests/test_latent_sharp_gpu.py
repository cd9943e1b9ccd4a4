"""Latent attention behind one large weight: a first token that most of a row's weight is on, and the rest of a
long sequence 6 to 13 nats below it, in units that one CTA holds whole; values that repeat with a period, so that
errors which go by a key's place add up instead of averaging out.

Two bounds, against the definition in float64 (u = 2^-8, half of bf16's eps; docs in csrc/latent_attn.cu):
* element by element: u |out| for the output's rounding; a weight is off by at most u of itself (two terms, of 4
  and 3 significant bits, the second of what the first leaves) and 2^-11 (float16 on the way), and by 2^-13 where
  that is more, against a largest weight of 2^3.5 or more: 2^-16 of it.  Logits: Q's rounding, 2^-16.4 `reach` each.
* the 2-norm of a row's error: rounding to nearest is even over its step, so bf16's is at most u / sqrt(3) of the
  elements in 2-norm (0.00226, where all of them were just above a power of two); the weights' part, were it as
  large as that of a row of few equal weights (two independent terms of at most u, even over their steps, with
  shares that add to 1: u / sqrt(3) / sqrt(2) / sqrt(2) = 0.00113), gives 0.0026 in all.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_fp8_speculative_gb300 import api

pytestmark = pytest.mark.gpu

DESCALE, SCALE = 0.75, 0.0721


def definition(q, keys, see):
    """out, weight, flat, reach of q [rows, 576], keys [n, 576] float64, see [rows, n] (or None: all)."""
    s = SCALE * (q @ keys.T)
    if see is not None:
        s = s.masked_fill(~see, -torch.inf)
    p = torch.softmax(s, -1)
    V = keys[:, :512]
    reach = SCALE * q.abs().amax(-1, keepdim=True) * keys.abs().sum(-1).max()
    return p @ V, p @ V.abs(), p.amax(-1, keepdim=True) * V.abs().sum(0), reach


class Sharp:
    """`seqs` sequences of `length` tokens, the first with a logit `gap` nats above the others', which differ
    by about `spread`; values of the given period (0: all of their own)."""

    def __init__(self, seqs, length, heads, nodes, gap, period, spread=0.0, seed=0, tree=False):
        g = torch.Generator("cuda").manual_seed(seed)
        pages = -(-length // 16)
        self.seqs, self.length, self.heads, self.nodes = seqs, length, heads, nodes
        kinds = period or length
        values = torch.randn(seqs, kinds, 512, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        codes = torch.zeros(seqs, pages * 16, 576, dtype=torch.uint8, device="cuda")
        codes[:, :length, :512] = values[:, torch.arange(length, device="cuda") % kinds]
        codes[:, 0, :512] = torch.randn(seqs, 512, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        codes[:, 0, 512] = 0x38                          # 1.0
        codes[:, :length, 513] = torch.randn(seqs, length, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        order = torch.randperm(seqs * pages, generator=g, device="cuda")
        self.bt = order.view(seqs, pages).int()
        self.cache = torch.empty(seqs * pages, 16, 576, dtype=torch.uint8, device="cuda")
        self.cache[order] = codes.view(-1, 16, 576)
        self.keys = codes[:, :length]
        self.q = torch.zeros(seqs * nodes, heads, 576, dtype=torch.bfloat16, device="cuda")
        # (rows differ a little, so that their weights do)
        shift = torch.rand(seqs * nodes, heads, generator=g, device="cuda") * 0.5
        self.q[..., 512] = (gap + shift) / (SCALE * DESCALE)
        self.q[..., 513] = spread / (SCALE * DESCALE)
        self.sl = torch.full((seqs,), length, dtype=torch.int32, device="cuda")
        self.cu = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * nodes
        self.words = self.mask = None
        if tree:
            rng, words = np.random.default_rng(seed), [1]
            for i in range(1, nodes):
                words.append(words[int(rng.integers(0, i))] | 1 << i)
            self.words = words
            self.mask = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words] * seqs, dtype=torch.int64, device="cuda")

    def check(self, which):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = api.mtp_latent_attn_fwd(self.q, self.cache, self.bt, self.sl, self.cu, DESCALE, SCALE, tree_mask=self.mask, status=status)
        torch.cuda.synchronize()
        assert status.item() == 0 and torch.isfinite(out).all()
        n = self.nodes
        see = torch.ones(n, self.length, dtype=torch.bool)
        for i in range(n):
            word = (2 << i) - 1 if self.words is None else self.words[i]
            for j in range(n):
                see[i, self.length - n + j] = bool(word >> j & 1)
        see = see.repeat_interleave(self.heads, 0).cuda()
        for b in which:
            q = self.q[b * n:(b + 1) * n].double().flatten(0, 1)
            keys = self.keys[b].view(torch.float8_e4m3fn).double() * DESCALE
            want, weight, flat, reach = definition(q, keys, see)
            got = out[b * n:(b + 1) * n].double().flatten(0, 1)
            off = (got - want).abs()
            tol = want.abs() * 2.0 ** -8 + weight * (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -16.4 * reach) + flat * 2.0 ** -16
            assert bool((off <= tol).all()), float((off / tol).max())
            norm = (got - want).norm(dim=-1) / want.norm(dim=-1)
            assert float(norm.max()) <= 0.0026, float(norm.max())


@pytest.mark.parametrize("period", [2, 4, 8, 3, 16, 128, 256, 0])
@pytest.mark.parametrize("gap", [6.0, 7.0, 8.5, 9.5, 11.0, 13.0])
def test_a_full_batch(gap, period):
    """One token of 16 heads, 128 sequences: units of 16 rows."""
    Sharp(128, 4000, 16, 1, gap, period, seed=int(gap * 10) + period).check((0, 50, 127))


@pytest.mark.parametrize("period", [2, 4, 8, 0])
@pytest.mark.parametrize("gap", [7.0, 8.5, 9.5, 11.0])
def test_draft_trees(gap, period):
    """64 nodes of 16 heads over 8191 tokens: units of 64 rows."""
    Sharp(8, 8191, 16, 64, gap, period, seed=int(gap * 10) + period, tree=True).check((0, 7))


@pytest.mark.parametrize("period", [2, 8, 0])
@pytest.mark.parametrize("heads,nodes", [(32, 1), (8, 4), (128, 1)])
def test_other_rows(heads, nodes, period):
    """Units of 32 rows, and the units of 64 of all heads, over 8192 tokens."""
    Sharp(64 if heads == 128 else 152, 8192, heads, nodes, 9.5, period, seed=heads + period).check((0, 31))


@pytest.mark.parametrize("period", [2, 8, 0])
@pytest.mark.parametrize("seqs,length", [(128, 4000), (1, 30000)])
def test_others_that_differ(seqs, length, period):
    """The rest spread over about three nats, in whole units and in pieces."""
    Sharp(seqs, length, 16, 1, 9.5, period, spread=1.0, seed=period).check((0, seqs - 1))


@pytest.mark.parametrize("at", [1, 130, 2000, 3999])
def test_the_large_weight_elsewhere(at):
    """The large one in the middle or at the end: what was before it is scaled down."""
    s = Sharp(128, 4000, 16, 1, 9.5, 2, seed=at)
    pages, rows = s.bt.long(), torch.arange(128, device="cuda")
    flat = s.cache.view(-1, 576)
    first, other = pages[:, 0] * 16, pages[:, at // 16] * 16 + at % 16
    keep = flat[first].clone()
    flat[first] = flat[other]
    flat[other] = keep
    s.keys = s.keys.clone()
    s.keys[rows, 0], s.keys[rows, at] = s.keys[rows, at].clone(), s.keys[rows, 0].clone()
    s.check((0, 127))


@pytest.mark.parametrize("seqs,length,heads", [(128, 4000, 16), (152, 3000, 64), (1, 20000, 16)])
def test_a_large_weight_that_raises_no_reference(seqs, length, heads):
    """A second key 2 to 3.9 nats above the first large one: its weight is whatever the reference that the first one has
    left makes it, no power of two, and most of the row's."""
    s = Sharp(seqs, length, heads, 1, 9.5, 0, seed=heads)
    at = torch.randint(1, length - 1, (seqs,), generator=torch.Generator().manual_seed(1)).cuda()
    rows = torch.arange(seqs, device="cuda")
    s.cache.view(-1, 576)[s.bt.long()[rows, at // 16] * 16 + at % 16, 514] = 0x38
    s.keys[rows, at, 514] = 0x38
    above = 2.0 + 1.9 * torch.rand(seqs, heads, generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    s.q[..., 514] = s.q[..., 512] + (above / (SCALE * DESCALE)).bfloat16()
    s.check(sorted({0, seqs // 2, seqs - 1}))
