"""Latent attention on the GPU against the float64 definition.

The tolerance, element by element, from the arithmetic (docs in csrc/latent_attn.cu; u = 2^-8 is half of
bf16's eps):
* the output's rounding: u |out|;
* q in two e4m3 terms: an element is off by at most 2^-10 where the row's largest is 224 or more, so
  2^-17 of it, and float32 sums of 576 products add 2^-18 of the same: 2^-16.4 `reach` on a logit, twice
  that on a weight relative to the others;
* a weight in two e4m3 terms: 2^-8 of it (4 significant bits, then 4 of the rest), 2^-11 for float16 on the
  way, and an absolute part of 2^-9 against a largest weight of at least 2^7: 2^-16 of the largest.  (Where a
  reference has been raised in the middle of a long row, with room, the largest weight may be 2^3.5, and one key's
  absolute part 2^-12.5 of it.  The dither spreads such parts evenly about zero over a tile's keys, so that sums of
  many keep to 2^-16 all the same; rows of up to two tiles have no room.)
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from oracle.latent import latent_attention
from paged_fp8_speculative_gb300 import api, rope

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    def __init__(self, lens, nodes, heads, seed=0, q_scale=1.0, masks=None, spare=2, behind=0, base=0, pad=0, width=0):
        g = torch.Generator().manual_seed(seed)
        per = [-(-n // 16) for n in lens]
        self.pages = sum(per) + spare
        order = torch.randperm(self.pages, generator=g)
        bt = torch.full((len(lens), max(per + [1, width])), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            bt[b, :n] = order[at:at + n]
            at += n
        cu = [base]
        for n in nodes:
            cu.append(cu[-1] + n)
        self.total = cu[-1] + behind
        self.lens, self.nodes, self.heads, self.cu_list = lens, nodes, heads, cu
        codes = torch.randn(self.pages, 16, 576, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
        self.cache = codes.cuda()
        self.bt, self.sl, self.cu = bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(cu, dtype=torch.int32).cuda()
        rows = (torch.randn(self.total, heads, 576 + pad, generator=g) * q_scale).bfloat16().cuda()
        self.q = rows[..., :576]
        self.masks = masks
        self.mask = None if masks is None else torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.descale, self.scale = 0.75, 1.0 / np.sqrt(192)

    def run(self, **kw):
        out = kw.pop("out", None)
        if out is None:
            out = torch.full((self.total, self.heads, 512), 9.0, dtype=torch.bfloat16, device="cuda")
        api.mtp_latent_attn_fwd(self.q, self.cache, self.bt, self.sl, self.cu, self.descale, self.scale, tree_mask=self.mask,
                                out=out, status=self.status, **kw)
        torch.cuda.synchronize()
        return out

    def want(self):
        return latent_attention(f64(self.q), self.cache.cpu().numpy(), self.bt.cpu().numpy(), self.lens, self.cu_list, self.masks,
                                self.descale, self.scale)

    def check(self, out, skip=()):
        want, weight, flat, reach = self.want()
        got = f64(out)
        tol = np.abs(want) * 2.0 ** -8 + weight * (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -16.4 * reach) + flat * 2.0 ** -16
        rows = [t for b in range(len(self.lens)) if b not in skip for t in range(self.cu_list[b], self.cu_list[b + 1])]
        bad = np.abs(got - want)[rows] > tol[rows]
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], (np.abs(got - want) / np.maximum(tol, 1e-30))[rows].max())
        outside = [t for t in range(self.total) if not self.cu_list[0] <= t < self.cu_list[-1]]
        assert np.all(got[outside] == 9.0)


@pytest.mark.parametrize("heads", [1, 5, 16, 17, 32, 64, 100, 128])
@pytest.mark.parametrize("nodes", [1, 2, 4])
def test_heads_and_tokens(heads, nodes):
    b = Batch([300, 129, 128, nodes], [nodes] * 4, heads, seed=heads + nodes, behind=1, base=1)
    out = b.run()
    assert b.status.item() == 0
    b.check(out)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 112, 113, 127, 128, 129, 143, 144, 145, 255, 256, 257, 385])
def test_lengths(length):
    b = Batch([length, 1, length], [1, 1, min(length, 3)], 16, seed=length)
    b.check(b.run())


def chain(n):
    return [(2 << i) - 1 for i in range(n)]


def tree(n, seed):
    rng, words = np.random.default_rng(seed), [1]
    for i in range(1, n):
        words.append(words[int(rng.integers(0, i))] | 1 << i)
    return words


@pytest.mark.parametrize("heads", [1, 4, 16, 128])
@pytest.mark.parametrize("nodes", [[64], [5, 64, 1], [33, 17]])
def test_trees(heads, nodes):
    lens = [n + 50 * i for i, n in enumerate(nodes)]
    masks = sum((tree(n, i) for i, n in enumerate(nodes)), [])
    b = Batch(lens, nodes, heads, seed=heads, masks=masks)
    b.check(b.run())


WIDE = 20000                                             # pages a table: too many tiles for units of 16 rows


@pytest.mark.parametrize("heads", [5, 17, 32, 64, 100, 128])
@pytest.mark.parametrize("nodes", [1, 2, 4])
def test_wide_tables(heads, nodes):
    """Tables far longer than the sequences, so that a unit takes as many rows as there are, up to 64."""
    b = Batch([300, 129, 128, nodes], [nodes] * 4, heads, seed=heads + nodes, behind=1, base=1, width=WIDE)
    out = b.run()
    assert b.status.item() == 0
    b.check(out)


@pytest.mark.parametrize("length", [3, 15, 16, 17, 31, 33, 63, 64, 65, 112, 113, 127, 128, 129, 143, 144, 145, 255, 256, 257, 385])
@pytest.mark.parametrize("heads", [10, 20])
def test_lengths_of_wide_tables(length, heads):
    b = Batch([length, 3, length], [2, 3, 3], heads, seed=length, width=WIDE)
    b.check(b.run())


@pytest.mark.parametrize("heads", [1, 4, 16, 128])
@pytest.mark.parametrize("nodes", [[64], [5, 64, 1], [33, 17]])
def test_trees_of_wide_tables(heads, nodes):
    lens = [n + 50 * i for i, n in enumerate(nodes)]
    b = Batch(lens, nodes, heads, seed=heads, masks=sum((tree(n, i) for i, n in enumerate(nodes)), []), width=WIDE)
    b.check(b.run())


@pytest.mark.parametrize("length", [3, 200])
@pytest.mark.parametrize("heads", [10, 20])
def test_rows_of_wide_tables_that_see_little(length, heads):
    b = Batch([length, length], [3, 3], heads, masks=[0, 4, 1, 2, 0, 7], width=WIDE)
    out = b.run()
    b.check(out)
    if length == 3:
        assert not out[0].any() and not out[4].any()


@pytest.mark.parametrize("heads", [10, 20])
def test_codes_of_wide_tables_that_do_not_matter(heads):
    """NaN codes behind the sequences, and in a token that only itself sees; a row of q that is not finite."""
    b = Batch([70, 200], [3, 3], heads, masks=[1, 3, 5, 1, 3, 5], width=WIDE)
    clean = b.run()
    b.check(clean)
    used = torch.zeros(b.pages, 16, dtype=torch.bool)
    for s, n in enumerate(b.lens):
        at = torch.arange(n)
        used[b.bt[s].cpu().long()[at // 16], at % 16] = True
    b.cache[~used.cuda()] = 0x7f
    assert torch.equal(b.run(), clean)
    for s, n in enumerate(b.lens):
        b.cache[b.bt[s, (n - 1) // 16].long(), (n - 1) % 16] = 0xff
    b.q[1, 3, 570] = float("inf")
    out = b.run()
    assert torch.isnan(out[2]).all() and torch.isnan(out[5]).all() and torch.isnan(out[1, 3]).all()
    out[1, 3] = clean[1, 3]
    assert torch.equal(out[[0, 1, 3, 4]], clean[[0, 1, 3, 4]])


def test_errors_of_wide_tables():
    b = Batch([300, 300, 2000, 70], [4, 4, 4, 4], 16, width=WIDE)
    good = b.run()
    b.check(good)
    for change, bit in ((lambda: b.bt.__setitem__((1, 3), b.pages), api.ERR_PAGE), (lambda: b.sl.__setitem__(1, 3), api.ERR_QLEN_GT_SEQ),
                        (lambda: b.sl.__setitem__(1, WIDE * 16 + 1), api.ERR_SEQ_TOO_LONG)):
        bt, sl = b.bt.clone(), b.sl.clone()
        b.status.zero_()
        change()
        out = b.run()
        assert b.status.item() == bit and not out[4:8].any()
        out[4:8] = good[4:8]
        assert torch.equal(out, good)
        b.bt, b.sl = bt, sl


def test_chain_is_a_mask():
    """The same bits with the chain's words as without."""
    a, b = Batch([300, 70], [7, 20], 16), Batch([300, 70], [7, 20], 16, masks=chain(7) + chain(20))
    assert torch.equal(a.run(), b.run())


def test_bits_behind_the_tree_are_ignored():
    masks = [m | (1 << 64) - (1 << 7) for m in chain(7)]
    a, b = Batch([300], [7], 16), Batch([300], [7], 16, masks=masks)
    assert torch.equal(a.run(), b.run())


@pytest.mark.parametrize("length", [3, 200])
def test_rows_that_see_little(length):
    """Masks without the token itself, without anything, and with one token."""
    b = Batch([length], [3], 16, masks=[0, 4, 1])
    out = b.run()
    b.check(out)
    if length == 3:
        assert not out[0].any()


def test_first_tiles_unseen():
    """A row of a long tree whose only visible token is the last."""
    b = Batch([64], [64], 4, masks=[0] * 63 + [1 << 63])
    out = b.run()
    b.check(out)
    assert not out[:63].any() and out[63].any()


@pytest.mark.parametrize("q_scale", [1e-20, 0.01, 8.0, 50.0, 1e4])
def test_sharp_and_flat(q_scale):
    """Uniform weights at the one end, a single key at the other."""
    b = Batch([700, 40], [2, 3], 16, q_scale=q_scale, seed=7)
    b.check(b.run())


def test_growing_logits():
    """Every tile of keys has larger logits than the last, so every reference is raised again and again."""
    b = Batch([1500], [2], 16, seed=9)
    ramp = torch.linspace(0.0, 6.0, 1504)
    codes = b.cache[b.bt[0].long()].flatten(0, 1)
    codes[:, 512:] = 0
    codes[:, 512] = ramp.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    b.cache[b.bt[0].long()] = codes.view(-1, 16, 576)
    b.q[..., 512:] = 0
    b.q[..., 512] = 60.0
    b.check(b.run())
    b.q[..., 512] = -60.0                                # and falling ones
    b.check(b.run())


def test_one_large_weight_and_many_small():
    """One key with most of the weight and 30000 with 2^-19 of it each: together 5%, all equal, and each below
    the smallest step of a weight's terms.  The steps' dither keeps their sum: of 128 equal weights in a tile
    2^-19 * 2^7 = 2^-12 = 2^-3 steps, 16 round to one step and 112 to none."""
    n = 30000
    b = Batch([n], [1], 16, seed=11)
    codes = torch.zeros(b.pages * 16, 576, dtype=torch.uint8)
    one = int(torch.tensor([1.0]).to(torch.float8_e4m3fn).view(torch.uint8))
    codes[:, 0] = one                                    # the small ones' value
    order = b.bt[0].cpu().long()
    first = int(order[n // 2 // 16]) * 16 + n // 2 % 16
    codes[first] = 0
    codes[first, 1] = one
    codes[first, 512] = one
    b.cache = codes.view(-1, 16, 576).cuda()
    b.q.zero_()
    gap = 19.0 * np.log(2.0)
    b.q[..., 512] = gap / (b.scale * b.descale)
    got = f64(b.run())
    want = b.want()[0]
    small = want[0, 0, 0]
    assert 0.04 < small < 0.05
    # q's bf16 rounding is in both; the small weights' sum to 2% of itself
    assert np.abs(got[..., 0] - want[..., 0]).max() < 0.02 * small + 2.0 ** -8 * small
    assert np.abs(got[..., 1] - want[..., 1]).max() < 2.0 ** -8


@pytest.mark.parametrize("heads,nodes,lens", [(16, 4, [5000]), (16, 1, [20000, 300]), (128, 1, [9000]), (64, 3, [3000, 9000, 1]),
                                              (1, 1, [40000]), (40, 64, [2500])])
def test_every_key_counts_once(heads, nodes, lens):
    """Equal weights, and runs of keys with an output dim each: a key left out or counted twice shows.
    Weights are powers of two and exact, sums exact in float32, so only the output's rounding is left (and
    the division)."""
    b = Batch(lens, [min(nodes, n) for n in lens], heads, seed=3)
    b.q[..., 512:] = 0
    b.cache[..., 512:] = 0
    b.q[..., :512] = 0
    one = int(torch.tensor([1.0]).to(torch.float8_e4m3fn).view(torch.uint8))
    codes = torch.zeros(b.pages * 16, 576, dtype=torch.uint8)
    for s, n in enumerate(lens):
        at = torch.arange(n)
        rows = b.bt[s].cpu().long()[at // 16] * 16 + at % 16
        codes[rows, (at * 512 // n)] = one
    b.cache = codes.view(-1, 16, 576).cuda()
    got = f64(b.run())
    for s, n in enumerate(lens):
        run = np.arange(n) * 512 // n
        for i in range(b.nodes[s]):
            seen = n - b.nodes[s] + i + 1
            want = np.bincount(run[:seen], minlength=512) / seen * b.descale
            assert np.all(np.abs(got[b.cu_list[s] + i] - want) <= want * (2.0 ** -8 + 2.0 ** -20))


def test_unseen_codes_do_not_matter():
    """NaN codes behind a sequence, in pages of others, and in tokens of a tree that a row does not see."""
    masks = [0b0001, 0b0011, 0b0101, 0b1001]
    b = Batch([70, 200], [4, 4], 16, masks=masks * 2)
    clean = b.run()
    b.check(clean)
    used = torch.zeros(b.pages, 16, dtype=torch.bool)
    for s, n in enumerate(b.lens):
        at = torch.arange(n)
        used[b.bt[s].cpu().long()[at // 16], at % 16] = True
    b.cache[~used.cuda()] = 0x7f
    assert torch.equal(b.run(), clean)
    for s, n in enumerate(b.lens):                       # the last token of each tree: only itself sees it
        at = n - 1
        b.cache[b.bt[s, at // 16].long(), at % 16] = 0xff
    out = b.run()
    for t in range(8):
        assert torch.isnan(out[t]).all() if t % 4 == 3 else torch.equal(out[t], clean[t])


@pytest.mark.parametrize("dim", [0, 300, 511, 512, 575])
def test_a_nan_that_is_seen(dim):
    """A NaN code anywhere in a visible token: every output of the rows that see it."""
    b = Batch([1000, 300], [2, 2], 16)
    clean = b.run()
    b.cache[b.bt[0, 20].long(), 3, dim] = 0x7f
    out = b.run()
    assert torch.isnan(out[:2]).all() and torch.equal(out[2:], clean[2:])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim", [5, 570])
def test_rows_of_q_that_are_not_finite(bad, dim):
    b = Batch([400, 300], [2, 2], 16)
    clean = b.run()
    b.q[1, 3, dim] = bad
    out = b.run()
    assert torch.isnan(out[1, 3]).all()
    out[1, 3] = clean[1, 3]
    assert torch.equal(out, clean)


def test_extremes_of_q():
    """Rows of zeros, of bf16's largest and smallest, and one large element among small ones."""
    b = Batch([200], [4], 4, seed=2)
    b.q[0] = 0
    b.q[1] *= 1e-38
    b.q[2, :, 100:] *= 2.0 ** -12
    b.q[3] *= 2.0 ** 20
    b.check(b.run())


def test_errors():
    """A bad page, no tokens, too many tokens, too long, longer than the table: zeros, and the others right."""
    b = Batch([300, 300, 40, 40, 40, 70], [2, 2, 2, 2, 2, 2], 16, behind=1)
    good = b.run()
    b.check(good)
    for name, change, bit in (("page", lambda: b.bt.__setitem__((1, 3), b.pages), api.ERR_PAGE),
                              ("page", lambda: b.bt.__setitem__((1, 3), -1), api.ERR_PAGE),
                              ("short", lambda: b.sl.__setitem__(1, 1), api.ERR_QLEN_GT_SEQ),
                              ("negative", lambda: b.sl.__setitem__(1, -5), api.ERR_QLEN_GT_SEQ),
                              ("long", lambda: b.sl.__setitem__(1, b.bt.shape[1] * 16 + 1), api.ERR_SEQ_TOO_LONG),
                              ("longest", lambda: b.sl.__setitem__(1, 2 ** 31 - 1), api.ERR_SEQ_TOO_LONG)):
        bt, sl = b.bt.clone(), b.sl.clone()
        b.status.zero_()
        change()
        out = b.run()
        assert b.status.item() == bit, name
        assert not out[2:4].any(), name
        out[2:4] = good[2:4]
        assert torch.equal(out, good), name
        b.bt, b.sl = bt, sl


def test_boundaries():
    """A sequence with no new token or more than 64, and boundaries that do not ascend."""
    b = Batch([300, 200, 100], [2, 2, 2], 16)
    good = b.run()
    b.cu.copy_(torch.tensor([0, 4, 4, 6]))
    out = b.run()
    assert b.status.item() == api.ERR_QLEN and torch.equal(out[4:], good[4:])
    wide = Batch([300, 200], [64, 2], 4)
    ref = wide.run()
    wide2 = Batch([300, 200], [64, 2], 4)
    wide2.cu.copy_(torch.tensor([0, 65, 66]))
    out = wide2.run()
    assert wide2.status.item() == api.ERR_QLEN and not out[:65].any()
    for cu in ([0, 66, 64], [0, 64, 99], [-1, 64, 66], [70, 64, 66]):
        wide2.cu.copy_(torch.tensor(cu))
        wide2.run()
        assert wide2.status.item() & api.ERR_QLEN
    wide2.cu.copy_(torch.tensor([0, 64, 66]))
    assert torch.equal(wide2.run(), ref)


@pytest.mark.parametrize("lens", [[9000] * 3 + [9100], [300, 20000, 700, 5000], [4000] * 8, [20000, 1, 20000]])
@pytest.mark.parametrize("heads,nodes", [(128, 1), (128, 2), (64, 3)])
def test_row_tiles_together(lens, heads, nodes):
    """Two, four and three row tiles in every sequence, whose pieces several CTAs take together, with one
    sequence that cannot be computed among them."""
    lens = [max(n, nodes) for n in lens]
    b = Batch(lens, [nodes] * len(lens), heads, seed=heads + nodes)
    out = b.run()
    assert b.status.item() == 0
    short = [i for i, n in enumerate(lens) if n < 1000]
    want = Batch([lens[i] for i in short], [nodes] * len(short), heads) if short else None
    if want:                                             # (the long ones: rows against the same row computed alone)
        want.q = torch.cat([b.q[b.cu_list[i]:b.cu_list[i + 1]] for i in short])
        want.cache, want.bt = b.cache, b.bt[short].contiguous()
        want.check(torch.cat([out[b.cu_list[i]:b.cu_list[i + 1]] for i in short]))
    one = Batch([lens[-1]], [nodes], heads)
    one.q, one.cache, one.bt = b.q[-nodes:], b.cache, b.bt[-1:].contiguous()
    alone = f64(one.run())
    # both are within the output's rounding, and each other's, of the same sums
    assert np.abs(f64(out[-nodes:]) - alone).max() <= 2.0 ** -6 * np.abs(alone).max()
    b.bt[1, 0] = -1
    bad = b.run()
    assert b.status.item() == api.ERR_PAGE and not bad[nodes:2 * nodes].any()
    bad[nodes:2 * nodes] = out[nodes:2 * nodes]
    assert torch.equal(bad, out)


def test_many_units():
    """More row tiles than SMs, of one to three tokens over short contexts."""
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(3, 60, 400)]
    b = Batch(lens, [int(x) for x in rng.integers(1, 4, 400)], 16, seed=1)
    b.check(b.run())


@pytest.mark.parametrize("count,heads,nodes,width", [(33, 16, 1, 0), (160, 16, 2, 0), (1000, 2, 1, 0), (1024, 20, 2, WIDE // 100),
                                                     (1500, 3, 3, 0), (5000, 1, 1, 0)])
def test_many_sequences(count, heads, nodes, width):
    """The walk over batches of more than 32, 128 and 1024 sequences, some longer, one of which has no tokens."""
    rng = np.random.default_rng(count)
    lens = [int(x) for x in rng.integers(nodes, 40, count)]
    for i in (0, count // 2, count - 1):
        lens[i] = 600 + i % 100
    b = Batch(lens, [nodes] * count, heads, seed=count, width=width)
    good = b.run()
    assert b.status.item() == 0
    b.check(good)
    b.cu[10:count // 2 + 1] -= nodes                     # sequence 9 has none, and the long one twice as many
    b.cu_list = b.cu.tolist()
    b.nodes = [y - x for x, y in zip(b.cu_list, b.cu_list[1:])]
    assert b.nodes[9] == 0 and b.nodes[count // 2] == 2 * nodes
    out = b.run()
    assert b.status.item() == api.ERR_QLEN
    b.check(out)


def test_strides_and_outputs():
    b = Batch([300, 50], [3, 2], 5, pad=8)
    ref = b.run()
    b.check(ref)
    b.q = b.q.transpose(0, 1).contiguous().transpose(0, 1)
    store = torch.full((5, 5, 520), 9.0, dtype=torch.bfloat16, device="cuda")
    out = b.run(out=store[..., :512])
    assert torch.equal(out, ref) and (store[..., 512:] == 9.0).all()
    made = api.mtp_latent_attn_fwd(b.q, b.cache.view(torch.float8_e4m3fn), b.bt, b.sl, b.cu, torch.full((1,), 0.75, device="cuda"),
                                   b.scale)
    assert torch.equal(made, ref)


def test_repeats_streams_and_graphs():
    """The same bits again, on another stream with a workspace of garbage, and in graphs that follow their
    buffers; two graphs in turn on one workspace."""
    b = Batch([5000, 300, 9000], [4, 1, 2], 16, seed=4)
    ref = b.run()
    need = api.mtp_latent_attn_workspace_size(3, b.total, 16, b.bt.shape[1])
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    other = torch.cuda.Stream()
    out = torch.zeros_like(ref)
    torch.cuda.synchronize()
    api.mtp_latent_attn_fwd(b.q, b.cache, b.bt, b.sl, b.cu, 0.75, b.scale, out=out, workspace=ws, stream=other)
    other.synchronize()
    assert torch.equal(out, ref)
    d = torch.full((1,), 0.75, device="cuda")
    small = Batch([40], [3], 16, seed=5)
    graphs, outs = [], []
    for x in (b, small):
        outs.append(torch.zeros(x.total, 16, 512, dtype=torch.bfloat16, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.mtp_latent_attn_fwd(x.q, x.cache, x.bt, x.sl, x.cu, d, x.scale, out=outs[-1], workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], small.run())
    b.sl -= torch.tensor([4000, 7, 8000], dtype=torch.int32, device="cuda")
    b.lens = b.sl.tolist()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], b.run())
    b.check(outs[0])


@pytest.mark.parametrize("heads,nodes", [(16, 1), (16, 2), (16, 4), (128, 1)])
def test_no_wait_runs_out(heads, nodes):
    """Pieces that begin and end anywhere: with ever other lengths, CTAs whose first segment is one tile, two,
    and so on, one after the other on a stream; every call ends by itself (a wait that ran out would tell)."""
    b = Batch([9000] * 16, [nodes] * 16, heads, seed=8)
    d = torch.full((1,), 0.75, device="cuda")
    out = torch.zeros(b.total, heads, 512, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(api.mtp_latent_attn_workspace_size(16, b.total, heads, b.bt.shape[1]), dtype=torch.uint8, device="cuda")
    for n in list(range(8200, 9000, 16)) + list(range(1000, 1800, 16)):
        b.sl.fill_(n)
        for _ in range(4):
            api.mtp_latent_attn_fwd(b.q, b.cache, b.bt, b.sl, b.cu, d, b.scale, out=out, workspace=ws, status=b.status)
    torch.cuda.synchronize()
    assert b.status.item() == 0


def test_one_workspace_for_all_batches():
    """The size grows with every argument, and batches of all kinds run in the largest one's."""
    most = (40, 160, 128, 600)
    need = api.mtp_latent_attn_workspace_size(*most)
    for i, values in enumerate(((1, 2, 3, 39, 40), (40, 41, 99, 160), (1, 5, 16, 17, 127, 128), (1, 8, 9, 100, 600))):
        sizes = [api.mtp_latent_attn_workspace_size(*most[:i], v, *most[i + 1:]) for v in values]
        assert sizes == sorted(sizes) and 0 < sizes[0] and sizes[-1] == need
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for lens, nodes, heads in (([9000], [4], 16), ([300] * 40, [4] * 40, 128), ([9000, 5], [1, 1], 5), ([300] * 40, [1] * 40, 16), ([1], [1], 1)):
        b = Batch(lens, nodes, heads, seed=40 + heads)
        assert torch.equal(b.run(workspace=ws), b.run())


@pytest.mark.parametrize("width", [8, 9, 31, 32, 33, 40])
@pytest.mark.parametrize("heads,nodes", [(16, 1), (16, 4), (128, 1), (4, 30)])
def test_short_tables(width, heads, nodes):
    """Tables of up to 32 pages, whose units are never cut, and a little longer ones; more units than SMs."""
    lens = [max(nodes, n) for n in (width * 16, 1, 127, 129, width * 16 - 15) + (60,) * 30]
    lens = [min(n, width * 16) for n in lens]
    b = Batch(lens, [nodes] * len(lens), heads, seed=width + heads, width=width)
    out = b.run()
    assert b.status.item() == 0
    b.check(out)


def test_two_streams():
    """Two calls at once, each with its own workspace, in turn many times."""
    a, b = Batch([9000, 300], [4, 1], 16, seed=20), Batch([2000, 5000, 70], [1, 1, 1], 128, seed=21)
    refs = [a.run(), b.run()]
    d = torch.full((1,), 0.75, device="cuda")
    sets = []
    for x in (a, b):
        need = api.mtp_latent_attn_workspace_size(len(x.lens), x.total, x.heads, x.bt.shape[1])
        sets.append((x, torch.zeros(need, dtype=torch.uint8, device="cuda"), torch.cuda.Stream(),
                     [torch.zeros(x.total, x.heads, 512, dtype=torch.bfloat16, device="cuda") for _ in range(10)]))
    torch.cuda.synchronize()
    for i in range(10):
        for x, ws, stream, outs in sets:
            api.mtp_latent_attn_fwd(x.q, x.cache, x.bt, x.sl, x.cu, d, x.scale, out=outs[i], workspace=ws, status=x.status, stream=stream)
    torch.cuda.synchronize()
    for (x, _, _, outs), ref in zip(sets, refs):
        assert x.status.item() == 0 and all(torch.equal(o, ref) for o in outs)


@pytest.mark.parametrize("lens,nodes,heads", [([9000, 300], [4, 1], 16), ([700] * 5, [3] * 5, 100), ([40] * 300, [1] * 300, 5),
                                              ([20000, 20000], [1, 1], 128), ([1], [1], 1)])
def test_nothing_else_is_written(lens, nodes, heads):
    """The bytes around a workspace of exactly the size that is asked for, and around the output."""
    b = Batch(lens, nodes, heads, seed=30)
    need = api.mtp_latent_attn_workspace_size(len(lens), b.total, heads, b.bt.shape[1])
    room = torch.full((need + 2048,), 0xAB, dtype=torch.uint8, device="cuda")
    store = torch.full((b.total + 2, heads, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    b.run(out=store[1:-1], workspace=room[1024:1024 + need])
    assert b.status.item() == 0 and torch.equal(store[1:-1], b.run())
    assert (room[:1024] == 0xAB).all() and (room[1024 + need:] == 0xAB).all()
    assert (store[0] == 9.0).all() and (store[-1] == 9.0).all()


def test_trees_in_a_graph():
    """A captured call with a tree mask follows the mask's, the lengths' and the tables' buffers."""
    masks = tree(20, 1) + tree(7, 2)
    b = Batch([700, 300], [20, 7], 16, seed=31, masks=masks)
    d = torch.full((1,), 0.75, device="cuda")
    ws = torch.zeros(api.mtp_latent_attn_workspace_size(2, b.total, 16, b.bt.shape[1]), dtype=torch.uint8, device="cuda")
    out = torch.zeros(b.total, 16, 512, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.mtp_latent_attn_fwd(b.q, b.cache, b.bt, b.sl, b.cu, d, b.scale, tree_mask=b.mask, out=out, workspace=ws, status=b.status)
    g.replay()
    torch.cuda.synchronize()
    b.check(out)
    b.masks = tree(20, 3) + chain(7)
    b.mask.copy_(torch.tensor(b.masks, dtype=torch.int64))
    b.bt[:, :18] = b.bt[:, :18].flip(1)
    b.sl.copy_(torch.tensor([290, 288], dtype=torch.int32))
    b.lens = [290, 288]
    g.replay()
    torch.cuda.synchronize()
    b.check(out)
    assert b.status.item() == 0


def test_a_far_page():
    """A page beyond 2^31 bytes of the cache."""
    pages = (1 << 31) // (16 * 576) + 100
    b = Batch([300], [2], 16)
    ref = b.run()
    big = torch.zeros(pages, 16, 576, dtype=torch.uint8, device="cuda")
    far = torch.arange(pages - b.bt.shape[1], pages, device="cuda", dtype=torch.int32)[None]
    big[far[0].long()] = b.cache[b.bt[0].long()]
    b.cache, b.bt = big, far.contiguous()
    assert torch.equal(b.run(), ref)


def test_appended_and_read():
    """A step as a decode loop has it: new tokens appended, then attention over the cache, twice, against
    the definition over what the cache holds and over the tokens themselves."""
    heads, inv = 8, rope.inv_freq(64)[0]
    freqs = api.mtp_rope_freqs(inv, device="cuda")
    g = torch.Generator("cuda").manual_seed(6)
    b = Batch([120, 45], [100, 30], heads, seed=6)
    b.descale = 0.02
    before = b.cache.clone()
    for step in range(2):
        nodes = [4, 2] if step else [64, 30]
        lens = [124, 47] if step else [120, 45]
        cu = [0, nodes[0], sum(nodes)]
        total = cu[-1]
        b.sl, b.cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, cu))
        b.lens, b.nodes, b.cu_list, b.total = lens, nodes, cu, total
        x = torch.randn(total, 576, generator=g, device="cuda").bfloat16()
        b.q = torch.randn(total, heads, 576, generator=g, device="cuda").bfloat16()
        raw = b.q[..., 512:].clone()
        pos = torch.tensor([lens[s] - nodes[s] + i for s in range(2) for i in range(nodes[s])], dtype=torch.int32, device="cuda")
        api.mtp_rope_latent_append(raw, x[:, :512], x[:, 512:], pos, freqs, b.cache, b.bt, b.sl, b.cu, 0.02, 1.0, True,
                                   q_out=b.q[..., 512:], status=b.status)
        out = b.run()
        assert b.status.item() == 0
        b.check(out)
        from oracle import rope as oracle_rope
        turned = oracle_rope.rotate(f64(raw), pos.cpu().numpy(), inv, 1.0, True)
        assert np.all(np.abs(f64(b.q[..., 512:]) - turned) <= np.abs(turned) * 2.0 ** -8 + 2.0 ** -17)
    assert not torch.equal(before, b.cache)


def test_workspace_refusals():
    b = Batch([300], [2], 16)
    need = api.mtp_latent_attn_workspace_size(1, 2, 16, b.bt.shape[1])
    assert need > 0
    for ws in (torch.zeros(need - 1, dtype=torch.uint8, device="cuda"), torch.zeros(need + 16, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(api.MtpAttnError) as e:
            b.run(workspace=ws)
        assert e.value.code == api.E_WORKSPACE
    assert api.mtp_latent_attn_workspace_size(1, 2, 129, 4) == 0
