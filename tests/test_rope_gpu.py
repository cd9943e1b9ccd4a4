"""Rotary positions, appending and the prefill operands on the GPU against the float64 definitions.

Tolerances, from the arithmetic: a rotated value is two float32 products and a sum with sines and cosines
that are off by at most 2^-21 (an angle rounded to 2^-24 half turns, sincospif's 2 units): 2^-20 of
mscale * (|a| + |b|) in all.  A code is off by half a step of its own beyond that, bf16 by 2^-8
of the value (half of its eps).  The product with 1 / descale adds 2^-23 of the value.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import rope as oracle
from paged_fp8_speculative_gb300 import api, rope

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def values(codes):
    return codes.view(torch.float8_e4m3fn).double().cpu().numpy()


def reach(x, pairs, mscale, interleaved):
    """mscale * (|a| + |b|) of every element's pair, the element's own size where nothing is rotated."""
    out = np.abs(x).astype(np.float64)
    if pairs:
        a = np.abs(x[..., :2 * pairs])
        both = (a.reshape(a.shape[:-1] + (pairs, 2)).sum(-1) if interleaved else a[..., :pairs] + a[..., pairs:])
        out[..., :2 * pairs] = mscale * (np.repeat(both, 2, -1) if interleaved else np.concatenate([both, both], -1))
    return out


def check_bf16(got, want, scale):
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + scale * 2.0 ** -20)


def check_codes(got, want, scale, descale):
    """want: before the rounding, in the codes' units."""
    y = oracle.clipped(want, descale)
    slack = scale / descale * 2.0 ** -20 + np.abs(y) * 2.0 ** -23
    assert np.all(np.abs(got - y) <= oracle.half_step(np.abs(y) + slack) + slack)


class Batch:
    """Tokens of a batch with shuffled pages, the output's memory marked."""

    def __init__(self, lens, nodes, hq, hkv, pairs, dtype="bf16", seed=0, behind=0, base=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.nodes = lens, nodes
        per = [-(-n // 16) for n in lens]
        self.pages = sum(per) + 2
        order = torch.randperm(self.pages, generator=torch.Generator().manual_seed(seed))
        self.bt = torch.full((len(lens), max(per + [1]) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            self.bt[b, :n] = order[at:at + n]
            at += n
        cu = [base]
        for n in nodes:
            cu.append(cu[-1] + n)
        self.total = cu[-1] + behind
        self.hq, self.hkv, self.pairs = hq, hkv, pairs
        joint = torch.randn(self.total, hq + 2 * hkv, 256, generator=g, device="cuda").to(DTYPES[dtype])
        self.q, self.k, self.v = joint[:, :hq], joint[:, hq:hq + hkv], joint[:, hq + hkv:]
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.table = self.bt.cuda()
        self.pos = torch.randint(0, 200000, (self.total,), generator=g, device="cuda", dtype=torch.int32)
        self.inv, _ = rope.inv_freq(2 * pairs) if pairs else ([], 1.0)
        self.freqs = api.mtp_rope_freqs(self.inv, device="cuda") if pairs else None
        shape = (self.pages, 16, hkv, 256)
        self.kc = torch.full(shape, 0x55, dtype=torch.uint8, device="cuda")
        self.vc = torch.full(shape, 0x56, dtype=torch.uint8, device="cuda")
        self.out = torch.full((self.total, hq, 256), 9.0, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, kd=0.02, vd=0.03, mscale=1.0, interleaved=False, **kw):
        api.mtp_rope_append(self.q, self.k, self.v, self.pos, self.freqs, self.kc, self.vc, self.table, self.sl,
                            self.cu, kd, vd, mscale, interleaved, **{"q_out": self.out, "status": self.status, **kw})
        torch.cuda.synchronize()

    def check(self, kd=0.02, vd=0.03, mscale=1.0, interleaved=False, skip=()):
        """Every owned row right but those of the sequences in skip; nothing else written."""
        place = oracle.places(self.bt.numpy(), self.lens, self.cu.cpu().numpy(), self.total)
        cu = self.cu.tolist()
        lost = {t for b in skip for t in range(cu[b], cu[b + 1])}
        mine = [t for t in range(self.total) if place[t] is not None]
        q, k, v = f64(self.q), f64(self.k), f64(self.v)
        pos = self.pos.cpu().numpy()
        want_q = oracle.rotate(q, pos, self.inv, mscale, interleaved)
        want_k = oracle.rotate(k, pos, self.inv, mscale, interleaved)
        got = f64(self.out)
        check_bf16(got[mine], want_q[mine], reach(q, self.pairs, mscale, interleaved)[mine])
        assert np.all(got[[t for t in range(self.total) if place[t] is None]] == 9.0)
        marks_k, marks_v = np.full(self.kc.shape[:2], True), np.full(self.kc.shape[:2], True)
        kv, vv = values(self.kc), values(self.vc)
        for t in mine:
            if t in lost:
                continue
            check_codes(kv[place[t]], want_k[t], reach(k[t], self.pairs, mscale, interleaved), kd)
            check_codes(vv[place[t]], v[t], np.abs(v[t]), vd)
            marks_k[place[t]] = marks_v[place[t]] = False
        assert np.all(self.kc.cpu().numpy()[marks_k] == 0x55) and np.all(self.vc.cpu().numpy()[marks_v] == 0x56)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("pairs,hq,hkv", [(128, 16, 1), (32, 6, 2), (8, 1, 1), (0, 3, 3), (40, 5, 1), (112, 2, 2)])
def test_append(interleaved, dtype, pairs, hq, hkv):
    b = Batch([300, 17, 1, 64, 40], [4, 17, 1, 3, 0], hq, hkv, pairs, dtype, behind=2)
    b.run(mscale=1.25, interleaved=interleaved)
    assert b.status.item() == 0
    b.check(mscale=1.25, interleaved=interleaved)


@pytest.mark.parametrize("nodes", [[1], [1, 0, 0, 1], [0, 0, 5, 0], [33] * 40, [1] * 1100, [0] * 50 + [7] + [0] * 60 + [9]])
def test_append_many_sequences(nodes):
    lens = [n + 7 * (i % 5) for i, n in enumerate(nodes)]
    b = Batch(lens, nodes, 2, 1, 16, behind=3, base=2, seed=len(nodes))
    b.run()
    assert b.status.item() == 0
    b.check()


def test_append_a_long_prompt():
    b = Batch([3001, 1500], [3001, 700], 4, 2, 64, seed=5)
    b.run(interleaved=True)
    b.check(interleaved=True)


def test_append_in_place_and_without_q():
    b = Batch([50, 20], [9, 20], 4, 2, 128)
    before = b.q.clone()
    plain = Batch([50, 20], [9, 20], 4, 2, 128)
    plain.run()
    out = api.mtp_rope_append(b.q, b.k, b.v, b.pos, b.freqs, b.kc, b.vc, b.table, b.sl, b.cu, 0.02, 0.03, q_out=b.q)
    assert out.data_ptr() == b.q.data_ptr() and torch.equal(b.q, plain.out) and torch.equal(b.kc, plain.kc)
    assert not torch.equal(b.q, before)
    b.kc.fill_(0x55)
    assert api.mtp_rope_append(None, b.k, b.v, b.pos, b.freqs, b.kc, b.vc, b.table, b.sl, b.cu, 0.02, 0.03) is None
    assert torch.equal(b.kc, plain.kc) and torch.equal(b.vc, plain.vc)


def test_append_makes_its_output():
    b = Batch([50, 20], [9, 20], 4, 2, 128)
    b.run()
    kd, vd = torch.full((1,), 0.02, device="cuda"), torch.full((1,), 0.03, device="cuda")
    out = api.mtp_rope_append(b.q, b.k, b.v, b.pos, b.freqs, b.kc, b.vc, b.table, b.sl, b.cu, kd, vd)
    assert out.is_contiguous() and torch.equal(out, b.out)


def test_append_extreme_values():
    """Beyond the largest code both ways, infinities, NaN, subnormal codes and zeros."""
    b = Batch([40], [40], 1, 1, 0)
    special = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1e-30, 448 * 0.5, 464 * 0.5,
                            2.0 ** -10, 2.0 ** -11, 3 * 2.0 ** -11, -17 * 0.5], device="cuda")
    b.k[:, :, :14] = special.to(b.k.dtype)
    b.run(kd=0.5)
    got = values(b.kc[b.bt[0, 0], 0, 0])[:14]
    want = [448, -448, 448, -448, np.nan, 0, 0, 0, 448, 448, 2.0 ** -9, 2.0 ** -9 * 0, 2.0 ** -9 * 2, -16]
    # 2^-10 / 0.5 is one step of the subnormal codes, 2^-11 / 0.5 half of one (to even: 0), 3 * 2^-10 one and
    # a half (to even: 2); -17 lies between -16 and -18
    assert np.array_equal(got, np.array(want), equal_nan=True)


def test_append_far_and_negative_positions():
    b = Batch([16], [16], 2, 1, 128, "f32")
    b.pos[:] = torch.tensor([0, 1, -1, 2 ** 20, 10 ** 7, 2 ** 31 - 1, -2 ** 31, 12345678] * 2, dtype=torch.int32)
    b.run(interleaved=True)
    b.check(interleaved=True)


def test_append_errors():
    """A sequence shorter than its tokens, one longer than its table, a page outside the pool."""
    b = Batch([20, 20, 20, 20, 20], [5, 5, 5, 5, 5], 2, 1, 16)
    b.sl[1] = 4
    b.sl[2] = b.table.shape[1] * 16 + 1
    b.table[3, 0] = b.pages
    b.run()
    assert b.status.item() == api.ERR_QLEN_GT_SEQ | api.ERR_SEQ_TOO_LONG | api.ERR_PAGE
    # of sequence 3 the last four tokens are on its second page
    place = oracle.places(b.bt.numpy(), b.lens, b.cu.cpu().numpy(), b.total)
    kc = b.kc.clone()
    for t in (16, 17, 18, 19):
        assert not (b.kc[place[t]] == 0x55).all()
        kc[place[t]], b.vc[place[t]] = 0x55, 0x56
    b.kc = kc
    b.check(skip=(1, 2, 3))


def test_append_bad_page_numbers_write_nothing():
    b = Batch([20], [5], 2, 1, 16)
    for bad in (-1, -2 ** 31, 2 ** 31 - 1, b.pages):
        b.table[:] = bad
        b.run()
        assert (b.kc == 0x55).all() and (b.vc == 0x56).all() and b.status.item() == api.ERR_PAGE


def test_append_boundaries_out_of_order():
    """Nothing is written out of bounds, known rows are right or left alone, and the status tells."""
    b = Batch([20, 20, 20], [5, 5, 5], 2, 1, 16)
    good = b.cu.clone()
    for cu in ([0, 10, 5, 15], [0, 5, 10, 99], [-3, 5, 10, 15], [7, 5, 10, 15], [0, -9, 99, 15]):
        b.cu.copy_(torch.tensor(cu))
        b.run()
    b.cu.copy_(good)
    assert b.status.item() & api.ERR_QLEN
    b.run()
    b.kc.fill_(0x55), b.vc.fill_(0x56)
    b.run()
    b.check()


def test_append_strides():
    """Tokens and heads in the other order, and rows of a wider buffer."""
    b = Batch([60], [33], 4, 2, 64)
    b.q = b.q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.zeros(33, 3, 264, dtype=torch.bfloat16, device="cuda")
    wide[:, :2, :256] = b.k
    b.k = wide[:, :2, :256]
    store = torch.full((33, 4, 264), 9.0, dtype=torch.bfloat16, device="cuda")
    b.out = store[..., :256]
    b.run()
    b.check()
    assert (store[..., 256:] == 9.0).all()


def test_append_single_token_strides():
    """One token, one head: axes whose strides mean nothing."""
    b = Batch([1], [1], 1, 1, 64)
    for t in ("q", "k", "v"):
        x = getattr(b, t)
        setattr(b, t, torch.as_strided(x.contiguous(), (1, 1, 256), (1, 1, 1)))
    b.run()
    b.check()


def test_append_on_a_stream_and_in_a_graph():
    b = Batch([100, 30], [26, 7], 4, 2, 128)
    other = torch.cuda.Stream()
    b.run()
    ref_out, ref_k = b.out.clone(), b.kc.clone()
    b.out.fill_(9.0), b.kc.fill_(0x55)
    torch.cuda.synchronize()
    api.mtp_rope_append(b.q, b.k, b.v, b.pos, b.freqs, b.kc, b.vc, b.table, b.sl, b.cu, 0.02, 0.03, q_out=b.out, stream=other)
    other.synchronize()
    assert torch.equal(b.out, ref_out) and torch.equal(b.kc, ref_k)
    kd, vd = torch.full((1,), 0.02, device="cuda"), torch.full((1,), 0.03, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.mtp_rope_append(b.q, b.k, b.v, b.pos, b.freqs, b.kc, b.vc, b.table, b.sl, b.cu, kd, vd, q_out=b.out)
    for shift in (0, 3):                                 # lengths and positions are read anew
        b.kc.fill_(0x55), b.vc.fill_(0x56), b.out.fill_(9.0)
        b.sl -= shift
        b.lens = b.sl.tolist()
        b.pos += shift
        graph.replay()
        torch.cuda.synchronize()
        b.check()


# ---- the latent cache ------------------------------------------------------------------------------


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("heads", [0, 1, 16, 128])
def test_latent_append(interleaved, dtype, heads):
    lens, nodes = [300, 17, 1, 64, 40], [4, 17, 1, 3, 0]
    b = Batch(lens, nodes, 1, 1, 32, dtype, behind=2, base=1)
    g = torch.Generator("cuda").manual_seed(3)
    both = torch.randn(b.total, 576, generator=g, device="cuda").to(DTYPES[dtype])
    q = torch.randn(b.total, max(heads, 1), 192, generator=g, device="cuda").to(DTYPES[dtype])[..., 128:]
    cache = torch.full((b.pages, 16, 576), 0x55, dtype=torch.uint8, device="cuda")
    rows = torch.full((b.total, max(heads, 1), 576), 9.0, dtype=torch.bfloat16, device="cuda")
    out = api.mtp_rope_latent_append(q if heads else None, both[:, :512], both[:, 512:], b.pos, b.freqs, cache, b.table, b.sl,
                                     b.cu, 0.02, 0.75, interleaved, q_out=rows[..., 512:] if heads else None,
                                     status=b.status)
    torch.cuda.synchronize()
    assert b.status.item() == 0 and (out is None) == (heads == 0)
    place = oracle.places(b.bt.numpy(), lens, b.cu.cpu().numpy(), b.total)
    mine = [t for t in range(b.total) if place[t] is not None]
    pos, x = b.pos.cpu().numpy(), f64(both)
    part = oracle.rotate(x[:, None, 512:], pos, b.inv, 0.75, interleaved)[:, 0]
    want = np.concatenate([x[:, :512], part], -1)
    scale = np.concatenate([np.abs(x[:, :512]), reach(x[:, 512:], 32, 0.75, interleaved)], -1)
    got, left = values(cache), np.full(cache.shape[:2], True)
    for t in mine:
        check_codes(got[place[t]], want[t], scale[t], 0.02)
        left[place[t]] = False
    assert np.all(cache.cpu().numpy()[left] == 0x55)
    assert (rows[..., :512] == 9.0).all()
    if heads:
        y = f64(rows[..., 512:])
        check_bf16(y[mine], oracle.rotate(f64(q), pos, b.inv, 0.75, interleaved)[mine],
                   reach(f64(q), 32, 0.75, interleaved)[mine])
        assert np.all(y[[t for t in range(b.total) if place[t] is None]] == 9.0)


def test_latent_append_errors_and_in_place():
    b = Batch([20, 20], [5, 5], 1, 1, 32)
    x = torch.randn(b.total, 576, device="cuda").bfloat16()
    cache = torch.full((b.pages, 16, 576), 0x55, dtype=torch.uint8, device="cuda")
    q = torch.randn(b.total, 3, 64, device="cuda").bfloat16()
    want = api.mtp_rope_latent_append(q, x[:, :512], x[:, 512:], b.pos, b.freqs, cache, b.table, b.sl, b.cu, 0.02)
    good = cache.clone()
    b.table[1, 1] = -1
    cache.fill_(0x55)
    assert api.mtp_rope_latent_append(q, x[:, :512], x[:, 512:], b.pos, b.freqs, cache, b.table, b.sl, b.cu, 0.02, q_out=q,
                                      status=b.status).data_ptr() == q.data_ptr()
    assert b.status.item() == api.ERR_PAGE and torch.equal(q, want)
    good[b.bt[1, 1], :4] = 0x55
    assert torch.equal(cache, good)


# ---- the prefill's operands ------------------------------------------------------------------------


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,hq,hkv", [(1, 1, 1), (5, 6, 2), (300, 16, 16), (1000, 3, 1)])
def test_prefill(interleaved, dtype, tokens, hq, hkv):
    g = torch.Generator("cuda").manual_seed(tokens)
    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(DTYPES[dtype])
    q, kv, kr = normal(tokens, hq, 192), normal(tokens, hkv, 256), normal(tokens, 576)[:, 512:]
    pos = torch.randint(-5, 200000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    inv, m = rope.inv_freq(64, scaling="parts", factor=40.0)
    freqs = api.mtp_rope_freqs(inv, device="cuda")
    q8, k8, v8 = api.mtp_rope_prefill(q, kv[..., :128], kr, kv[..., 128:], pos, freqs, 0.03, 0.0171, 0.02, m, interleaved)
    torch.cuda.synchronize()
    p = pos.cpu().numpy()
    def turned(x):
        return oracle.rotate(x, p, inv, m, interleaved), reach(x, 32, m, interleaved)
    qw, ks = f64(q), f64(kv)
    a, ra = turned(qw[..., 128:])
    check_codes(values(q8), np.concatenate([qw[..., :128], a], -1), np.concatenate([np.abs(qw[..., :128]), ra], -1), 0.03)
    a, ra = (np.repeat(x, hkv, 1) for x in turned(f64(kr)[:, None]))
    check_codes(values(k8), np.concatenate([ks[..., :128], a], -1), np.concatenate([np.abs(ks[..., :128]), ra], -1), 0.0171)
    check_codes(values(v8), ks[..., 128:], np.abs(ks[..., 128:]), 0.02)
    given = [torch.empty_like(t).view(torch.uint8) for t in (q8, k8, v8)]
    api.mtp_rope_prefill(q, kv[..., :128], kr, kv[..., 128:], pos, freqs, 0.03, 0.0171, 0.02, m, interleaved, *given)
    assert all(torch.equal(x, y.view(torch.uint8)) for x, y in zip(given, (q8, k8, v8)))


def test_prefill_feeds_the_attention():
    """The operands as fmha_fwd_fp8_varlen reads them, against attention in float64 over the codes' values."""
    g = torch.Generator("cuda").manual_seed(1)
    t, h = 200, 4
    q, kv, kr = (torch.randn(t, *s, generator=g, device="cuda").bfloat16() for s in ((h, 192), (h, 256), (64,)))
    pos = torch.arange(t, device="cuda", dtype=torch.int32)
    inv, m = rope.inv_freq(64)
    q8, k8, v8 = api.mtp_rope_prefill(q, kv[..., :128], kr, kv[..., 128:], pos, api.mtp_rope_freqs(inv, device="cuda"), 0.01,
                                      0.01, 0.01, m, True)
    cu = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    out = api.fmha_fwd_fp8_varlen(q8, k8, v8, 0.01, 0.01, 0.01, cu, cu, t, t, is_causal=True)
    full_q, full_k = f64(q), np.concatenate([f64(kv)[..., :128], np.zeros((t, h, 64))], -1)
    p = pos.cpu().numpy()
    full_q[..., 128:] = oracle.rotate(full_q[..., 128:], p, inv, 1.0, True)
    full_k[..., 128:] = oracle.rotate(f64(kr)[:, None], p, inv, 1.0, True)
    s = np.einsum("thd,khd->htk", full_q, full_k) / np.sqrt(192)
    s = np.where(np.tril(np.ones((t, t), bool)), s, -np.inf)
    w = np.exp(s - s.max(-1, keepdims=True))
    want = np.einsum("htk,khd->thd", w / w.sum(-1, keepdims=True), f64(kv)[..., 128:])
    # q and k rounded to 2^-4 of each element: the logits, sums of 192 products of unit values over
    # sqrt(192), are off by about 2^-4 / sqrt(3) * sqrt(2) = 0.05; v as much: 0.15 covers three times both
    assert np.abs(f64(out) - want).max() < 0.15 * np.abs(want).max()
