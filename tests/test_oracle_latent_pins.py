"""Pins of the rotary and latent oracles: complex products, dense attention, closed forms, invariants."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from oracle import latent, rope


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, pos, f = rng.normal(size=(5, 3, 40)), np.array([0, 1, -7, 100000, 2 ** 31 - 1]), np.array([1.0, 0.1, 1e-3, 0.5])
    y = rope.rotate(x, pos, f, 1.25, interleaved)
    z = x[..., 0:8:2] + 1j * x[..., 1:8:2] if interleaved else x[..., :4] + 1j * x[..., 4:8]
    w = 1.25 * z * np.exp(1j * np.outer(pos, f))[:, None]
    got = y[..., 0:8:2] + 1j * y[..., 1:8:2] if interleaved else y[..., :4] + 1j * y[..., 4:8]
    assert np.allclose(got, w, atol=1e-12) and np.array_equal(y[..., 8:], x[..., 8:])


def test_rotation_keeps_relative_angles():
    """Products of a query at m and a key at n depend on m - n only."""
    rng = np.random.default_rng(2)
    a, b, f = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16)), 10.0 ** -np.arange(8)
    def dot(m, n):
        return float(np.sum(rope.rotate(a, [m], f) * rope.rotate(b, [n], f)))
    assert dot(5, 2) == pytest.approx(dot(1005, 1002), abs=1e-9)
    assert np.allclose(rope.rotate(rope.rotate(a, [9], f), [-9], f), a)


def test_half_step_is_torchs():
    values = oracle.E4M3_TABLE[:0x7f]                    # ascending, 0 .. 448
    for lo, hi in zip(values[:-1], values[1:]):
        mid = (lo + hi) / 2
        assert rope.half_step(mid) == (hi - lo) / 2
        assert abs(float(torch.tensor(mid * 1.0001).to(torch.float8_e4m3fn)) - mid) <= rope.half_step(mid) * 1.001


def test_places():
    bt = np.array([[7, 3], [1, 2]])
    got = rope.places(bt, [17, 20], [0, 2, 5], 6)
    assert got == [(7, 15), (3, 0), (2, 1), (2, 2), (2, 3), None]


def batch(seed, lens, nodes, heads):
    rng = np.random.default_rng(seed)
    pages = [-(-n // 16) for n in lens]
    codes = rng.integers(0, 256, size=(sum(pages) + 1, 16, 576), dtype=np.uint8)
    codes[(codes & 0x7f) == 0x7f] = 0
    codes &= 0xbf                                        # small values
    bt = np.full((len(lens), max(pages)), -1, np.int64)
    order, at = rng.permutation(sum(pages)), 0
    for b, n in enumerate(pages):
        bt[b, :n] = order[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(nodes)])
    return rng.normal(size=(cu[-1], heads, 576)), codes, bt, np.array(lens), cu


def test_latent_is_dense_attention():
    q, codes, bt, lens, cu = batch(3, [40, 17, 5], [3, 1, 5], 2)
    out = latent.latent_attention(q, codes, bt, lens, cu, None, 0.5, 0.1)[0]
    for b, L in enumerate(lens):
        rows = torch.tensor(codes[bt[b, :-(-L // 16)]].reshape(-1, 576)[:L]).view(torch.float8_e4m3fn).double() * 0.5
        n = cu[b + 1] - cu[b]
        s = torch.einsum("thd,kd->htk", torch.tensor(q[cu[b]:cu[b + 1]]), rows) * 0.1
        s = s.masked_fill(~torch.ones(n, L, dtype=torch.bool).tril(L - n), -torch.inf)
        want = torch.einsum("htk,kd->thd", s.softmax(-1), rows[:, :512])
        assert np.allclose(out[cu[b]:cu[b + 1]], want.numpy(), atol=1e-12)


def test_latent_masks():
    q, codes, bt, lens, cu = batch(4, [20, 3], [4, 3], 2)
    chain = latent.latent_attention(q, codes, bt, lens, cu, None, 1.0, 0.1)[0]
    words = [1, 3, 7, 15, 1, 3, 7]
    assert np.array_equal(chain, latent.latent_attention(q, codes, bt, lens, cu, words, 1.0, 0.1)[0])
    words[4] = 0                                         # sees nothing: no token is before the new ones
    out = latent.latent_attention(q, codes, bt, lens, cu, words, 1.0, 0.1)[0]
    assert not out[4].any() and np.array_equal(out[5:], chain[5:])
    words[4] = 4                                         # one token alone: its own values
    out = latent.latent_attention(q, codes, bt, lens, cu, words, 1.0, 0.1)[0]
    assert np.allclose(out[4], oracle.E4M3_TABLE[codes[bt[1, 0], 2]][:512])


def test_latent_scales():
    q, codes, bt, lens, cu = batch(5, [30], [2], 3)
    a = latent.latent_attention(q, codes, bt, lens, cu, None, 2.0, 0.05)
    b = latent.latent_attention(q, codes, bt, lens, cu, None, 1.0, 0.1)
    assert np.allclose(a[0], 2 * b[0]) and np.allclose(a[1], 2 * b[1]) and np.allclose(a[3], b[3])
