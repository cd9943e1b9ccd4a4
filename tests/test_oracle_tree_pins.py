"""The draft-tree and cache oracles against what is known otherwise: dense attention, closed
forms, the target's own distribution, and invariants of the book-keeping."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from paged_fp8_speculative_gb300 import synth
from tests.helpers import dense_sdpa_reference, oracle_args


def test_masks_of_a_chain_and_of_a_star():
    assert oracle.tree.ancestors([-1, 0, 1, 2]) == [1, 3, 7, 15]
    assert oracle.tree.ancestors([-1, 0, 0, 0]) == [1, 3, 5, 9]
    assert oracle.tree.ancestors([-1] + list(range(63)))[63] == (1 << 64) - 1


def test_a_chain_is_the_verify_attention():
    b = synth.make_batch([70, 5, 33], [4, 3, 1], 16, 2, seed=3, k_descale=0.5, v_descale=2.0,
                         kv_recipe="unit")
    masks = [m for n in (4, 3, 1) for m in oracle.tree.ancestors([i - 1 for i in range(n)])]
    a = oracle_args(b)
    out, weight, reach = oracle.tree.tree_attention(*a[:6], masks, *a[6:])
    assert np.allclose(out, dense_sdpa_reference(b), rtol=1e-12, atol=1e-12)
    assert (weight >= np.abs(out) - 1e-12).all() and (reach > 0).all()


def test_a_branch_is_the_sequence_without_the_other_branches():
    # nodes 0 - 1 - 3 and 0 - 2: node 3's row is the chain over keys prefix, 0, 1, 3
    b = synth.make_batch([20], [4], 8, 1, seed=4, kv_recipe="unit")
    masks = oracle.tree.ancestors([-1, 0, 0, 1])
    a = oracle_args(b)
    out, _, _ = oracle.tree.tree_attention(*a[:6], masks, *a[6:])
    seen = list(range(17)) + [17, 19]
    table = b.block_tables[0].numpy()
    k = oracle.E4M3_TABLE[b.k_cache.numpy()[table[np.array(seen) // 16], np.array(seen) % 16, 0]]
    v = oracle.E4M3_TABLE[b.v_cache.numpy()[table[np.array(seen) // 16], np.array(seen) % 16, 0]]
    q = b.q[3].double().numpy()
    w = np.exp(b.softmax_scale * q @ k.T)
    assert np.allclose(out[3], w / w.sum(1, keepdims=True) @ v, rtol=1e-10)


def test_no_visible_key_gives_zeros():
    b = synth.make_batch([3], [3], 8, 1, seed=5, kv_recipe="unit")
    a = oracle_args(b)
    out, _, _ = oracle.tree.tree_attention(*a[:6], [0, 1, 0], *a[6:])
    assert not out[0].any() and not out[2].any() and out[1].any()


def test_greedy_walk():
    z = np.zeros((5, 4))
    z[0, 2] = z[1, 3] = z[3, 1] = 1          # root -> 2, node 1 -> 3, node 3 -> 1
    tokens, parents = [9, 2, 2, 3, 0], [-1, 0, 0, 1, 3]
    index, n, said = oracle.tree.verify_greedy(z, tokens, parents, 8)
    assert n == 2 and list(index[:3]) == [0, 1, 3] and list(said[:3]) == [2, 3, 1]
    assert (index[3:] == -1).all() and (said[3:] == -1).all()
    index, n, said = oracle.tree.verify_greedy(z, tokens, parents, 2)      # one accepted at most
    assert n == 1 and list(said) == [2, 3]


@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("width", [1, 3])
def test_first_emitted_token_follows_the_target(drafter, width):
    """Rejection sampling keeps the target's distribution whatever the drafter's: the first
    emitted token's counts, 20000 walks, within 5 standard deviations per token."""
    rng = np.random.default_rng(7 + width)
    V, N = 6, 20000
    p, q = rng.dirichlet(np.ones(V), size=2)
    p, q = np.tile(p, (width + 1, 1)), np.tile(q, (width + 1, 1))
    parents = [-1] + [0] * width
    counts = np.zeros(V)
    fixed = rng.choice(V, size=width, replace=False)
    for _ in range(N):
        tokens = [0] + list(rng.choice(V, size=width, p=q[0]) if drafter else fixed)
        _, _, said = oracle.tree.verify_sample(p, q if drafter else None, tokens, parents,
                                               rng.random(width + 1), 4)
        counts[said[0]] += 1
    sd = np.sqrt(N * p[0] * (1 - p[0]))
    assert (np.abs(counts - N * p[0]) < 5 * sd).all(), (counts / N, p[0])


def _random_cache(rng, rows, width, pool, layers=2):
    caches = [rng.integers(0, 256, (layers, pool, 16, 1, 4), dtype=np.uint8) for _ in range(2)]
    return (caches, np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32),
            np.zeros(pool, np.int32))


def _tokens(caches, tables, lens, b):
    pos = np.arange(lens[b])
    return [c[:, tables[b, pos // 16], pos % 16].copy() for c in caches]


def test_book_keeping_keeps_its_invariants():
    rng = np.random.default_rng(11)
    caches, tables, lens, counts = _random_cache(rng, 6, 8, 40)
    for step in range(200):
        before = {b: _tokens(caches, tables, lens, b) for b in range(6)}
        old = lens.copy()
        empty = [b for b in range(6) if lens[b] == 0]
        if empty and rng.random() < 0.4:
            src = int(rng.integers(6))
            if src not in empty and oracle.cache.fork(caches, tables, lens, counts, [src], [empty[0]]):
                for x, y in zip(before[src], _tokens(caches, tables, lens, empty[0])):
                    assert np.array_equal(x, y)
        else:
            new = [int(rng.integers(0, 129)) if rng.random() < 0.5 else int(n) for n in lens]
            oracle.cache.resize(caches, tables, lens, counts, new)
        for b in range(6):                         # what a row held it still holds
            n = min(old[b], lens[b])
            for x, y in zip(before[b], _tokens(caches, tables, lens, b)):
                assert np.array_equal(x[:, :n], y[:, :n])
        held = np.zeros_like(counts)
        for b in range(6):
            n = -(-lens[b] // 16)
            assert (tables[b, n:] == -1).all() and (tables[b, :n] >= 0).all()
            np.add.at(held, tables[b, :n], 1)
            if lens[b] % 16:
                assert counts[tables[b, n - 1]] == 1
        assert np.array_equal(held, counts)


def test_compaction_keeps_the_path():
    rng = np.random.default_rng(12)
    caches, tables, lens, counts = _random_cache(rng, 2, 4, 10)
    oracle.cache.resize(caches, tables, lens, counts, [40, 9])
    was = [_tokens(caches, tables, lens, b) for b in range(2)]
    index = np.array([[0, 2, 5, 6], [0, -1, -1, -1]])
    new = oracle.cache.compact(caches, tables, lens, [10, 9], index, [3, 0])
    assert list(new) == [34, 1]
    now = _tokens(caches, tables, new, 0)
    for x, y in zip(was[0], now):
        assert np.array_equal(y, x[:, list(range(30)) + [30, 32, 35, 36]])
