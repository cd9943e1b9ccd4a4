"""The cache's upkeep on latent vectors, and a decode loop with draft trees over a latent cache: append,
attend, verify, compact, resize, against lists of vectors kept on the host."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import rope as oracle_rope
from oracle.latent import latent_attention
from paged_fp8_speculative_gb300 import api, rope
from tests.test_tree_host import COMPACT, COMPACT_GOOD, RESIZE, RESIZE_GOOD, call

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def random_cache(g, *shape):
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device=DEV)


def held(cache, bt, length):
    """The vectors of a row, [layers, length, 576]."""
    at = torch.arange(length)
    return cache[:, bt.cpu()[at // 16].long(), at % 16].cpu()


@pytest.mark.parametrize("name,fields,good", [("mtp_cache_resize", RESIZE, RESIZE_GOOD),
                                              ("mtp_cache_compact", COMPACT, COMPACT_GOOD)], ids=["resize", "compact"])
def test_latent_caches_have_neither_values_nor_heads(name, fields, good):
    assert call(name, fields, good, v=None) == api.E_ARG
    assert call(name, fields, good, hkv=0) == api.E_ARG
    assert call(name, fields, good, v=None, hkv=0) == api.E_ARG      # layers of 256 bytes a token: too close
    assert call(name, fields, good, v=None, hkv=0, stride=10 * 16 * 576) == api.E_DEVICE


@pytest.mark.parametrize("bad", [torch.zeros(5, 16, 512, dtype=torch.uint8), torch.zeros(5, 16, 1, 256, dtype=torch.uint8),
                                 torch.zeros(2, 3, 5, 16, 576, dtype=torch.uint8), torch.zeros(5, 16, 576),
                                 torch.zeros(5, 16, 640, dtype=torch.uint8)[..., :576]])
def test_binding_refuses_other_shapes(bad):
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.mtp_cache_copy_pages(bad, None, z, z)


@pytest.mark.gpu
@pytest.mark.parametrize("layers", [1, 3])
def test_pages_are_copied(layers):
    g = torch.Generator(DEV).manual_seed(1)
    cache = random_cache(g, layers, 9, 16, 576)
    want = cache.clone()
    want[:, [5, 8]] = want[:, [0, 3]]
    api.mtp_cache_copy_pages(cache if layers > 1 else cache[0], None, i32([0, 3]), i32([5, 8]))
    assert torch.equal(cache, want)


@pytest.mark.gpu
@pytest.mark.parametrize("layers", [1, 4])
@pytest.mark.parametrize("strided", [False, True])
def test_compact(layers, strided):
    g = torch.Generator(DEV).manual_seed(2)
    lens, nodes = [40, 70, 64, 9], [9, 64, 1, 9]
    room = torch.zeros(layers, 31, 16, 576, dtype=torch.uint8, device=DEV)
    room[:] = random_cache(g, *room.shape)
    cache = room[:, :20] if strided and layers > 1 else room[:, :20].contiguous()
    bt = torch.full((4, 6), -1, dtype=torch.int32)
    order, at = torch.randperm(20), 0
    for b, n in enumerate(lens):
        k = -(-n // 16)
        bt[b, :k] = order[at:at + k]
        at += k
    bt = bt.to(DEV)
    paths = [[0, 2, 3, 8], list(range(0, 64, 3)), [0], [0, 1, 2, 3]]
    index = torch.full((4, 64), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        index[b, :len(p)] = torch.tensor(p)
    before = [held(cache, bt[b], lens[b]) for b in range(4)]
    status = i32([0])
    kept = api.mtp_cache_compact(cache if layers > 1 else cache[0], None, bt, i32(lens), i32([0, 9, 73, 74, 83]), index.to(DEV),
                                 i32([len(p) - 1 for p in paths]), status=status)
    assert status.item() == 0 and kept.tolist() == [n - m + len(p) for n, m, p in zip(lens, nodes, paths)]
    for b, p in enumerate(paths):
        start = lens[b] - nodes[b]
        want = torch.cat([before[b][:, :start], before[b][:, [start + i for i in p]]], 1)
        assert torch.equal(held(cache, bt[b], int(kept[b])), want)


@pytest.mark.gpu
def test_a_fork_and_its_growth_keep_both_rows():
    g = torch.Generator(DEV).manual_seed(3)
    cache = random_cache(g, 2, 12, 16, 576)
    bt, lens, refs = torch.full((3, 5), -1, dtype=torch.int32, device=DEV), i32([0, 0, 0]), torch.zeros(12, dtype=torch.int32, device=DEV)
    status = i32([0])
    api.mtp_cache_resize(cache, None, bt, lens, refs, i32([37, 20, 0]), status=status)
    first = held(cache, bt[0], 37)
    api.mtp_cache_fork(cache, None, bt, lens, refs, i32([0]), i32([2]), status=status)
    assert torch.equal(held(cache, bt[2], 37), first) and bt[2, 2] != bt[0, 2]
    api.mtp_cache_resize(cache, None, bt, lens, refs, i32([50, 0, 33]), status=status)
    assert torch.equal(held(cache, bt[0], 37), first) and torch.equal(held(cache, bt[2], 33), first[:, :33])
    assert status.item() == 0 and int(refs.sum()) == 4 + 3


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_a_decode_loop(captured):
    """Three steps of two sequences: tokens at any page border, a tree each, a path kept, pages given back.
    What the cache holds is compared with vectors kept on the host, and the attention with the definition
    over what the cache should hold.  Captured, a whole step is one graph replayed."""
    heads, pool, width, descale = 4, 24, 6, 0.02
    inv = rope.inv_freq(64)[0]
    freqs = api.mtp_rope_freqs(inv, device=DEV)
    g = torch.Generator(DEV).manual_seed(4)
    cache = torch.zeros(pool, 16, 576, dtype=torch.uint8, device=DEV)
    bt = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    lens, refs, status = i32([0, 0]), torch.zeros(pool, dtype=torch.int32, device=DEV), i32([0])
    d = torch.full((1,), descale, device=DEV)
    nodes = [7, 3]
    parents = [-1, 0, 0, 1, 1, 2, 3] + [-1, 0, 1]
    depth = [0, 1, 1, 2, 2, 2, 3] + [0, 1, 2]
    cu, par = i32([0, 7, 10]), i32(parents)
    rows = 10
    x = torch.zeros(rows, 576, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(rows, heads, 576, dtype=torch.bfloat16, device=DEV)
    pos, new_lens = torch.zeros(rows, dtype=torch.int32, device=DEV), i32([0, 0])
    logits, tokens = torch.zeros(rows, 50, device=DEV), torch.zeros(rows, dtype=torch.int32, device=DEV)
    out = torch.zeros(rows, heads, 512, dtype=torch.bfloat16, device=DEV)
    mask = torch.zeros(rows, dtype=torch.int64, device=DEV)
    index, count, said = (torch.zeros(2, 8, dtype=torch.int32, device=DEV), i32([0, 0]), torch.zeros(2, 8, dtype=torch.int32, device=DEV))
    kept = i32([0, 0])
    ws = torch.zeros(api.mtp_latent_attn_workspace_size(2, rows, heads, width), dtype=torch.uint8, device=DEV)
    ws2 = torch.zeros(api.mtp_cache_workspace_size(2, width), dtype=torch.uint8, device=DEV)
    ws3 = torch.zeros_like(ws2)

    def step():
        api.mtp_cache_resize(cache, None, bt, lens, refs, new_lens, ws2, status)
        api.mtp_rope_latent_append(q[..., 512:], x[:, :512], x[:, 512:], pos, freqs, cache, bt, lens, cu, d, 1.0, True,
                                   q_out=q[..., 512:], status=status)
        api.mtp_tree_mask(par, cu, mask, status)
        api.mtp_latent_attn_fwd(q, cache, bt, lens, cu, d, 0.1, tree_mask=mask, out=out, workspace=ws, status=status)
        api.mtp_tree_verify_greedy(logits, tokens, par, cu, 8, index, count, said, status)
        api.mtp_cache_compact(cache, None, bt, lens, cu, index, count, kept, status)
        api.mtp_cache_resize(cache, None, bt, lens, refs, kept, ws3, status)

    graph = None
    truth = [np.zeros((0, 576)), np.zeros((0, 576))]        # codes' values that the cache should hold
    for n in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        q.copy_(torch.randn(q.shape, generator=g, device=DEV))
        raw_q = q.clone()
        start = [len(t) for t in truth]
        if n == 0:
            start = [0, 0]
        new_lens.copy_(i32([start[0] + 7, start[1] + 3]))
        pos.copy_(i32([start[b] + depth[i] for b, first in ((0, 0), (1, 7)) for i in range(first, first + nodes[b])]))
        logits.copy_(torch.randn(logits.shape, generator=g, device=DEV))
        best = logits.argmax(-1).cpu().tolist()
        want_path = [[0, 2, 5], [0]] if n % 2 else [[0, 1, 3, 6], [0, 1, 2]]
        said_tokens = [51] * rows
        for b, first in ((0, 0), (1, 7)):
            for i in want_path[b][1:]:
                said_tokens[first + i] = best[first + parents[first + i]]
        tokens.copy_(i32(said_tokens))
        if captured and graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            saved = [t.clone() for t in (cache, bt, lens, refs, q)]
            with torch.cuda.graph(graph):
                step()
            for t, s in zip((cache, bt, lens, refs, q), saved):
                t.copy_(s)
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert status.item() == 0
        # the appended codes' values, from the definition
        p = pos.cpu().numpy()
        xv = x.double().cpu().numpy()
        turned = oracle_rope.rotate(xv[:, None, 512:], p, inv, 1.0, True)[:, 0]
        exact = oracle_rope.clipped(np.concatenate([xv[:, :512], turned], -1), descale)
        codes = torch.tensor(exact).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
        full = [np.concatenate([truth[0], codes[:7]]), np.concatenate([truth[1], codes[7:]])]
        # attention over a cache of these vectors in order
        words = mask.cpu().tolist()
        flat = np.zeros((2 * width, 16, 576), np.uint8)
        table = np.arange(2 * width).reshape(2, width)
        for b in range(2):
            v = torch.tensor(full[b]).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            for j in range(len(v)):
                flat[table[b, j // 16], j % 16] = v[j]
        qv = raw_q.double().cpu().numpy()
        qv[..., 512:] = torch.tensor(oracle_rope.rotate(qv[..., 512:], p, inv, 1.0, True)).to(torch.bfloat16).double().numpy()
        want = latent_attention(qv, flat, table, [len(f) for f in full], [0, 7, 10], words, descale, 0.1)[0]
        got = out.double().cpu().numpy()
        # a rotated element of q or of a code may lie on the other side of a rounding: 2^-7 of q's, 2^-3 of a
        # code's on few of the 576 terms of a logit; in all less than 0.05 of the outputs' spread
        assert np.abs(got - want).max() < 0.05 * want.std() + 2.0 ** -8 * np.abs(want).max()
        for b, first in ((0, 0), (1, 7)):
            path = want_path[b]
            assert index[b, :len(path)].tolist() == path and int(count[b]) == len(path) - 1
            truth[b] = np.concatenate([truth[b], codes[first:first + nodes[b]][path]])
            assert int(lens[b]) == len(truth[b])
            have = held(cache[None], bt[b], len(truth[b]))[0].view(torch.float8_e4m3fn).double().numpy()
            off = np.abs(have - truth[b]) > 0
            assert off.mean() < 1e-3 and np.all(np.abs(have - truth[b]) <= 2 * oracle_rope.half_step(truth[b]))
        assert int((refs > 0).sum()) == sum(-(-len(t) // 16) for t in truth)
