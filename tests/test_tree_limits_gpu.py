"""The draft-tree and cache calls at their limits: nothing to do, byte offsets past 2^31, the
largest tables, calls side by side on two streams, graphs that share a workspace, distributions that
are not, comparisons that hang on a last bit."""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

import oracle
from paged_fp8_speculative_gb300 import api
from tests.test_cache_pages_gpu import Pair
from tests.test_tree_attn_gpu import Batch, check, run
from tests.test_tree_verify_gpu import draw, greedy, packed, sample, trees_of, walkable

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_calls_with_nothing_to_do():
    none, cu = i32([]), i32([0])
    k = torch.zeros(4, 16, 2, 256, dtype=torch.uint8, device="cuda")
    assert api.mtp_tree_mask(none, cu).shape == (0,)
    q = torch.zeros(0, 8, 256, dtype=torch.bfloat16, device="cuda")
    out = api.mtp_tree_attn_fwd(q, k, k, i32([]).view(0, 3), none, cu, none.long(), 1.0, 1.0, 0.1)
    assert out.shape == (0, 8, 256)
    rows = torch.zeros(0, 100, device="cuda")
    for got in (api.mtp_tree_verify_greedy(rows, none, none, cu),
                api.mtp_tree_verify_sample(rows, None, none, none, cu, torch.zeros(0, device="cuda"))):
        assert [tuple(x.shape) for x in got] == [(0, 64), (0,), (0, 64)]
    refs = i32([0] * 4)
    api.mtp_cache_resize(k, k, i32([]).view(0, 3), none, refs, none)
    api.mtp_cache_fork(k, k, i32([[-1, -1]]), i32([0]), refs, none, none)
    api.mtp_cache_copy_pages(k, k, none, none)
    assert api.mtp_cache_compact(k, k, i32([]).view(0, 3), none, cu, i32([]).view(0, 8), none).shape == (0,)
    torch.cuda.synchronize()
    assert not k.any() and not refs.any()


@pytest.mark.parametrize("lens,nodes,hkv,ratio", [
    ([300] * 400, [3] * 400, 1, 8),                 # several whole units a CTA
    ([260 + 7 * (i % 20) for i in range(310)], [1 + i % 9 for i in range(310)], 1, 16),
    ([129] * 33 + [128] * 100 + [640] * 70, [2] * 203, 2, 4),
    ([64 + i for i in range(90)], [64] * 90, 1, 16),   # eight row tiles a sequence
    ([120000], [9], 1, 2),                          # one unit, a piece for every CTA
    ([50000, 33], [64, 33], 1, 16),
], ids=["whole", "mixed", "short", "wide", "long", "longwide"])
def test_many_units_and_long_ones(lens, nodes, hkv, ratio):
    batch = Batch(lens, nodes, hkv, ratio, seed=len(lens))
    check(run(batch), batch)


def test_sequences_that_claim_the_same_rows_again_and_again():
    """cu_seqlens_q 0, 320, 0, 320, ...: nothing is computed; the next call is as ever."""
    batch = Batch([200] * 64, [5] * 64, 1, 8, seed=9)
    want = run(batch)
    args = batch.device()
    good = args["cu_seqlens_q"]
    args["cu_seqlens_q"] = i32([0] + [320, 0] * 32)
    out, status = torch.full_like(want, 5.0), i32([0])
    api.mtp_tree_attn_fwd(**args, out=out, status=status)
    assert status.item() == api.ERR_QLEN and bool((out == 5.0).all())
    args["cu_seqlens_q"] = good
    assert torch.equal(api.mtp_tree_attn_fwd(**args, out=out), want)


@pytest.fixture(scope="module")
def huge():
    """A cache of 66000 pages of 32 KB: byte offsets of the last ones pass 2^31 (and 2^32 in all)."""
    hkv, pages = 8, 66000
    assert pages * 16 * hkv * 256 > 1 << 31
    k = torch.zeros(2, pages, 16, hkv, 256, dtype=torch.uint8, device="cuda")
    yield k, torch.zeros_like(k)


def test_attention_over_far_pages(huge):
    batch = Batch([700, 90], [11, 5], 8, 2, seed=5)
    want = run(batch)
    args = batch.device()
    pool = args["k_cache"].shape[0]
    for name, cache in (("k_cache", huge[0]), ("v_cache", huge[1])):
        cache[1, -pool:] = args[name]
        args[name] = cache[1]
    args["block_tables"] = torch.where(args["block_tables"] < 0, -1, args["block_tables"] + huge[0].shape[1] - pool)
    assert torch.equal(api.mtp_tree_attn_fwd(**args), want)


def test_upkeep_of_far_pages(huge):
    k, v = huge
    pages = k.shape[1]
    g = torch.Generator(device="cuda").manual_seed(3)
    fill = torch.randint(0, 255, (2, 2, 16, 8, 256), dtype=torch.uint8, device="cuda", generator=g)
    a, b = pages - 1, pages - 7
    k[:, a], v[:, a] = fill[0], fill[1]
    api.mtp_cache_copy_pages(k, v, i32([a]), i32([b]))
    assert torch.equal(k[:, b], fill[0]) and torch.equal(v[:, b], fill[1])
    # a tree of 6 nodes behind 9 tokens in page a: nodes 0, 2, 5 are kept
    lens = api.mtp_cache_compact(k, v, i32([[a]]), i32([15]), i32([0, 6]), i32([[0, 2, 5, -1]]), i32([2]))
    assert lens.tolist() == [12]
    for c, f in ((k, fill[0]), (v, fill[1])):
        assert torch.equal(c[:, a, :10], f[:, :10])
        assert torch.equal(c[:, a, 10], f[:, 11]) and torch.equal(c[:, a, 11], f[:, 14])
    # the only free page is far out; the fork's half-filled last page is copied into it
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[b] = 0
    bt, sl = i32([[a, -1], [-1, -1]]), i32([12, 0])
    api.mtp_cache_fork(k, v, bt, sl, refs, i32([0]), i32([1]))
    assert bt.tolist() == [[a, -1], [b, -1]] and sl.tolist() == [12, 12] and refs[b].item() == 1
    assert torch.equal(k[:, b], k[:, a]) and torch.equal(v[:, b], v[:, a])


def test_rows_of_scores_far_apart():
    """Element offsets past 2^31 between the rows of one tree."""
    vocab, stride = 5003, (1 << 30) + 9
    memory = torch.zeros(2 * stride + vocab, dtype=torch.bfloat16, device="cuda")
    logits = memory.as_strided((3, vocab), (stride, 1))
    rng = np.random.default_rng(0)
    logits.copy_(torch.randn(3, vocab, device="cuda"))
    tokens = walkable(logits, [[-1, 0, 1]], rng, vocab)
    best = logits.float().argmax(1).tolist()
    greedy(logits, [[-1, 0, 1]], [0, best[0], best[1]])
    greedy(logits, [[-1, 0, 1]], tokens)
    p = torch.softmax(torch.randn(3, vocab, device="cuda"), -1).bfloat16()
    logits.copy_(p)
    u = torch.tensor([0.3, 0.0, 0.0], device="cuda")     # both are accepted
    assert sample(logits, None, [[-1, 0, 1]], [0, 7, 9], u)[1][1].item() == 2


def test_the_largest_table():
    """8192 rows, forks of 4096 of them, and back to nothing."""
    c = Pair(8192, 3, 20000, layers=1, hkv=1, seed=4)
    rng = np.random.default_rng(4)
    c.resize([int(x) for x in np.where(np.arange(8192) < 4096, rng.integers(0, 49, 8192), 0)])
    c.fork([int(x) for x in rng.permutation(4096)], list(range(4096, 8192)))
    c.resize([min(48, int(n) + int(x)) for n, x in zip(c.lens, rng.integers(0, 9, 8192))])
    c.resize([0] * 8192)
    assert not c.counts.any()


def test_forks_of_a_few_rows_into_all_others():
    """More pairs than a plan has threads."""
    c = Pair(8192, 2, 9000, layers=1, hkv=1, seed=6)
    c.resize([17, 5, 32, 16] + [0] * 8188)
    c.fork([int(x) for x in np.random.default_rng(6).integers(0, 4, 8188)], list(range(4, 8192)))
    assert min(c.lens) == 5


def test_two_streams_side_by_side():
    """Calls on two streams, issued by two host threads, each with outputs and workspaces of its own."""
    batches = [Batch([3000, 40], [16, 5], 1, 16, seed=21), Batch([2500], [64], 2, 8, seed=22)]
    wants = [run(b) for b in batches]
    draws = [draw([20, 30], 9000, s) for s in (23, 24)]
    said = []
    for p, q, trees, tokens, u in draws:
        said.append(sample(p, q, trees, tokens, u)[1])
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        args = batches[i].device()
        p, q, trees, tokens, u = draws[i]
        tree = packed(trees, tokens)
        torch.cuda.synchronize()
        for _ in range(30):
            out = api.mtp_tree_attn_fwd(**args, stream=stream)
            got = api.mtp_tree_verify_sample(p, q, *tree, u, stream=stream)
            stream.synchronize()
            if not torch.equal(out, wants[i]) or not all(torch.equal(x, y) for x, y in zip(got, said[i])):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_graphs_that_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn on one stream, and eager ones between."""
    batches = [Batch([5000, 40], [16, 5], 1, 16, seed=31), Batch([2500, 900, 31], [64, 3, 9], 1, 16, seed=32)]
    size = max(api.mtp_tree_attn_workspace_size(len(b.lens), int(b.cu[-1]), 16, 1, b.bt.shape[1]) for b in batches)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    wants, args, outs, graphs = [run(b) for b in batches], [], [], []
    for b in batches:
        args.append(b.device())
        outs.append(torch.empty_like(args[-1]["q"]))
    torch.cuda.synchronize()
    for a, out in zip(args, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            api.mtp_tree_attn_fwd(**a, out=out, workspace=ws)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        other = api.mtp_tree_attn_fwd(**args[1 - i], workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(outs[i], wants[i]) and torch.equal(other, wants[1 - i])


def test_comparisons_that_hang_on_a_last_bit():
    """u q Z < p is decided exactly, whatever the numbers' sizes: q = p is accepted for every u, a p of
    half of q where u < 1/2, and where u is 1/2 it is not."""
    vocab = 64
    for size in (1.0, 2.0 ** -20, 2.0 ** -60, 2.0 ** -126, 2.0 ** -140):
        p, q = torch.zeros(2, vocab, device="cuda"), torch.zeros(2, vocab, device="cuda")
        p[0, 3] = q[0, 3] = 0.75 * size
        p[0, 4] = p[1, 5] = 0.25
        below = float(np.nextafter(np.float32(0.5), np.float32(0)))
        for u, half, kept in ((1 - 2.0 ** -24, 1.0, 1), (below, 0.5, 1), (0.5, 0.5, 0), (2.0 ** -140, 0.5, 1)):
            p[0, 3] = 0.75 * size * half
            got = api.mtp_tree_verify_sample(p, q, *packed([[-1, 0]], [0, 3]),
                                             torch.tensor([0.1, u], device="cuda"))
            assert got[1].item() == kept, (size, u, half)


def test_rows_that_are_no_distributions():
    """Infinities, negative numbers and NaN are taken into [0, 1]; rows need not sum to 1."""
    vocab = 3001
    p, q, trees, tokens, u = draw([12, 9], vocab, 41)
    p[:, ::7], q[:, 1::11] = float("inf"), float("inf")
    p[:, 3::13], q[:, 5::17] = float("nan"), -1.0
    clean = lambda x: torch.nan_to_num(x, nan=0.0).clamp(0, 1)
    tree = packed(trees, tokens)
    for drafter in (q, None):
        got = api.mtp_tree_verify_sample(p, drafter, *tree, u)
        want = api.mtp_tree_verify_sample(clean(p), None if drafter is None else clean(q), *tree, u)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        sample(clean(p), None if drafter is None else clean(q), trees, tokens, u)


def test_a_token_outside_is_refused_whatever_the_row_sums_to():
    """Without a drafter, behind refused children that had nearly all, or more than all, of the mass."""
    p = torch.zeros(5, 10, device="cuda")
    for first, second in ((0.875, 0.124), (1.0 - 2.0 ** -23, 2.0 ** -30), (0.75, 0.125)):
        p[0, :3] = torch.tensor([first, second, 0.5])
        u = torch.tensor([0.5, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 0.0, 0.5], device="cuda")
        for last in ([10, -1], [1 << 30, 10]):
            assert sample(p, None, [[-1, 0, 0, 0, 0]], [0, 0, 1] + last, u)[1][1].item() == 0


def test_the_same_rows_whatever_the_batch():
    """A sequence's result does not depend on how many CTAs it gets: alone, and among 200."""
    p, q, trees, tokens, u = draw([26], 20000, 51, spread=1.0)
    one = sample(p, q, trees, tokens, u)[1]
    n = 200
    tree = packed(trees * n, tokens * n)
    many = api.mtp_tree_verify_sample(p.repeat(n, 1), q.repeat(n, 1), *tree, u.repeat(n))
    for x, y in zip(one, many):
        assert all(torch.equal(x[0], row) for row in y)


def test_a_status_word_of_another_type_is_refused():
    logits = torch.zeros(1, 10, device="cuda")
    for status in (torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int16, device="cuda"), i32([])):
        with pytest.raises(ValueError, match="status"):
            api.mtp_tree_verify_greedy(logits, *packed([[-1]], [0]), status=status)
