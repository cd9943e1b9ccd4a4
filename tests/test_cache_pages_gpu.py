"""The cache's upkeep against the host oracle: tables, counts, lengths and contents, all equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from paged_fp8_speculative_gb300 import api

pytestmark = pytest.mark.gpu


class Pair:
    """The same cache on the host (oracle) and on the device."""

    def __init__(self, rows, width, pool, layers=2, hkv=1, seed=0):
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.caches = [rng.integers(0, 256, (layers, pool, 16, hkv, 256), dtype=np.uint8) for _ in range(2)]
        self.tables = np.full((rows, width), -1, np.int32)
        self.lens = np.zeros(rows, np.int32)
        self.counts = np.zeros(pool, np.int32)
        d = lambda x: torch.as_tensor(x.copy()).cuda()
        self.dev = [d(self.caches[0]), d(self.caches[1]), d(self.tables), d(self.lens), d(self.counts)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def resize(self, new, **more):
        fits = oracle.cache.resize(self.caches, self.tables, self.lens, self.counts, new)
        api.mtp_cache_resize(*self.dev, torch.tensor(new, dtype=torch.int32, device="cuda"),
                             status=self.status, **more)
        self.same(0 if fits else api.ERR_FULL)

    def fork(self, src, dst):
        fits = oracle.cache.fork(self.caches, self.tables, self.lens, self.counts, src, dst)
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        api.mtp_cache_fork(*self.dev, i(src), i(dst), status=self.status)
        self.same(0 if fits else api.ERR_FULL)

    def same(self, status=0):
        assert self.status.item() == status
        self.status.zero_()
        for x, y in zip(self.dev, self.caches + [self.tables, self.lens, self.counts]):
            assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("rows,width,pool,layers,hkv", [(1, 1, 1, 1, 1), (3, 4, 9, 2, 1), (6, 9, 40, 1, 3),
                                                        (40, 6, 300, 2, 2), (100, 20, 5000, 1, 1),
                                                        (300, 12, 4097, 1, 1)])
def test_random_sequences_of_calls(rows, width, pool, layers, hkv):
    c = Pair(rows, width, pool, layers, hkv, seed=rows)
    for step in range(25):
        empty = [b for b in range(rows) if c.lens[b] == 0]
        full = [b for b in range(rows) if c.lens[b]]
        if empty and full and c.rng.random() < 0.5:
            n = int(c.rng.integers(1, len(empty) + 1))
            dst = [int(x) for x in c.rng.permutation(empty)[:n]]
            c.fork([int(x) for x in c.rng.choice(full, n)], dst)
        else:
            new = []
            for b in range(rows):
                r = c.rng.random()
                new.append(int(c.lens[b]) if r < 0.4 else 0 if r < 0.55 else
                           int(c.rng.integers(0, 16 * width + 1)) if r < 0.75 else
                           max(0, min(16 * width, int(c.lens[b]) + int(c.rng.integers(-40, 41)))))
            c.resize(new)


def test_a_pool_that_is_too_small_changes_nothing_but_what_shrinks():
    c = Pair(3, 8, 10)
    c.resize([64, 40, 16])                     # 4 + 3 + 1 pages: two are free
    c.resize([80, 40 + 16, 32])                # wants three
    assert list(c.lens) == [64, 40, 16]
    c.resize([128, 16, 0])                     # gives three back first: 4 + 2 + 2 + 1 free
    assert list(c.lens) == [128, 16, 0]
    c.resize([120, 24, 0])
    c.fork([0], [2])                           # its last page needs a copy; none is free
    assert list(c.lens) == [120, 24, 0]


def test_forks_of_one_row_share_its_full_pages():
    c = Pair(6, 6, 30)
    c.resize([70, 0, 0, 32, 0, 0])
    c.fork([0, 0, 3, 0], [1, 2, 4, 5])         # 32 = two full pages: nothing copied
    assert c.counts[c.tables[0, 0]] == 4 and c.counts[c.tables[3, 0]] == 2
    c.resize([20, 70, 75, 32, 20, 0])          # shrunk into shared pages: copied first
    c.resize([90, 70, 80, 40, 33, 1])


def test_two_rows_shrunk_into_the_same_shared_page():
    c = Pair(3, 5, 12)
    c.resize([50, 0, 0])
    c.fork([0, 0], [1, 2])
    c.resize([20, 21, 50])                     # rows 0 and 1 part from row 2's page 1
    c.resize([4, 4, 4])


def test_no_row_and_every_row():
    c = Pair(5, 3, 15)
    c.resize([48] * 5)                         # the whole pool
    c.resize([48] * 5)                         # nothing to do
    c.resize([0] * 5)
    assert not c.counts.any()


def test_a_large_pool():
    c = Pair(1000, 30, 60000, layers=1, seed=3)
    for _ in range(3):
        c.resize([int(x) for x in c.rng.integers(0, 481, 1000)])
    dst = [b for b in range(1000) if c.lens[b] == 0]
    c.resize([0 if b % 2 else int(c.lens[b]) for b in range(1000)])
    c.fork(list(range(0, 1000, 2)), list(range(1, 1000, 2)))


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_pairs_that_are_not():
    c = Pair(6, 4, 20)
    c.resize([40, 30, 0, 0, 0, 20])
    want = [x.clone() for x in c.dev]
    # outside, onto itself, onto a row that holds tokens; then a dst named twice: the first stands
    for src, dst in (([0], [6]), ([-1], [2]), ([0], [-2]), ([9], [2]), ([2], [2]), ([0], [1])):
        api.mtp_cache_fork(*c.dev, _ints(src), _ints(dst), status=c.status)
        assert c.status.item() == api.ERR_CACHE_ROW, (src, dst)
        c.status.zero_()
        assert all(torch.equal(a, b) for a, b in zip(c.dev, want))
    api.mtp_cache_fork(*c.dev, _ints([5, 0, 1, 0]), _ints([3, 2, 2, 1]), status=c.status)
    assert c.status.item() == api.ERR_CACHE_ROW
    c.status.zero_()
    oracle.cache.fork(c.caches, c.tables, c.lens, c.counts, [5, 0], [3, 2])
    c.same()
    # a source that is another pair's dst has no tokens yet: its fork is empty too
    api.mtp_cache_fork(*c.dev, _ints([4]), _ints([4]), status=c.status)
    c.status.zero_()
    c.resize([40, 30, 0, 0, 0, 20])
    api.mtp_cache_fork(*c.dev, _ints([2, 0]), _ints([3, 2]), status=c.status)
    oracle.cache.fork(c.caches, c.tables, c.lens, c.counts, [0], [2])
    c.same()


def test_bad_lengths_tables_and_counts():
    c = Pair(4, 4, 20)
    c.resize([40, 30, 20, 10])
    api.mtp_cache_resize(*c.dev, _ints([65, -1, 33, 1 << 30]), status=c.status)
    assert c.status.item() == api.ERR_LEN
    c.status.zero_()
    oracle.cache.resize(c.caches, c.tables, c.lens, c.counts, [40, 30, 33, 10])
    c.same()                                   # the good row went through, the others stayed
    c.dev[2][0, 2] = 20                        # outside the pool: only cleared
    api.mtp_cache_resize(*c.dev, _ints([32, 30, 33, 10]), status=c.status)
    assert c.status.item() == 4
    assert c.dev[2][0, 2].item() == -1 and c.dev[3][0].item() == 32
    c.status.zero_()
    page = int(c.dev[2][1, 1])
    c.dev[4][page] = 0                         # a count that was lost
    api.mtp_cache_resize(*c.dev, _ints([32, 16, 33, 10]), status=c.status)
    assert c.status.item() == api.ERR_REF and c.dev[4][page].item() == 0


def test_fork_of_a_row_with_a_bad_entry():
    c = Pair(4, 4, 20)
    c.resize([40, 30, 0, 0])
    c.dev[2][0, 1] = -7
    api.mtp_cache_fork(*c.dev, _ints([0, 1]), _ints([2, 3]), status=c.status)
    assert c.status.item() == 4
    assert c.dev[3].tolist() == [40, 30, 0, 30] and (c.dev[2][2] == -1).all()


@pytest.mark.parametrize("layers,hkv,pool,pairs", [(1, 1, 3, 1), (3, 2, 200, 60), (60, 1, 50, 25)])
def test_copy_pages(layers, hkv, pool, pairs):
    c = Pair(1, 1, pool, layers, hkv, seed=5)
    perm = c.rng.permutation(pool)
    src, dst = perm[:pairs], perm[pairs:2 * pairs]
    for x in c.caches:
        x[:, dst] = x[:, src]
    api.mtp_cache_copy_pages(c.dev[0], c.dev[1], _ints(src), _ints(dst), status=c.status)
    c.same()
    api.mtp_cache_copy_pages(c.dev[0], c.dev[1], _ints([0, -1, pool, 1]), _ints([pool, 0, 1, 1]),
                             status=c.status)
    c.same(4)


def test_one_layer_and_layers_with_gaps():
    c = Pair(1, 1, 8, layers=4, hkv=2)
    k, v = c.dev[0], c.dev[1]
    want = [k.clone(), v.clone()]
    api.mtp_cache_copy_pages(k[::2], v[::2], _ints([1]), _ints([5]))      # layers 0 and 2
    for w in want:
        w[::2, 5] = w[::2, 1]
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    api.mtp_cache_copy_pages(k[3], v[3], _ints([2]), _ints([6]))
    for w in want:
        w[3, 6] = w[3, 2]
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.parametrize("layers,hkv,nodes,lens", [
    (1, 1, [1], [1]), (1, 1, [8], [8]), (2, 3, [5, 64, 33], [16, 64, 500]),
    (7, 2, [20] * 30, list(range(20, 50))), (40, 1, [64, 64], [79, 81])])
def test_compact(layers, hkv, nodes, lens):
    rows = len(lens)
    width = max(-(-n // 16) for n in lens)
    c = Pair(rows, width, sum(-(-n // 16) for n in lens) + 4, layers, hkv, seed=rows + layers)
    c.resize(lens)
    index, count = np.full((rows, 64), -1, np.int32), np.zeros(rows, np.int32)
    for b, n in enumerate(nodes):
        path = [0] + [i for i in range(1, n) if c.rng.random() < 0.5]
        index[b, :len(path)], count[b] = path, len(path) - 1
    new = oracle.cache.compact(c.caches, c.tables, c.lens, nodes, index, count)
    got = api.mtp_cache_compact(*c.dev[:4], _ints(np.cumsum([0] + nodes)), _ints(index), _ints(count),
                                status=c.status)
    assert np.array_equal(got.cpu().numpy(), new)
    c.same()
    c.resize([int(x) for x in new])            # what is not kept goes back


def test_compact_of_paths_that_are_not():
    c = Pair(7, 4, 40)
    c.resize([30] * 7)
    index = np.full((7, 6), -1, np.int32)
    index[:, 0] = 0
    index[0, 1:3] = [3, 2]                     # not ascending
    index[1, 1:3] = [4, 4]                     # the same node twice
    index[2, 1] = 8                            # past the tree of 8
    index[3, 0] = 1                            # not from the root
    index[4, 1:3] = [2, 5]
    count = [2, 2, 1, 0, 2, -1, 6]
    nodes = [8] * 7
    got = api.mtp_cache_compact(*c.dev[:4], _ints(np.cumsum([0] + nodes)), _ints(index), _ints(count),
                                status=c.status)
    assert c.status.item() == api.ERR_LEN
    c.status.zero_()
    only = np.array([[0] + [-1] * 5] * 7, np.int32)
    only[4] = index[4]
    oracle.cache.compact([x for x in c.caches], c.tables, c.lens, nodes, only, [0, 0, 0, 0, 2, 0, 0])
    c.same()
    assert got.tolist() == [30, 30, 30, 30, 25, 30, 30]


@pytest.mark.parametrize("what,bit", [("page", 4), ("short", 2), ("long", 8), ("qlen", 1)])
def test_compact_of_bad_rows(what, bit):
    c = Pair(2, 4, 20)
    c.resize([30, 30])
    nodes = [8, 8]
    cu = _ints(np.cumsum([0] + nodes))
    if what == "page":
        c.dev[2][0, 1] = c.tables[0, 1] = 20
    elif what == "short":
        c.dev[3][0] = c.lens[0] = 7
    elif what == "long":
        c.dev[3][0] = c.lens[0] = 65
    else:
        cu[0] = 9
    index = _ints([[0, 3], [0, 5]])
    got = api.mtp_cache_compact(*c.dev[:4], cu, index, _ints([1, 1]), status=c.status)
    assert c.status.item() == bit
    assert got[0].item() == c.lens[0]
    if what != "qlen":
        for x in c.caches:
            x[:, c.tables[1, 23 // 16], 23 % 16] = x[:, c.tables[1, 27 // 16], 27 % 16]
        c.same(bit)


def test_streams_and_graphs():
    c = Pair(4, 6, 40)
    c.resize([50, 20, 0, 0])
    ws = torch.full((api.mtp_cache_workspace_size(4, 6),), 0xFF, dtype=torch.uint8, device="cuda")
    new, src, dst = _ints([50, 20, 0, 0]), _ints([0, 1]), _ints([2, 3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.mtp_cache_resize(*c.dev, new, workspace=ws, status=c.status)
        api.mtp_cache_fork(*c.dev, src, dst, workspace=ws, status=c.status)
    for lens in ([50, 20, 0, 0], [60, 10, 0, 0], [7, 90, 0, 0]):
        new.copy_(_ints(lens))
        graph.replay()
        oracle.cache.resize(c.caches, c.tables, c.lens, c.counts, lens)
        oracle.cache.fork(c.caches, c.tables, c.lens, c.counts, [0, 1], [2, 3])
        c.same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    oracle.cache.resize(c.caches, c.tables, c.lens, c.counts, [1, 2, 3, 4])
    api.mtp_cache_resize(*c.dev, _ints([1, 2, 3, 4]), status=c.status, stream=side)
    side.synchronize()
    c.same()
