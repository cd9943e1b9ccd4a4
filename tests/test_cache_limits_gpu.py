"""The cache's upkeep at the limits of its arguments."""
from __future__ import annotations

import os
import subprocess
import sys
import threading

import pytest
import torch

from paged_fp8_speculative_gb300 import _lib, api
from tests.test_cache_pages_gpu import Pair

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOP = (1 << 31) - 1


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("length,bit", [(65, 8), (TOP - 16, 8), (TOP - 15, 8), (TOP - 14, 8), (TOP, 8),
                                        (7, 2), (0, 2), (-1, 2), (-TOP - 1, 2)])
def test_compact_of_lengths_that_no_table_holds(length, bit):
    """A length past the table's 64 tokens, up to the largest number, where a count of pages made by
    adding would wrap (from 2^31 - 15 on): refused, nothing of the sequence moved, its length as it was."""
    c = Pair(2, 4, 20)
    c.resize([30, 30])
    c.dev[3][0] = c.lens[0] = length
    got = api.mtp_cache_compact(*c.dev[:4], ints([0, 8, 16]), ints([[0, 3], [0, 5]]), ints([1, 1]),
                                status=c.status)
    assert c.status.item() == bit
    assert got.tolist() == [length, 24]
    for x in c.caches:                         # the other sequence's node 5 goes to its place 1
        x[:, c.tables[1, 23 // 16], 23 % 16] = x[:, c.tables[1, 27 // 16], 27 % 16]
    c.same(bit)


PLANS = """
import sys
import numpy as np
sys.path.insert(0, {root!r})
from tests.test_cache_pages_gpu import Pair

def resize(rows):
    c = Pair(rows, 1, 4096, layers=1, hkv=1, seed=rows)
    c.resize([int(x) for x in np.random.default_rng(rows).integers(0, 17, rows)])

def fork(pairs):
    c = Pair(2 * pairs, 1, 4096, layers=1, hkv=1, seed=pairs)
    c.resize([5 if b < 40 else 16 if b < pairs else 0 for b in range(2 * pairs)])
    c.fork(list(range(pairs)), list(range(pairs, 2 * pairs)))

for n in range({lo}, {hi}):
    {kind}(n)
print("plans ok")
"""


@pytest.mark.parametrize("kind,lo,hi", [("resize", 4074, 4094), ("fork", 2326, 2341)])
def test_plans_of_any_size_in_a_process_that_made_no_larger_one(kind, lo, hi):
    """A plan's shared memory passes the 48 KB that a kernel has without asking at 4078 rows (a fork's
    at 2330 pairs among 4660 rows), its static part counted; in a process of its own, where no larger
    plan has asked before.  (The fork is a kernel of its own: the resize before it asks for itself.)"""
    r = subprocess.run([sys.executable, "-c", PLANS.format(root=ROOT, kind=kind, lo=lo, hi=hi)], cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "plans ok" in r.stdout, r.stdout + r.stderr


def test_plans_of_several_threads():
    """Host threads with tables of their own, of different sizes: no call is refused."""
    lib, said = _lib.lib(), []

    def work(rows):
        stream = torch.cuda.Stream()
        cache = torch.zeros(2, 1, 16, 16, 1, 256, dtype=torch.uint8, device="cuda")
        table, lens = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda"), ints([0] * rows)
        refs, new = ints([0] * 16), ints([0] * rows)
        ws = torch.empty(api.mtp_cache_workspace_size(rows, 1), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for _ in range(4000):
            rc = lib.mtp_cache_resize(
                cache[0].data_ptr(), cache[1].data_ptr(), 1, 16 * 16 * 256, 16, 1, table.data_ptr(), 1,
                lens.data_ptr(), rows, refs.data_ptr(), new.data_ptr(), ws.data_ptr(), ws.numel(), None,
                stream.cuda_stream)
            if rc:
                said.append((rows, rc))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(rows,)) for rows in (8192, 4300, 4200, 6000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not said, (len(said), said[:3])


def test_the_largest_pool_and_table():
    """2^22 pages, the free ones at their end, and 8192 rows, all resized and half of them forked: the
    largest plan there is.  No row has a partly filled page, so the caches' contents are not touched."""
    lib, pages, rows, width = _lib.lib(), 1 << 22, 8192, 4
    cache = torch.empty(pages * 16 * 256, dtype=torch.uint8, device="cuda")     # 16 GB, K's and V's
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    lens, half = ints([0] * rows), rows // 2
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    first = pages - half * width - 5
    refs[first:] = 0
    ws = torch.empty(api.mtp_cache_workspace_size(rows, width), dtype=torch.uint8, device="cuda")
    status, stream = ints([0]), torch.cuda.current_stream().cuda_stream
    pool = (cache.data_ptr(), cache.data_ptr(), 1, pages * 16 * 256, pages, 1, table.data_ptr(), width, lens.data_ptr(), rows,
            refs.data_ptr())
    tail = (ws.data_ptr(), ws.numel(), status.data_ptr(), stream)
    new = ints([16 * width] * half + [0] * half)
    src, dst = ints(list(range(half))), ints(list(range(half, rows)))
    assert lib.mtp_cache_resize(*pool, new.data_ptr(), *tail) == 0
    assert lib.mtp_cache_fork(*pool, src.data_ptr(), dst.data_ptr(), half, *tail) == 0
    want = torch.arange(half * width, device="cuda").int().view(half, width) + first
    assert status.item() == 0
    assert torch.equal(table, torch.cat([want, want])) and (lens == 16 * width).all()
    assert (refs[first:-5] == 2).all() and (refs[-5:] == 0).all() and (refs[:first] == 1).all()
    new.zero_()
    assert lib.mtp_cache_resize(*pool, new.data_ptr(), *tail) == 0
    assert status.item() == 0 and not lens.any() and (table == -1).all() and not refs[first:].any()
