"""The cache's upkeep at the limits of its arguments."""
from __future__ import annotations

import pytest
import torch

from paged_fp8_speculative_gb300 import api
from tests.test_cache_pages_gpu import Pair

pytestmark = pytest.mark.gpu

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
