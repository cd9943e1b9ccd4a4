"""What the verification calls make for their caller."""
from __future__ import annotations

import pytest
import torch

from paged_fp8_speculative_gb300 import api
from tests.test_tree_verify_gpu import packed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("side", [False, True])
def test_outputs_are_tensors_of_their_own(sampled, side):
    """Each has a storage of its own size: one that is kept keeps no other, and one that grows in place
    runs into no other."""
    rows = torch.softmax(torch.randn(9, 100, device="cuda"), -1)
    tree = packed([[-1, 0, 1, 1], [-1], [-1, 0, 0, 0]], [3] * 9)
    more = {"stream": torch.cuda.Stream()} if side else {}
    torch.cuda.synchronize()
    got = api.mtp_tree_verify_sample(rows, None, *tree, torch.rand(9, device="cuda"), **more) if sampled else \
        api.mtp_tree_verify_greedy(rows, *tree, **more)
    torch.cuda.synchronize()
    assert [tuple(x.shape) for x in got] == [(3, 64), (3,), (3, 64)]
    for x in got:
        assert x.storage_offset() == 0 and x.untyped_storage().nbytes() == x.numel() * 4
    want = [x.clone() for x in got]
    for i in range(3):
        got[i].resize_(1000).fill_(-7)
        for j in range(i + 1, 3):
            assert torch.equal(got[j], want[j])
