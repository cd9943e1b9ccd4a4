"""What the verification calls make for their caller, and what a caller sees where no memory is left."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from paged_fp8_speculative_gb300 import api
from tests.test_tree_verify_gpu import packed

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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

NO_MEMORY = """
import sys
import torch
sys.path.insert(0, {root!r})
from paged_fp8_speculative_gb300 import api
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
torch.cuda.set_per_process_memory_fraction((600 << 20) / torch.cuda.get_device_properties(0).total_memory)
n = 625                                             # trees of 64 nodes: q has 328 MB, and so has the output
q = torch.empty(64 * n, 16, 256, dtype=torch.bfloat16, device="cuda")
kv = torch.zeros(4, 16, 1, 256, dtype=torch.uint8, device="cuda")
args = (q, kv, kv, i32([[0, 1, 2, 3]] * n), i32([64] * n), i32([64 * b for b in range(n + 1)]),
        torch.zeros(64 * n, dtype=torch.int64, device="cuda"), torch.ones(1, device="cuda"), torch.ones(1, device="cuda"), 0.1)
try:
    api.mtp_tree_attn_fwd(*args)
except torch.OutOfMemoryError as e:
    print("no memory:", str(e)[:60])
q.zero_()
out = api.mtp_tree_attn_fwd(*args, out=q)           # and the next call is as ever: no node sees a key
torch.cuda.synchronize()
assert not out.any()
print("carried on")
"""


def test_no_memory_is_told_by_torchs_own_error():
    r = subprocess.run([sys.executable, "-c", NO_MEMORY.format(root=ROOT)], cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "no memory:" in r.stdout and "carried on" in r.stdout, r.stdout + r.stderr
