"""Tree attention over sequences that are cut into pieces: what a row sees in a piece of no weight is
not lost."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_fp8_speculative_gb300 import api
from tests.test_tree_attn_gpu import KD, NAN_CODE, Batch


@pytest.mark.gpu
@pytest.mark.parametrize("lens,nodes", [([20011], [8]), ([60000, 50], [16, 3]), ([700], [8]), ([120], [8])],
                         ids=["cut", "long", "short", "whole"])
def test_a_nan_in_a_piece_of_no_weight_is_seen(lens, nodes):
    """One key takes all the weight: the others' lies 2^-200 below it, 0 in 32 bits.  A NaN that stands
    in the values of one of them is the row's all the same, in its own dims, wherever the pieces end;
    a row that does not see it (a node of the tree) is left as it is."""
    batch = Batch(lens, nodes, 1, 4, seed=3, poison=False)
    n, tree = lens[0], lens[0] - nodes[0]
    batch.q.zero_()
    batch.q[:, :, 0] = 1.0
    batch.k[:] = 0
    at = lambda j: (batch.bt[0, j // 16], j % 16)
    top = n // 2
    batch.k[(*at(top), 0, 0)] = 0x7E               # 448
    args = batch.device()
    args["softmax_scale"] = 200 * np.log(2.0) / (448 * KD)
    want = api.mtp_tree_attn_fwd(**args)
    assert torch.isfinite(want).all()
    first, last = int(batch.cu[0]), int(batch.cu[1])
    for key, dims in ((0, [0, 131]), (17, [5]), (n // 3, [255]), (tree - 1, [64]), (tree + nodes[0] - 2, [7, 200])):
        v = batch.v.copy()
        v[(*at(key), 0)][dims] = NAN_CODE
        args["v_cache"] = torch.as_tensor(v).cuda()
        got = api.mtp_tree_attn_fwd(**args)
        sees = torch.zeros(got.shape[0], dtype=torch.bool, device="cuda")
        for t in range(first, last):
            sees[t] = key < tree or bool((batch.masks[t] >> (key - tree)) & 1)
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[:, :, dims] = sees[:, None, None]
        assert got[hit].isnan().all(), (key, got[hit])
        assert torch.equal(got[~hit], want[~hit])
