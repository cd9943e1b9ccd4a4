"""Tree attention over sequences that are cut into pieces: every key counts once, in whatever piece,
and what a row sees in a piece of no weight is not lost.

The keys of `Told` batches are told apart in the output.  K has one dim that is not 0, which goes
through SIZES by turns of 48 keys, so that logits lie within a unit and each is one product; V has a 1
in one dim only, key j's being j // ceil(L / 256).  Output dim d is then the weight of its own run of
keys, at most 469 of them, and a page of 16 keys that is left out, or counted twice, changes it by
a few percent.  (With random values an output is the mean of many that cancel: the same bound, which
goes by the values' sizes, is then half as large as the output itself, and a lost piece is within it.)

Tolerance: that of tests/test_tree_attn_gpu.py.  With one product a logit, `reach` is the row's largest
|q| (about 4) x 1.5 x SCALE x KD, 0.6, and W is the output itself: about
2^-8 + 2^-11 + 2 x 0.6 (2^-17 + 2^-15) + 4 sqrt(n) 2^-24 = 0.0045 of it.
"""
from __future__ import annotations

import functools

import numpy as np
import pytest
import torch

import oracle
from paged_fp8_speculative_gb300 import api
from tests.test_tree_attn_gpu import KD, NAN_CODE, SCALE, VD, Batch, bound, check, run

SIZES = (0.0, 1.5, -1.0, 0.5, -1.5, 1.0, -0.5)
ONE = 0x38                                         # e4m3 1.0


class Told(Batch):
    def __init__(self, lens, nodes, hkv, ratio, seed=0):
        super().__init__(lens, nodes, hkv, ratio, seed=seed, poison=False)
        steps = np.array([int(np.nonzero(oracle.E4M3_TABLE == x)[0][0]) for x in SIZES], np.uint8)
        self.k[:], self.v[:] = 0, 0
        for b, L in enumerate(lens):
            j = np.arange(L)
            page, at = self.bt[b, j // 16], j % 16
            self.k[page, at, :, 3] = steps[j // 48 % len(SIZES)][:, None]
            for h in range(hkv):
                self.v[page, at, h, j // -(-L // 256)] = ONE


# what the call makes of them: one unit over every CTA; two row tiles a unit's sequence; three long
# ones that CTAs share; long and short together; units that are cut once or not at all; two KV heads
CUT = [([120000], [9], 1, 2), ([50000, 33], [64, 33], 1, 16), ([9100, 12001, 30003], [16, 5, 11], 1, 16),
       ([20011, 40, 3000, 17], [64, 2, 7, 9], 1, 16), ([1290] * 40, [3] * 40, 2, 8),
       ([40001, 2500], [4, 20], 2, 5)]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,nodes,hkv,ratio", CUT, ids=[f"{len(c[0])}x{max(c[0])}" for c in CUT])
def test_every_key_counts_once(lens, nodes, hkv, ratio):
    batch = Told(lens, nodes, hkv, ratio, seed=len(lens))
    check(run(batch), batch)


@functools.lru_cache
def told_one():
    """One long sequence: (batch, oracle's output, bound)."""
    batch = Told([120000], [2], 1, 2, seed=1)
    out, weight, reach = batch.exact()
    return batch, out, bound(out, weight, reach, batch.lens)


@pytest.mark.parametrize("first,count,times", [(0, 768, 0), (5376, 768, 0), (119296, 704, 0), (768, 768, 2),
                                               (64000, 128, 0), (64000, 128, 2), (31999 * 2, 16, 0), (31999 * 2, 16, 2)])
def test_the_bound_notices_keys_left_out_or_counted_twice(first, count, times):
    """A piece of 768 keys, a key tile, a page: the oracle's own sum without them, or with them twice."""
    batch, out, limit = told_one()
    L = batch.lens[0]
    q = batch.q.double().numpy()[:, :, 3]          # K's dim
    s = SCALE * KD * q[:, :, None] * np.array(SIZES)[np.arange(L) // 48 % len(SIZES)]
    e = np.exp(s)
    e[:, :, L - 2:] *= np.array([[1, 0], [1, 1]])[:, None, :]            # the root does not see its child
    mine = np.arange(L) // -(-L // 256)
    sums = lambda w: VD * np.stack([np.bincount(mine, r, minlength=256) for r in w.reshape(-1, L)]).reshape(2, 2, 256) / \
        w.sum(-1, keepdims=True)
    assert (np.abs(sums(e) - out) <= 1e-9).all()   # the same definition
    e[:, :, first:first + count] *= times
    off = np.abs(sums(e) - out) / limit
    assert off.max() > (2.0 if count > 16 else 1.2), off.max()


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


@pytest.mark.gpu
def test_sequences_whose_places_are_not_in_order():
    """cu_seqlens_q 0, 30, 14, 20 of 20 rows: the first two sequences' rows are not known and not
    written; the third's are the attention of that sequence."""
    batch = Batch([100, 300, 40], [5, 9, 6], 2, 8, seed=16)
    args = batch.device()
    args["cu_seqlens_q"][1] = 30
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(args["q"], 5.0)
    api.mtp_tree_attn_fwd(**args, out=out, status=status)
    assert status.item() == api.ERR_QLEN
    assert (out[:14] == 5.0).all()
    exact, weight, reach = (x[14:] for x in batch.exact())
    off = np.abs(out[14:].float().cpu().numpy() - exact) / bound(exact, weight, reach, batch.lens)
    assert off.max() <= 1.0
