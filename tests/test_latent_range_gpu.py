"""Latent attention where logits pass the ends of float32's range: the row is NaN, as the header
says, whichever end it is, and other rows keep their bits."""
from __future__ import annotations

import pytest
import torch

from paged_fp8_speculative_gb300 import api
from tests.test_latent_gpu import Batch

pytestmark = pytest.mark.gpu


def alike(b):
    """Keys with 1.0 in the first rotated dim and nothing else in their rotated part; q only there."""
    b.cache[..., 512:] = 0
    b.cache[..., 512] = 0x38
    b.q.zero_()


SHAPES = [([300, 40], 2, 16, 0), ([20000], 1, 16, 0), ([9000, 9000], 1, 128, 0), ([300, 129], 3, 10, 20000), ([2000], 4, 8, 20000)]


@pytest.mark.parametrize("lens,nodes,heads,width", SHAPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_all_logits_leave_the_range(lens, nodes, heads, width, sign):
    b = Batch(lens, [nodes] * len(lens), heads, seed=1, width=width)
    alike(b)
    b.q[..., 512] = 1.0
    clean = b.run()
    assert torch.isfinite(clean).all()
    b.scale = 100.0                                      # 100 x 0.75 x 3e37 is beyond 3.4e38
    clean = b.run()
    b.q[0, heads // 2, 512] = sign * 3e37
    out = b.run()
    assert torch.isnan(out[0, heads // 2]).all()
    out[0, heads // 2] = clean[0, heads // 2]
    assert torch.equal(out, clean) and b.status.item() == 0


@pytest.mark.parametrize("lens,nodes,heads,width", SHAPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("late", [False, True])
def test_one_logit_leaves_the_range(lens, nodes, heads, width, sign, late):
    """One key of all, the first or the last that all rows see; unseen, it is nothing."""
    b = Batch(lens, [nodes] * len(lens), heads, seed=2, width=width)
    alike(b)
    b.scale = 100.0
    b.q[..., 512] = 1e-3
    b.cache[..., 513] = 0
    at = lens[0] - nodes if late else 0                  # (row 0 is token 0, which sees that far)
    b.cache[b.bt[0, at // 16].long(), at % 16, 513] = 0x38
    clean = b.run()
    b.q[0, 0, 513] = sign * 3e37
    out = b.run()
    assert torch.isnan(out[0, 0]).all()
    out[0, 0] = clean[0, 0]
    assert torch.equal(out, clean)
    if nodes > 1:                                        # the key after it, which row 0 does not see
        page = b.bt[0, (lens[0] - 1) // 16].long()
        b.cache[..., 513] = 0
        b.cache[page, (lens[0] - 1) % 16, 513] = 0x38
        assert torch.equal(b.run(), clean)


def test_rows_that_see_nothing_stay_zeros():
    b = Batch([3, 200], [3, 3], 16, masks=[0, 4, 1, 0, 7, 1])
    alike(b)
    b.scale = 100.0
    b.q[..., 512] = -3e37
    out = b.run()
    assert not out[0].any()
    assert torch.isnan(out[1:3]).all() and torch.isnan(out[3:]).all()
