"""Latent attention with logits far down float32's range, whole and joined from pieces: the largest decides, also
where a piece has nothing that a row sees."""
from __future__ import annotations

import pytest
import torch

from tests.test_latent_gpu import Batch
from tests.test_latent_range_gpu import SHAPES, alike

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,nodes,heads,width", SHAPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_inside_the_range(lens, nodes, heads, width, sign):
    """Up to 1e38: the key with the largest one has all the weight, so far apart are they."""
    b = Batch(lens, [nodes] * len(lens), heads, seed=3, width=width)
    alike(b)
    b.scale = 1.0
    at = 70 if lens[0] > 100 else 3
    b.cache[b.bt[0, at // 16].long(), at % 16, 512] = 0x38 + 8 if sign > 0 else 0x38 - 8    # 2.0, 0.5
    b.q[0, :, 512] = sign * 6e37
    out = b.run()
    value = b.cache[b.bt[0, at // 16].long(), at % 16, :512].view(torch.float8_e4m3fn).double() * 0.75
    assert torch.allclose(out[0].double(), value.expand(heads, -1), rtol=2.0 ** -7, atol=0)
    assert torch.isfinite(out).all() and b.status.item() == 0


def test_a_piece_that_a_row_does_not_see():
    """64 new tokens that make a tile of their own, which is the last piece (205 tiles, 4 units of 16 rows taken together
    by groups of 4 of 152 CTAs: pieces of 6 places, 211 = 35 x 6 + 1), and rows that see none of them."""
    b = Batch([204 * 128 + 64], [64], 1, seed=5, masks=[0] * 32 + [1 << i for i in range(32, 64)])
    alike(b)
    b.scale = 1.0
    b.q[..., 512] = -1e33
    at = 1000
    b.cache[b.bt[0, at // 16].long(), at % 16, 512] = 0x30     # 0.5
    out = b.run()
    value = b.cache[b.bt[0, at // 16].long(), at % 16, :512].view(torch.float8_e4m3fn).double() * 0.75
    assert torch.allclose(out.double(), value.expand(64, 1, -1), rtol=2.0 ** -7, atol=0)
    assert b.status.item() == 0
