"""rope.inv_freq(scaling="parts") where the slowest pair of all turns more than `slow` times within the original
length, so that the border between the shares lies behind the last pair."""
from __future__ import annotations

import math

import pytest

from paged_fp8_speculative_gb300 import rope


def test_hand_worked_shares():
    """rot_dim 64, base 10000, 131072 positions: the pair that turns 32 times is number 32 ln(131072 / (64 pi)) /
    ln 10000 = 22.5, the one that turns once 34.6; so the shares go from 1 at 22 to 0 at 35, in steps of 1/13."""
    plain, _ = rope.inv_freq(64)
    got, _ = rope.inv_freq(64, scaling="parts", factor=4.0, original_length=131072)
    for pair, keep in ((21, 1.0), (22, 1.0), (23, 12 / 13), (25, 10 / 13), (28, 7 / 13), (31, 4 / 13)):
        assert got[pair] == pytest.approx(plain[pair] * (keep + (1.0 - keep) / 4.0), rel=1e-12), pair


@pytest.mark.parametrize("rot_dim,length,factor", [(64, 65536, 40.0), (64, 131072, 4.0), (128, 65536, 8.0), (128, 131072, 32.0),
                                                   (256, 131072, 16.0), (64, 4096, 40.0)])
def test_the_rule(rot_dim, length, factor):
    """Pairs that turn `fast` times are left alone, those that turn at most `slow` times divided by the factor, and
    from the last pair that turns more than `fast` times on the share falls by the same amount from pair to pair."""
    plain, _ = rope.inv_freq(rot_dim)
    got, _ = rope.inv_freq(rot_dim, scaling="parts", factor=factor, original_length=length)
    share = [(a / b - 1.0 / factor) / (1.0 - 1.0 / factor) for a, b in zip(got, plain)]
    turns = [length * f / (2.0 * math.pi) for f in plain]
    for s, n in zip(share, turns):
        if n >= 32.0:
            assert s == pytest.approx(1.0, abs=1e-12)
        elif n <= 1.0:
            assert s == pytest.approx(0.0, abs=1e-12)
        else:
            assert 0.0 < s < 1.0
    between = [i for i, n in enumerate(turns) if 1.0 < n < 32.0]
    falls = [share[i - 1] - share[i] for i in between]
    # the borders are whole pairs on either side of the two that the rule names
    pairs = rot_dim // 2 * math.log(32.0) / math.log(10000.0)
    assert all(f == pytest.approx(falls[0], rel=1e-9) for f in falls[1:])
    assert 1.0 / (pairs + 2.0) <= falls[-1] <= 1.0 / pairs
