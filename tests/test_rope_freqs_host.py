"""mtp_rope_freqs against exact arithmetic: the nearest whole number of 2^-64 turns, as its header says."""
from __future__ import annotations

import random
from fractions import Fraction

from paged_fp8_speculative_gb300 import api

# 1 / (2 pi) to 60 digits
TURN = Fraction("0.159154943091895335768883763372514362034459645740456448747667")


def test_freqs_are_the_nearest():
    """Frequencies of all sizes and the usual ones; half a unit, and 2^-19 of one for the sum's own rounding."""
    rng = random.Random(1)
    values = [rng.uniform(0.1, 2.0) * 10.0 ** rng.uniform(-9, 5) for _ in range(20000)]
    values += [base ** (-2.0 * i / rot) for base in (10000.0, 500000.0) for rot in (64, 128, 256) for i in range(rot // 2)]
    for value, got in zip(values, api.mtp_rope_freqs(values).tolist()):
        off = (Fraction(got) - Fraction(value) * TURN * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 2 ** 19), value
