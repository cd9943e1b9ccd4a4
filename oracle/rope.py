"""Rotary positions, and where new tokens go in a paged cache, in float64.  Plain definitions, shared with
no code of the product."""
from __future__ import annotations

import numpy as np


def rotate(x, positions, inv_freq, mscale=1.0, interleaved=False):
    """x [tokens, heads, dim]: the first 2 * len(inv_freq) elements of every head, turned pair by pair."""
    out = np.array(x, dtype=np.float64)
    pairs = len(inv_freq)
    for t, m in enumerate(positions):
        for i, f in enumerate(inv_freq):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
            c, s = mscale * np.cos(float(m) * f), mscale * np.sin(float(m) * f)
            xa, xb = x[t, :, a].astype(np.float64), x[t, :, b].astype(np.float64)
            out[t, :, a] = xa * c - xb * s
            out[t, :, b] = xb * c + xa * s
    return out


def clipped(x, descale):
    """What a code stands for before its rounding."""
    return np.clip(np.asarray(x, np.float64) / descale, -448.0, 448.0)


def half_step(x):
    """Half the distance of two neighbouring e4m3 values around x."""
    exponent = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    return 2.0 ** (exponent - 4)


def places(block_tables, seq_lens, cu_seqlens_q, total):
    """Per row (page, row in the page), or None where it belongs to no sequence."""
    out = [None] * total
    for b, length in enumerate(seq_lens):
        q0, q1 = int(cu_seqlens_q[b]), int(cu_seqlens_q[b + 1])
        for t in range(q0, q1):
            at = int(length) - (q1 - t)
            out[t] = (int(block_tables[b, at // 16]), at % 16)
    return out
