"""The usual rotary frequencies, plain and scaled for long contexts, as numbers for api.mtp_rope_freqs.

Worked out once when a model is loaded, in Python floats (64 bits).
"""
from __future__ import annotations

import math
from typing import List, Tuple


def inv_freq(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
             original_length: int = 4096, fast: float = 32.0, slow: float = 1.0,
             mscale: float = None) -> Tuple[List[float], float]:
    """(radians a position for each of rot_dim / 2 pairs, the factor on sines and cosines).

    Pair i turns base^(-2i / rot_dim) radians a position.  For contexts ``factor`` times as long as
    ``original_length``, the length that the model was trained with, ``scaling`` is one of

    * "none";
    * "linear": all positions interpolated, every frequency divided by factor;
    * "ntk": a larger base, base * factor^(d / (d - 2)), which leaves the fastest pair alone and
      divides the slowest one's frequency by factor;
    * "parts": pairs that turn at least ``fast`` times within the original length are left alone, those
      that turn at most ``slow`` times are divided by factor, and between the two the share goes linearly
      with the pair's number (the method published as YaRN); the factor on sines and cosines is
      0.1 ln(factor) + 1 unless ``mscale`` is given;
    * "bands": the same with the share going linearly with the number of turns, and a factor of 1.
    """
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1, factor 1 or more")
    half = rot_dim // 2
    plain = [base ** (-2.0 * i / rot_dim) for i in range(half)]
    given = 1.0 if mscale is None else float(mscale)
    if scaling == "none":
        return plain, given
    if scaling == "linear":
        return [f / factor for f in plain], given
    if scaling == "ntk":
        if rot_dim == 2:
            return plain, given
        wider = base * factor ** (rot_dim / (rot_dim - 2.0))
        return [wider ** (-2.0 * i / rot_dim) for i in range(half)], given
    if scaling not in ("parts", "bands"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not fast > slow > 0.0 or original_length <= 0:
        raise ValueError("fast must be above slow, slow and original_length above 0")

    def pair_of(turns: float) -> float:       # the pair (not a whole one) that turns so often
        return half * math.log(original_length / (2.0 * math.pi * turns)) / math.log(base)

    # (the upper border may lie behind the last pair, half - 1: then no pair is slow enough for the whole factor)
    first, last = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), rot_dim - 1)
    out = []
    for i, f in enumerate(plain):
        if scaling == "parts":
            keep = 1.0 - min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
        else:
            turns = original_length * f / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
        out.append(f * keep + f / factor * (1.0 - keep))
    if scaling == "parts" and mscale is None:
        given = 0.1 * math.log(factor) + 1.0
    return out, given
