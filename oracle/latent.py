"""Latent attention over a paged e4m3 cache in float64: keys of 576 whose first 512 are the values.  A plain
definition, shared with no code of the product."""
from __future__ import annotations

import numpy as np

from .formats import E4M3_TABLE


def latent_attention(q, codes, block_tables, seq_lens, cu_seqlens_q, masks, descale, softmax_scale):
    """(out, weight, flat, reach) of q [total, heads, 576] float64, codes [pages, 16, 576]: the attention;
    sum_j p_j |V_j| beside it (the scale of a relative error of the weights); the largest p times
    sum_j |V_j| (the scale of an absolute one); and per row the largest sum of |terms| of a visible
    key's logit with each |q| put at the row's largest (the scale of what rounding q does).  masks: a word
    per row, or None (a chain)."""
    total, heads, _ = q.shape
    out, weight = np.zeros((total, heads, 512)), np.zeros((total, heads, 512))
    flat, reach = np.zeros((total, heads, 512)), np.zeros((total, heads, 1))
    for b, length in enumerate(int(x) for x in seq_lens):
        q0, q1 = int(cu_seqlens_q[b]), int(cu_seqlens_q[b + 1])
        n = q1 - q0
        at = np.arange(length)
        keys = E4M3_TABLE[codes[block_tables[b, at // 16], at % 16]] * descale
        for i in range(n):
            word = (2 << i) - 1 if masks is None else int(masks[q0 + i])
            see = [j for j in range(length) if j < length - n or (word >> (j - length + n)) & 1]
            if not see:
                continue
            K = keys[see]
            V = K[:, :512]
            for h in range(heads):
                row = q[q0 + i, h]
                with np.errstate(invalid="ignore"):
                    s = softmax_scale * (K @ row)
                    e = np.exp(s - s.max())
                    e /= e.sum()
                    out[q0 + i, h] = e @ V
                    weight[q0 + i, h] = e @ np.abs(V)
                    flat[q0 + i, h] = e.max() * np.abs(V).sum(0)
                    reach[q0 + i, h] = abs(softmax_scale) * np.abs(row).max() * np.abs(K).sum(1).max()
    return out, weight, flat, reach
