"""Draft trees in float64: the ancestors' masks, the attention over a paged e4m3 cache, and the
verification of the drafted tokens.  Plain definitions, shared with no code of the product.

A sequence's tree has n nodes; node i > 0 hangs on parents[i] < i.  Its nodes are the last n of
the sequence's cached keys.
"""
from __future__ import annotations

import numpy as np

from .formats import E4M3_TABLE, bf16_bits_to_f64


def ancestors(parents) -> list:
    """One Python int per node: the bits of the node and of every node above it."""
    words = []
    for i, p in enumerate(parents):
        words.append((1 << i) | (words[p] if i else 0))
    return words


def tree_attention(q_bits, k_codes, v_codes, block_tables, seq_lens, cu_seqlens_q, masks, k_descale,
                   v_descale, softmax_scale, num_kv_heads):
    """(out, weight, reach): the attention; sum_j p_j |V_j| beside it (the scale of what rounding
    the probabilities does); and per row the largest sum of |terms| of a visible key's logit with
    each |q| put at the row's largest (the scale of what rounding q does)."""
    q = bf16_bits_to_f64(q_bits)
    total, hq, dim = q.shape
    page = k_codes.shape[1]
    ratio = hq // num_kv_heads
    out, weight = np.zeros(q.shape), np.zeros(q.shape)
    reach = np.zeros((total, hq))
    for b, L in enumerate(int(x) for x in seq_lens):
        q0, q1 = int(cu_seqlens_q[b]), int(cu_seqlens_q[b + 1])
        n = q1 - q0
        pos = np.arange(L)
        phys = block_tables[b, pos // page]
        see = np.ones((n, L), dtype=bool)
        for t in range(n):
            word = int(masks[q0 + t])
            for i in range(n):
                see[t, L - n + i] = bool((word >> i) & 1)
        see = np.repeat(see, ratio, axis=0)
        for h in range(num_kv_heads):
            K = E4M3_TABLE[k_codes[phys, pos % page, h]]
            V = E4M3_TABLE[v_codes[phys, pos % page, h]]
            heads = slice(h * ratio, (h + 1) * ratio)
            rows = q[q0:q1, heads].reshape(n * ratio, dim)
            with np.errstate(invalid="ignore"):
                s = softmax_scale * k_descale * (rows @ K.T)
                top = np.max(np.abs(rows), axis=1)[:, None] * np.sum(np.abs(K), axis=1)[None, :]
            s = np.where(see, s, -np.inf)
            for r in range(n * ratio):
                at = np.nonzero(see[r])[0]
                if not len(at):
                    continue
                e = np.exp(s[r, at] - np.max(s[r, at]))
                e /= e.sum()
                t, g = divmod(r, ratio)
                out[q0 + t, h * ratio + g] = v_descale * (e @ V[at])
                weight[q0 + t, h * ratio + g] = abs(v_descale) * (e @ np.abs(V[at]))
                reach[q0 + t, h * ratio + g] = abs(softmax_scale * k_descale) * np.max(top[r, at])
    return out, weight, reach


def _emit(path, tokens, last, width):
    index = np.full(width, -1, np.int32)
    said = np.full(width, -1, np.int32)
    index[:len(path)] = path
    said[:len(path)] = [tokens[i] for i in path[1:]] + [last]
    return index, len(path) - 1, said


def verify_greedy(logits, tokens, parents, max_path=64):
    """One sequence: (accept_index, accept_len, out_tokens)."""
    at, path = 0, [0]
    while True:
        row = np.asarray(logits[at], np.float64)
        known = np.nonzero(~np.isnan(row))[0]
        last = int(known[np.argmax(row[known])]) if len(known) else -1
        nxt = [i for i in range(1, len(tokens)) if parents[i] == at and tokens[i] == last]
        if last < 0 or not nxt or len(path) == max_path:
            return _emit(path, tokens, last, max_path)
        at = nxt[0]
        path.append(at)


def verify_sample(p, q, tokens, parents, u, max_path=64):
    """One sequence by rejection sampling, all in float64; q may be None."""
    clean = lambda x: np.clip(np.nan_to_num(np.asarray(x, np.float64), nan=0.0), 0.0, 1.0)
    u = np.clip(np.nan_to_num(np.asarray(u, np.float64), nan=0.0), 0.0, 1.0 - 2.0 ** -24)
    at, path = 0, [0]
    vocab = np.asarray(p).shape[1]
    while True:
        w = clean(p[at])
        drafter = None if q is None else clean(q[at])
        mass, taken = 1.0, None
        if len(path) < max_path:
            for i in range(1, len(tokens)):
                if parents[i] != at:
                    continue
                x = int(tokens[i])
                known = 0 <= x < vocab
                qx = 1.0 if drafter is None else (drafter[x] if known else 0.0)
                if known and u[i] * qx * mass < w[x]:
                    taken = i
                    break
                if drafter is not None:
                    w = np.maximum(w - mass * drafter, 0.0)
                    mass = w.sum()
                elif known:
                    mass -= w[x]
                    w[x] = 0.0
        if taken is None:
            if not w.sum() > 0:
                w = clean(p[at])
            run = np.cumsum(w)
            over = np.nonzero(run > u[0] * run[-1])[0]
            return _emit(path, tokens, int(over[0]) if len(over) else -1, max_path)
        at = taken
        path.append(at)
