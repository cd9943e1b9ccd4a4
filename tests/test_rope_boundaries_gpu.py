"""Appending with cu_seqlens_q out of order: the status tells of every kind, rows that one sequence alone claims are
written where they belong, and nothing else is."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_fp8_speculative_gb300 import api
from tests.test_rope_gpu import Batch

pytestmark = pytest.mark.gpu

ORDERS = [[0, 10, 5, 15], [0, 5, 10, 99], [-3, 5, 10, 15], [7, 5, 10, 15], [0, -9, 99, 15], [0, 5, 3, 15], [12, 9, 4, 1],
          [0, 15, 0, 15], [5, 5, 2, 2], [0, 16, 16, 16], [0, 5, 10, -1]]


def claims(cu, total):
    """Per row the sequence that alone claims it, or None."""
    own = [[] for _ in range(total)]
    for b, (q0, q1) in enumerate(zip(cu, cu[1:])):
        if 0 <= q0 <= q1 <= total:
            for t in range(q0, q1):
                own[t].append(b)
    return [x[0] if len(x) == 1 else None for x in own]


def expected_rows(cu, lens, table, total):
    place = {}
    for t, b in enumerate(claims(cu, total)):
        if b is not None:
            at = lens[b] - (cu[b + 1] - t)
            place[t] = int(table[b, at // 16]) * 16 + at % 16
    return place


@pytest.mark.parametrize("cu", ORDERS)
def test_append(cu):
    b = Batch([20, 20, 20], [5, 5, 5], 2, 1, 16)
    b.run()
    assert b.status.item() == 0
    rows, good_k = b.kc.view(-1, 256), b.kc.clone().view(-1, 256)
    good_v, good_q = b.vc.clone().view(-1, 256), b.out.clone()
    codes = {}                                           # a token's codes, wherever it goes
    for t, at in expected_rows([0, 5, 10, 15], b.lens, b.bt, 15).items():
        codes[t] = (good_k[at].clone(), good_v[at].clone())
    b.kc.fill_(0x55), b.vc.fill_(0x56), b.out.fill_(9.0)
    b.cu.copy_(torch.tensor(cu))
    b.run()
    assert b.status.item() == api.ERR_QLEN
    place = expected_rows(cu, b.lens, b.bt, 15)
    want_k, want_v = torch.full_like(rows, 0x55), torch.full_like(rows, 0x56)
    for t, at in place.items():
        want_k[at], want_v[at] = codes[t]
    assert torch.equal(rows, want_k) and torch.equal(b.vc.view(-1, 256), want_v)
    for t in range(15):
        assert torch.equal(b.out[t], good_q[t]) if t in place else (b.out[t] == 9.0).all(), t


@pytest.mark.parametrize("cu", ORDERS)
def test_latent_append(cu):
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(15, 576, generator=g, device="cuda").bfloat16()
    q = torch.randn(15, 3, 64, generator=g, device="cuda").bfloat16()
    pos = torch.arange(15, dtype=torch.int32, device="cuda")
    freqs = api.mtp_rope_freqs([1.0 / (i + 1) for i in range(32)], device="cuda")
    table = torch.tensor([[3, 0], [5, 2], [1, 4]], dtype=torch.int32, device="cuda")
    lens = torch.full((3,), 20, dtype=torch.int32, device="cuda")

    def run(bounds):
        cache = torch.full((6, 16, 576), 0x55, dtype=torch.uint8, device="cuda")
        out, status = torch.full_like(q, 9.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        api.mtp_rope_latent_append(q, x[:, :512], x[:, 512:], pos, freqs, cache, table, lens,
                                   torch.tensor(bounds, dtype=torch.int32, device="cuda"), 0.02, q_out=out, status=status)
        torch.cuda.synchronize()
        return cache.view(-1, 576), out, status.item()

    good, good_q, status = run([0, 5, 10, 15])
    assert status == 0
    codes = {t: good[at].clone() for t, at in expected_rows([0, 5, 10, 15], [20] * 3, table.cpu(), 15).items()}
    got, out, status = run(cu)
    assert status == api.ERR_QLEN
    place = expected_rows(cu, [20] * 3, table.cpu(), 15)
    want = torch.full_like(got, 0x55)
    for t, at in place.items():
        want[at] = codes[t]
    assert torch.equal(got, want)
    for t in range(15):
        assert torch.equal(out[t], good_q[t]) if t in place else (out[t] == 9.0).all(), t


@pytest.mark.parametrize("count,wrong", [(40, 33), (700, 5), (700, 699), (1500, 1200)])
def test_many_sequences(count, wrong):
    """One boundary of many goes back behind the one ahead of it, so that two sequences claim the row between them."""
    b = Batch([9] * count, [2] * count, 1, 1, 16, seed=count)
    b.run()
    assert b.status.item() == 0
    good = b.kc.clone()
    b.kc.fill_(0x55), b.vc.fill_(0x56), b.out.fill_(9.0)
    b.cu[wrong] = 2 * wrong - 3                          # (the one ahead: 2 wrong - 2)
    cu = b.cu.tolist()
    b.run()
    assert b.status.item() == api.ERR_QLEN
    known = np.array([x is not None for x in claims(cu, b.total)])
    assert known.sum() == b.total - 1 and not known[2 * wrong - 3]
    assert np.array_equal((b.out != 9.0).any(-1).any(-1).cpu().numpy(), known)
    for s in (0, wrong - 3, wrong, wrong + 1, count - 1):
        if s < count:
            page = int(b.bt[s, 0])
            assert torch.equal(b.kc[page, 7:9], good[page, 7:9]), s
