"""A whole step with draft trees as one captured graph: room for the trees, their keys and values,
masks, attention, verification, the accepted paths kept, the rest given back.  Replayed with other
trees, tokens and numbers each time, beside the same calls made eagerly on a cache of their own: all
that they leave is equal, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_fp8_speculative_gb300 import api, synth

pytestmark = pytest.mark.gpu

VOCAB, LAYERS, HKV, RATIO, ROWS, NODES = 3, 2, 2, 4, 5, 40


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Serving:
    """The buffers of a program that serves ROWS sequences, NODES tree nodes a step in all."""

    def __init__(self):
        g = torch.Generator().manual_seed(1)
        r = lambda *s: torch.randn(*s, generator=g)
        codes = lambda: synth.quantize_e4m3(r(VOCAB, LAYERS, HKV, 256), "unit").cuda()
        self.kv = [codes(), codes()]
        self.q, self.head = r(VOCAB, HKV * RATIO, 256).bfloat16().cuda(), r(HKV * RATIO * 256, VOCAB).cuda()
        pool, width = 120, 40
        self.cache = [torch.zeros(LAYERS, pool, 16, HKV, 256, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.tables, self.lens, self.refs = i32([[-1] * width] * ROWS), i32([0] * ROWS), i32([0] * pool)
        self.status = i32([0])
        self.tokens, self.parents, self.cu = i32([0] * NODES), i32([0] * NODES), i32([0] * (ROWS + 1))
        self.row, self.node = i32([0] * NODES).long(), i32([0] * NODES).long()
        self.u = torch.zeros(NODES, device="cuda")
        self.one = torch.ones(1, device="cuda")
        api.mtp_cache_resize(*self.cache, self.tables, self.lens, self.refs, i32([37, 16, 150, 0, 0]), status=self.status)
        api.mtp_cache_fork(*self.cache, self.tables, self.lens, self.refs, i32([0, 0]), i32([3, 4]), status=self.status)

    def load(self, tokens, trees, u):
        nodes = [len(t) for t in trees]
        self.tokens.copy_(i32(tokens))
        self.parents.copy_(i32([p for t in trees for p in t]))
        self.cu.copy_(i32(np.cumsum([0] + nodes).tolist()))
        self.row.copy_(i32([b for b, n in enumerate(nodes) for _ in range(n)]))
        self.node.copy_(i32([i for n in nodes for i in range(n)]))
        self.u.copy_(torch.tensor(u, dtype=torch.float32))

    def step(self, sampled):
        c, pool = self.cache, (*self.cache, self.tables, self.lens, self.refs)
        pos = self.lens.long()[self.row] + self.node
        api.mtp_cache_resize(*pool, self.lens + self.cu[1:] - self.cu[:-1], status=self.status)
        page = self.tables[self.row, pos // 16].long()
        for x, table in zip(c, self.kv):
            x[:, page, pos % 16] = table[self.tokens.long()].transpose(0, 1)
        mask = api.mtp_tree_mask(self.parents, self.cu, status=self.status)
        outs = [api.mtp_tree_attn_fwd(self.q[self.tokens.long()], c[0][la], c[1][la], self.tables, self.lens, self.cu, mask,
                                      self.one, self.one, 0.0625, status=self.status) for la in range(LAYERS)]
        hidden = sum(o.float() for o in outs).reshape(NODES, -1)
        logits = (hidden[:, :, None] * self.head).sum(1)
        if sampled:
            said = api.mtp_tree_verify_sample(torch.softmax(logits, -1), None, self.tokens, self.parents, self.cu, self.u,
                                              status=self.status)
        else:
            said = api.mtp_tree_verify_greedy(logits, self.tokens, self.parents, self.cu, status=self.status)
        kept = api.mtp_cache_compact(*c, self.tables, self.lens, self.cu, *said[:2], status=self.status)
        api.mtp_cache_resize(*pool, kept, status=self.status)
        return [*outs, logits, *said, kept]

    def all(self):
        return [*self.cache, self.tables, self.lens, self.refs, self.status]


@pytest.mark.parametrize("sampled", [False, True])
def test_a_captured_step_is_the_eager_one(sampled):
    rng = np.random.default_rng(5)
    eager, graph = Serving(), Serving()

    def inputs():
        nodes = [1] * ROWS
        for b in rng.integers(0, ROWS, NODES - ROWS):
            nodes[b] += 1
        trees = [[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)] for n in nodes]
        return [int(x) for x in rng.integers(0, VOCAB, NODES)], trees, rng.random(NODES)

    first = inputs()                               # a step before the capture: torch's own set-up
    for serving in (eager, graph):
        serving.load(*first)
        serving.step(sampled)
    torch.cuda.synchronize()
    captured = torch.cuda.CUDAGraph()
    with torch.cuda.graph(captured):
        got = graph.step(sampled)
    accepted = 0
    for _ in range(8):
        x = inputs()
        eager.load(*x)
        graph.load(*x)
        want = eager.step(sampled)
        captured.replay()
        torch.cuda.synchronize()
        assert graph.status.item() == 0
        for a, b in zip([*got, *graph.all()], [*want, *eager.all()]):
            assert torch.equal(a, b)
        accepted += int(want[LAYERS + 2].sum())    # accept_len
    assert accepted > 20
