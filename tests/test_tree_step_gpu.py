"""Speculative steps with draft trees, all the operators in their turn: room for the tree, its keys
and values, the attention, the verification, the accepted path kept, the rest given back.

A toy model stands in for the target: one attention layer whose keys, values and queries are
functions of a token and its position, so that the cache after any number of steps can be
compared with the cache of the emitted tokens laid out at once.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from paged_fp8_speculative_gb300 import api, synth

pytestmark = pytest.mark.gpu

VOCAB, LAYERS, HKV, RATIO = 97, 3, 2, 4


class Toy:
    def __init__(self):
        g = torch.Generator().manual_seed(1)
        r = lambda *s: torch.randn(*s, generator=g)
        self.k = synth.quantize_e4m3(r(VOCAB, LAYERS, HKV, 256), "unit").cuda()
        self.v = synth.quantize_e4m3(r(VOCAB, LAYERS, HKV, 256), "unit").cuda()
        self.q = r(VOCAB, HKV * RATIO, 256).bfloat16().cuda()
        self.head = r(HKV * RATIO * 256, VOCAB).cuda()

    def logits(self, tokens, out):
        return out.float().reshape(len(tokens), -1) @ self.head


def put(toy, cache, tables, tokens, rows, pos):
    page = tables[rows, pos // 16].long()
    for c, table in zip(cache, (toy.k, toy.v)):
        c[:, page, pos % 16] = table[tokens].transpose(0, 1)


def held(cache, tables, b, n):
    pos = torch.arange(n, device="cuda")
    return [c[:, tables[b, pos // 16].long(), pos % 16] for c in cache]


@pytest.mark.parametrize("sampled", [False, True])
def test_steps(sampled):
    toy = Toy()
    rng = np.random.default_rng(3)
    B, pool, width = 5, 200, 30
    cache = [torch.full((LAYERS, pool, 16, HKV, 256), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tables, lens, refs = i32([[-1] * width] * B), i32([0] * B), i32([0] * pool)
    status = i32([0])
    # prompts; the last two rows are forks of the first
    prompts = [[int(x) for x in rng.integers(0, VOCAB, n)] for n in (37, 16, 150)]
    api.mtp_cache_resize(*cache, tables, lens, refs, i32([len(p) for p in prompts] + [0, 0]), status=status)
    for b, p in enumerate(prompts):
        n = len(p)
        put(toy, cache, tables, torch.tensor(p, device="cuda"), torch.full((n,), b, device="cuda"),
            torch.arange(n, device="cuda"))
    api.mtp_cache_fork(*cache, tables, lens, refs, i32([0, 0]), i32([3, 4]), status=status)
    text = prompts + [list(prompts[0]), list(prompts[0])]
    last = [int(x) for x in rng.integers(0, VOCAB, B)]           # each row's newest token, not cached yet
    scale = 0.0625
    kd = torch.ones(1, device="cuda")
    accepted = 0
    for step in range(6):
        nodes = [int(x) for x in rng.integers(1, 13, B)]
        trees = [[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)] for n in nodes]
        tokens = [[last[b]] + [0] * (n - 1) for b, n in enumerate(nodes)]
        cu = i32(np.cumsum([0] + nodes).tolist())
        parents = i32([p for t in trees for p in t])
        old = lens.tolist()
        api.mtp_cache_resize(*cache, tables, lens, refs, i32([n + m for n, m in zip(old, nodes)]), status=status)
        rows = torch.tensor([b for b, n in enumerate(nodes) for _ in range(n)], device="cuda")
        pos = torch.tensor([old[b] + i for b, n in enumerate(nodes) for i in range(n)], device="cuda")

        def attend(flat):
            put(toy, cache, tables, flat, rows, pos)
            q = toy.q[flat]
            mask = api.mtp_tree_mask(parents, cu, status=status)
            outs = [api.mtp_tree_attn_fwd(q, cache[0][layer], cache[1][layer], tables, lens, cu, mask,
                                          kd, kd, scale, status=status) for layer in range(LAYERS)]
            return toy.logits(flat, sum(o.float() for o in outs))

        # a drafter that is often right: the greedy children, found level by level
        flat = torch.tensor([t for row in tokens for t in row], device="cuda")
        for _ in range(4):
            best = attend(flat).argmax(1).tolist()
            at = 0
            for b, t in enumerate(trees):
                for i in range(1, len(t)):
                    if (i + step) % 3:
                        flat[at + i] = best[at + t[i]]
                at += len(t)
        logits = attend(flat)
        if sampled:
            p = torch.softmax(logits, -1)
            u = torch.rand(len(flat), device="cuda")
            index, count, said = api.mtp_tree_verify_sample(p, None, flat.int(), parents, cu, u, status=status)
        else:
            index, count, said = api.mtp_tree_verify_greedy(logits, flat.int(), parents, cu, status=status)
        new = api.mtp_cache_compact(*cache, tables, lens, cu, index, count, status=status)
        api.mtp_cache_resize(*cache, tables, lens, refs, new, status=status)
        assert status.item() == 0
        for b in range(B):
            n = count[b].item()
            accepted += n
            text[b] = text[b] + [last[b]] + said[b, :n].tolist()
            last[b] = said[b, n].item()
            # the cache holds the emitted tokens in their order, in pages of the row's own length
            assert lens[b].item() == len(text[b])
            want = torch.tensor(text[b], device="cuda")
            for c, table in zip(held(cache, tables, b, len(text[b])), (toy.k, toy.v)):
                assert torch.equal(c, table[want].transpose(0, 1))
            if not sampled:
                # the step's argmaxes are those of the emitted text, one token after another (a chain)
                seq = torch.tensor(text[b][-(n + 1):], device="cuda")
                chain = i32([i - 1 for i in range(n + 1)])
                one = i32([0, n + 1])
                m = api.mtp_tree_mask(chain, one)
                outs = [api.mtp_tree_attn_fwd(toy.q[seq], cache[0][la], cache[1][la], tables[b:b + 1],
                                              lens[b:b + 1], one, m, kd, kd, scale) for la in range(LAYERS)]
                again = toy.logits(seq, sum(o.float() for o in outs)).argmax(1).tolist()
                assert again == text[b][len(text[b]) - n:] + [last[b]]
    assert accepted > 10
    held_pages = torch.bincount(tables[tables >= 0].long(), minlength=pool)
    assert torch.equal(held_pages.int(), refs)
    api.mtp_cache_resize(*cache, tables, lens, refs, i32([0] * B), status=status)
    assert status.item() == 0 and not refs.any() and (tables == -1).all()
