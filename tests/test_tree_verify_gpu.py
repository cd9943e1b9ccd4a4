"""Verification of drafted tokens against the float64 oracle: whole numbers, so equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from paged_fp8_speculative_gb300 import api

pytestmark = pytest.mark.gpu

def trees_of(nodes, rng, back=4):
    return [[-1] + [int(rng.integers(max(0, (i - 1) // back - 1), (i - 1) // back + 1))
                    for i in range(1, n)] for n in nodes]


def packed(trees, tokens):
    cu = torch.tensor(np.cumsum([0] + [len(t) for t in trees]), dtype=torch.int32, device="cuda")
    par = torch.tensor([p for t in trees for p in t], dtype=torch.int32, device="cuda")
    return torch.tensor(tokens, dtype=torch.int32, device="cuda"), par, cu


def expect(rows, trees, tokens, max_path, fn):
    at, out = 0, []
    for t in trees:
        out.append(fn(at, at + len(t), tokens[at:at + len(t)], t, max_path))
        at += len(t)
    return out


def same(got, want):
    index, count, said = (x.cpu().numpy() for x in got)
    for b, (i, n, s) in enumerate(want):
        assert count[b] == n and np.array_equal(index[b], i) and np.array_equal(said[b], s), \
            (b, index[b][:8], i[:8], said[b][:8], s[:8])


def greedy(logits, trees, tokens, max_path=64, **more):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.mtp_tree_verify_greedy(logits, *packed(trees, tokens), max_path, status=status, **more)
    host = logits.float().cpu().numpy()
    same(got, expect(host, trees, tokens, max_path,
                     lambda a, z, tok, par, w: oracle.tree.verify_greedy(host[a:z], tok, par, w)))
    return status.item()


def walkable(logits, trees, rng, vocab):
    """Tokens of which about two in three are their parents' argmax."""
    tokens, at = [], 0
    best = logits.float().argmax(1).tolist()
    for t in trees:
        for p in t:
            tokens.append(best[at + max(p, 0)] if rng.random() < 0.65 else int(rng.integers(vocab)))
        at += len(t)
    return tokens


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab,nodes", [(1, [1, 2]), (2, [5]), (31, [64, 1, 7]), (1000, [3] * 70),
                                         (4099, [20, 33]), (50257, [8]), (20000, [5] * 160),
                                         (1 << 20, [2, 1])])
def test_greedy(dtype, vocab, nodes):
    rng = np.random.default_rng(vocab + len(nodes))
    g = torch.Generator(device="cuda").manual_seed(vocab)
    logits = torch.randn(sum(nodes), vocab, generator=g, device="cuda").to(dtype)
    trees = trees_of(nodes, rng)
    assert greedy(logits, trees, walkable(logits, trees, rng, vocab)) == 0


@pytest.mark.parametrize("max_path", [1, 2, 5, 64])
def test_greedy_paths_end_at_max_path(max_path):
    rng = np.random.default_rng(3)
    logits = torch.randn(64 + 9, 777, device="cuda")
    trees = [[i - 1 for i in range(64)], [i - 1 for i in range(9)]]
    best = logits.argmax(1).tolist()
    tokens = [0] + best[:63] + [0] + best[64:72]
    assert greedy(logits, trees, tokens, max_path) == 0


def test_greedy_ties_zeros_infinities_and_nan():
    V = 5000
    z = torch.full((8, V), -1.0, device="cuda")
    z[0, 4000] = z[0, 17] = z[0, 3999] = 2.0            # ties: the lowest
    z[1] = float("-inf")                                # all alike: token 0
    z[2, :] = 0.0
    z[2, ::2] = -0.0                                    # zeros of both signs are alike
    z[3] = float("nan")
    z[3, 4999] = -5.0                                   # the only number
    z[4, 9], z[4, 8] = float("inf"), float("nan")
    z[5] = float("nan")                                 # nothing to choose from
    z[6, 1] = 3e38
    trees = [[-1]] * 5 + [[-1, 0]] + [[-1]]
    status = greedy(z, trees, [0] * 8)
    assert status == api.ERR_ROW
    got = api.mtp_tree_verify_greedy(z, *packed(trees, [0] * 8))
    assert [int(x) for x in got[2][:, 0]] == [17, 0, 0, 4999, 9, -1, 0]


def test_greedy_first_of_equal_children_and_tokens_outside():
    z = torch.zeros(6, 100, device="cuda")
    z[0, 42] = z[3, 7] = 1
    greedy(z, [[-1, 0, 0, 0, 3, 3]], [0, 41, 100, 42, -1, 7])
    greedy(z, [[-1, 0, 0, 0, 1, 3]], [0, 1 << 30, 42, 42, -5, 7])


def test_rows_with_strides():
    rng = np.random.default_rng(5)
    wide = torch.randn(21, 3003, device="cuda").bfloat16()
    logits = wide[:, 1:2999]                            # rows at odd addresses
    trees = trees_of([10, 11], rng)
    greedy(logits, trees, walkable(logits, trees, rng, logits.shape[1]))


def sample(p, q, trees, tokens, u, max_path=64, **more):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.mtp_tree_verify_sample(p, q, *packed(trees, tokens), u, max_path, status=status, **more)
    hp = p.float().cpu().numpy()
    hq = None if q is None else q.float().cpu().numpy()
    hu = u.cpu().numpy()
    same(got, expect(hp, trees, tokens, max_path,
                     lambda a, z, tok, par, w: oracle.tree.verify_sample(
                         hp[a:z], None if hq is None else hq[a:z], tok, par, hu[a:z], w)))
    return status.item(), got


def draw(nodes, vocab, seed, spread=3.0, dtype=torch.float32, back=4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    trees = trees_of(nodes, rng, back)
    n = sum(nodes)
    z = torch.randn(n, vocab, generator=g, device="cuda") * spread
    p = torch.softmax(z, -1)
    q = torch.softmax(z + torch.randn(n, vocab, generator=g, device="cuda"), -1)
    up, at = [], 0
    for t in trees:
        up += [at + max(x, 0) for x in t]
        at += len(t)
    tokens = torch.multinomial(q[torch.tensor(up, device="cuda")], 1, generator=g)[:, 0].tolist()
    u = torch.rand(n, generator=g, device="cuda")
    return p.to(dtype), q.to(dtype), trees, tokens, u


@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab,nodes", [(1, [1, 3]), (2, [9, 4]), (33, [64, 1, 7]), (1024, [30] * 20),
                                         (1025, [12] * 30), (4099, [20, 33]), (32000, [4, 26, 1]),
                                         (9000, [5] * 160)])
def test_sample(vocab, nodes, dtype, drafter):
    p, q, trees, tokens, u = draw(nodes, vocab, vocab + len(nodes), dtype=dtype)
    assert sample(p, q if drafter else None, trees, tokens, u)[0] == 0


@pytest.mark.parametrize("seed", range(20))
def test_sample_random(seed):
    """Flat and peaked rows, wide trees whose nodes refuse many children."""
    rng = np.random.default_rng(seed)
    nodes = [int(x) for x in rng.integers(1, 65, int(rng.integers(1, 20)))]
    p, q, trees, tokens, u = draw(nodes, int(np.exp(rng.uniform(1, 10))), seed,
                                  spread=float(rng.uniform(0.01, 6)), back=int(rng.choice([1, 4, 63])))
    assert sample(p, q if seed % 3 else None, trees, tokens, u)[0] == 0


def test_sample_the_largest_vocabulary():
    p, q, trees, tokens, u = draw([3, 2], 1 << 20, 9, spread=0.5)
    assert sample(p, q, trees, tokens, u)[0] == 0


@pytest.mark.parametrize("max_path", [1, 3])
def test_sample_paths_end_at_max_path(max_path):
    p, _, trees, tokens, u = draw([9, 9, 9], 500, 10, back=1)
    assert sample(p, p.clone(), trees, tokens, u, max_path)[0] == 0      # p = q: all are accepted


def test_sample_p_equal_to_q_accepts_the_whole_chain():
    p, _, _, _, u = draw([20], 300, 11)
    tree = [[i - 1 for i in range(20)]]
    tokens = [0] + torch.multinomial(p[:19], 1)[:, 0].tolist()
    _, got = sample(p, p.clone(), tree, tokens, u)
    assert got[1].item() == 19


def test_sample_edges():
    V = 2100
    p = torch.zeros(8, V, device="cuda")
    p[0, 2099] = 1.0                                     # all mass on the last token
    p[1, 5] = p[1, 1500] = 0.5
    p[2, 7] = 1.0
    p[4] = float("nan")
    p[4, 3] = 0.25                                       # NaN is nothing
    p[5, 9], p[5, 10] = 5.0, -3.0                        # taken into [0, 1]
    p[6] = 1.0 / V
    p[7] = 1.0 / V
    trees = [[-1]] * 8
    u = torch.tensor([0.99999994, 0.5, 0.0, 0.3, 0.7, 0.2, 1.0, float("nan")], device="cuda")
    status, got = sample(p, None, trees, [0] * 8, u)
    assert status == api.ERR_ROW                         # row 3 has no mass
    assert [int(x) for x in got[2][:, 0]] == [2099, 1500, 7, -1, 3, 9, 2099, 0]


def test_sample_a_residual_without_mass_falls_back_to_the_target():
    # p <= q everywhere (q does not sum to 1): a refusal leaves nothing, p itself is drawn from
    p = torch.full((2, 64), 1 / 64, device="cuda")
    q = torch.full((2, 64), 1 / 32, device="cuda")
    u = torch.tensor([0.4, 0.9], device="cuda")
    status, got = sample(p, q, [[-1, 0]], [0, 3], u)
    assert status == 0 and got[1].item() == 0 and got[2][0, 0].item() == int(0.4 * 64)


def test_sample_the_same_token_twice_and_tokens_outside():
    p, q, _, _, _ = draw([6], 400, 12)
    for u in torch.rand(20, 6, device="cuda"):
        sample(p, q, [[-1, 0, 0, 0, 0, 0]], [0, 7, 7, -3, 400, 9], u)
        sample(p, None, [[-1, 0, 0, 0, 0, 0]], [0, 7, 7, -3, 400, 9], u)


@pytest.mark.parametrize("nodes,parents", [([4], [-1, 0, 2, 1]), ([4], [-1, 0, -1, 1]), ([3], [-1, 0, 7])])
def test_bad_trees_are_refused_on_the_device(nodes, parents):
    z = torch.randn(6, 50, device="cuda")
    cu = torch.tensor([0, nodes[0], 6], dtype=torch.int32, device="cuda")
    par = torch.tensor(parents + [i - 1 for i in range(6 - nodes[0])], dtype=torch.int32, device="cuda")
    tok = torch.zeros(6, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    index, count, said = api.mtp_tree_verify_greedy(z, tok, par, cu, 4, status=status)
    assert status.item() == api.ERR_PARENT
    assert count[0].item() == -1 and (index[0] == -1).all() and (said[0] == -1).all()
    assert said[1, 0].item() >= 0 and count[1].item() >= 0


@pytest.mark.parametrize("cu", [[0, 0, 6], [0, 7, 6], [-1, 3, 6], [0, 66, 70]])
def test_bad_lengths_are_refused_on_the_device(cu):
    n = max(6, cu[2])
    p = torch.softmax(torch.randn(n, 50, device="cuda"), -1)
    par = torch.tensor([max(i - 1, 0) if i < 6 else 0 for i in range(n)], dtype=torch.int32, device="cuda")
    tok = torch.zeros(n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, count, _ = api.mtp_tree_verify_sample(p, None, tok, par,
                                             torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                             torch.rand(n, device="cuda"), status=status)
    assert status.item() & api.ERR_QLEN and -1 in count.tolist()


def test_streams_graphs_and_given_outputs():
    p, q, trees, tokens, u = draw([12, 7, 30], 3001, 13)
    tok, par, cu = packed(trees, tokens)
    want = api.mtp_tree_verify_sample(p, q, tok, par, cu, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.mtp_tree_verify_sample(p, q, tok, par, cu, u, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.empty_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.mtp_tree_verify_sample(p, q, tok, par, cu, u, 64, *outs)
    for seed in (14, 15):
        new = draw([12, 7, 30], 3001, seed)
        p.copy_(new[0])
        q.copy_(new[1])
        u.copy_(new[4])
        tok.copy_(torch.tensor(new[3], dtype=torch.int32))
        par.copy_(packed(new[2], new[3])[1])
        graph.replay()
        want = api.mtp_tree_verify_sample(p, q, tok, par, cu, u)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
