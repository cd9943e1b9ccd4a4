"""Tree attention against the float64 oracle, where it can go wrong: tree sizes, tile and page
borders, head layouts, masks that leave nothing, NaN codes in places that are not seen, strides,
bad tables and lengths, streams and captured graphs.

Tolerance, per element (derived before the first run).  The output's rounding to bf16 is off by
at most 2^-8 |o|.  In sum_j p_j V_j a probability is off by its rounding to f16 (2^-11 p) and by
what its logit is off, d (p grows by e^d - 1, the sum by as much again: 2 d together).  A logit's
error is that of q as two e4m3 terms, 2^-17 of the row's largest |q| an element, and of 512 f32
additions, 2^-15 of the sum of |terms| at worst; both sums are at most `reach` (every |q| put at the
row's largest).  The f32 sums over n keys add about 4 sqrt(n) 2^-24.  With W = sum_j p_j |V_j|:
    |error| <= 2^-8 |o| + W (2^-11 + 2 reach (2^-17 + 2^-15) + 4 sqrt(n) 2^-24).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from paged_fp8_speculative_gb300 import api, synth

pytestmark = pytest.mark.gpu

KD, VD, SCALE = 0.75, 1.25, 0.0625 * 2
NAN_CODE = 0x7F


class Batch:
    """Sequences of `lens` tokens (trees of `nodes`), pages shuffled, unused places NaN."""

    def __init__(self, lens, nodes, hkv, ratio, seed=0, masks=None, poison=True):
        rng = np.random.default_rng(seed)
        self.lens, self.nodes, self.hkv, self.ratio = lens, nodes, hkv, ratio
        per = [-(-n // 16) for n in lens]
        pool, width = sum(per) + 3, max(per) + 1
        perm = rng.permutation(pool)
        self.bt = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.bt[b, :n] = perm[at:at + n]
            at += n
        g = torch.Generator().manual_seed(seed)
        codes = lambda: synth.quantize_e4m3(torch.randn(pool, 16, hkv, 256, generator=g), "unit").numpy()
        self.k, self.v = codes(), codes()
        if poison:                                  # behind each sequence, and in spare pages
            for b, L in enumerate(lens):
                for c in (self.k, self.v):
                    if L % 16:
                        c[self.bt[b, L // 16], L % 16:] = NAN_CODE
            for page in perm[at:]:
                self.k[page] = self.v[page] = NAN_CODE
        self.cu = np.cumsum([0] + list(nodes)).astype(np.int32)
        self.q = torch.randn(int(self.cu[-1]), hkv * ratio, 256, generator=g).bfloat16()
        if masks is None:
            masks = []
            for n in nodes:
                parents = [-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)]
                masks += oracle.tree.ancestors(parents)
        self.masks = [m - (1 << 64) if m >> 63 else m for m in masks]

    def device(self):
        d = lambda x: torch.as_tensor(x).cuda()
        return dict(q=self.q.cuda(), k_cache=d(self.k), v_cache=d(self.v), block_tables=d(self.bt),
                    seq_lens=torch.tensor(self.lens, dtype=torch.int32).cuda(), cu_seqlens_q=d(self.cu),
                    tree_mask=torch.tensor(self.masks, dtype=torch.int64).cuda(),
                    k_descale=torch.full((1,), KD).cuda(), v_descale=torch.full((1,), VD).cuda(),
                    softmax_scale=SCALE)

    def exact(self):
        return oracle.tree.tree_attention(self.q.view(torch.int16).numpy(), self.k, self.v, self.bt,
                                          self.lens, self.cu, self.masks, KD, VD, SCALE, self.hkv)


def bound(out, weight, reach, lens):
    n = max(lens)
    per = 2.0 ** -11 + 2 * reach[:, :, None] * (2.0 ** -17 + 2.0 ** -15) + 4 * np.sqrt(n) * 2.0 ** -24
    return 2.0 ** -8 * np.abs(out) + weight * per + 1e-30


def check(got, batch, rows=slice(None)):
    out, weight, reach = batch.exact()
    got = got.float().cpu().numpy().astype(np.float64)
    off = np.abs(got - out) / bound(out, weight, reach, batch.lens)
    assert np.isfinite(got[rows]).all()
    assert off[rows].max() <= 1.0, off[rows].max()


def run(batch, **more):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.mtp_tree_attn_fwd(**batch.device(), status=status, **more)
    torch.cuda.synchronize()
    assert status.item() == 0, status.item()
    return out


SHAPES = [
    ([1], [1], 1, 1),                       # the smallest call
    ([2], [1], 1, 16),
    ([64], [64], 1, 16),                    # a tree and nothing before it
    ([63], [63], 1, 1),
    ([16, 17, 15, 32], [1, 2, 3, 4], 1, 8),            # pages that end at, before, behind
    ([127, 128, 129, 130, 256, 257], [5, 7, 9, 11, 1, 64], 1, 16),
    ([200, 191, 192, 193], [64, 63, 64, 33], 2, 16),   # the tree spans two tiles
    ([300], [8], 1, 8),
    ([1000, 77, 3], [26, 40, 3], 3, 5),     # odd ratios
    ([777, 640], [13, 61], 2, 3),
    ([500, 501], [17, 64], 4, 1),
    ([450, 90], [21, 60], 1, 12),
    ([2100, 35], [9, 35], 8, 4),
    ([1300] * 40, [3] * 40, 2, 8),          # more units than SMs can hold at once
    ([7] * 200, [7] * 200, 1, 2),           # many tiny ones
    ([20011, 40], [64, 2], 1, 16),          # one long one, cut into many pieces
    ([12000] * 3, [19] * 3, 1, 7),
]


@pytest.mark.parametrize("lens,nodes,hkv,ratio", SHAPES,
                         ids=[f"{len(s[0])}x{max(s[0])}n{max(s[1])}h{s[2]}r{s[3]}" for s in SHAPES])
def test_against_the_oracle(lens, nodes, hkv, ratio):
    batch = Batch(lens, nodes, hkv, ratio, seed=len(lens) + lens[0])
    check(run(batch), batch)


@pytest.mark.parametrize("seed", range(30))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    hkv, ratio = int(rng.integers(1, 5)), int(rng.integers(1, 17))
    seqs, top = int(rng.integers(1, 12)), int(rng.integers(1, 65))
    nodes = [int(x) for x in rng.integers(1, top + 1, seqs)]
    lens = [n + int(np.exp(rng.uniform(0, np.log(3000)))) - 1 for n in nodes]
    words = [int(rng.integers(0, 1 << 63)) * 2 + int(rng.integers(0, 2)) for _ in range(sum(nodes))]
    batch = Batch(lens, nodes, hkv, ratio, seed=seed, masks=words if seed % 2 else None)
    check(run(batch), batch)


def test_masks_that_leave_nothing():
    """No key before the tree: a node with an empty word gets zeros, others only what they see; bits
    past the tree mean nothing; a node need not see itself."""
    words = [0, 1, 0b101, (1 << 63) | (1 << 5), 1 << 1] + [0] * 9
    batch = Batch([5, 9], [5, 9], 2, 4, seed=5, masks=words)
    out = run(batch)
    check(out, batch)
    assert not out[0].any() and not out[3].any() and not out[5:].any()


def test_codes_that_are_not_seen_do_not_matter():
    """NaN keys and values in nodes that a row does not see leave it as it is; rows that see them
    are NaN: every dim for a NaN key, the value's own dims for a NaN value."""
    lens, nodes = [40, 150], [6, 30]
    batch = Batch(lens, nodes, 1, 16, seed=8)
    clean = run(batch)
    page = lambda b, j: (batch.bt[b, j // 16], j % 16)
    for b, key_node, value_node in ((0, 3, 4), (1, 7, 21)):
        start = lens[b] - nodes[b]
        p, s = page(b, start + key_node)
        batch.k[p, s, 0, 17] = NAN_CODE
        p, s = page(b, start + value_node)
        batch.v[p, s, 0, 100:103] = 0xFF
    got = run(batch)
    for b, key_node, value_node in ((0, 3, 4), (1, 7, 21)):
        for t in range(nodes[b]):
            row, word = batch.cu[b] + t, batch.masks[batch.cu[b] + t]
            if (word >> key_node) & 1:
                assert got[row].isnan().all()
                continue
            dims = torch.ones(256, dtype=torch.bool, device="cuda")
            if (word >> value_node) & 1:
                assert got[row][:, 100:103].isnan().all()
                dims[100:103] = False
            assert torch.equal(got[row][:, dims], clean[row][:, dims])


def test_nan_in_a_query_stays_in_its_row():
    batch = Batch([300, 90], [12, 12], 2, 4, seed=9)
    clean = run(batch)
    batch.q[3, 5, 200] = float("nan")
    batch.q[15, 0, 0] = float("inf")
    got = run(batch)
    bad = torch.zeros(24, 8, dtype=torch.bool, device="cuda")
    bad[3, 5] = bad[15, 0] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], clean[~bad])


def test_logits_far_apart():
    """One key far above the rest: the many far below it still count (2^-20 of it each)."""
    n = 4000
    batch = Batch([n], [1], 1, 1, seed=10, poison=False)
    batch.q.zero_()
    batch.q[0, 0, 0] = 1.0
    batch.k[:] = 0
    p = batch.bt[0, 3]
    batch.k[p, 5, 0, 0] = 0x7E                     # 448, the largest code
    scale = 13.0 / (448 * KD)                      # 13 nats above the others' 0
    args = batch.device()
    args["softmax_scale"] = scale
    out = api.mtp_tree_attn_fwd(**args)
    exact, weight, reach = oracle.tree.tree_attention(
        batch.q.view(torch.int16).numpy(), batch.k, batch.v, batch.bt, batch.lens, batch.cu,
        batch.masks, KD, VD, scale, 1)
    off = np.abs(out.float().cpu().numpy() - exact) / bound(exact, weight, reach, batch.lens)
    assert off.max() <= 1.0


@pytest.mark.parametrize("scale,kd", [(0.0, 1.0), (-0.125, 0.5), (0.125, -2.0), (0.1, 0.0)])
def test_scales_of_any_sign(scale, kd):
    batch = Batch([260, 40], [9, 40], 1, 8, seed=12)
    args = batch.device()
    args["softmax_scale"], args["k_descale"] = scale, torch.full((1,), kd).cuda()
    got = api.mtp_tree_attn_fwd(**args).float().cpu().numpy()
    out, weight, reach = oracle.tree.tree_attention(
        batch.q.view(torch.int16).numpy(), batch.k, batch.v, batch.bt, batch.lens, batch.cu,
        batch.masks, kd, VD, scale, 1)
    assert (np.abs(got - out) <= bound(out, weight, reach, batch.lens)).all()


def test_queries_of_any_size():
    """Rows scaled by powers of two, the scale taken out of the softmax scale: the same bits."""
    batch = Batch([300], [10], 1, 4, seed=13)
    want = run(batch)
    for e in (-60, 60):
        args = batch.device()
        args["q"] = args["q"] * 2.0 ** e
        args["softmax_scale"] = SCALE * 2.0 ** -e
        assert torch.equal(api.mtp_tree_attn_fwd(**args), want)


def test_strides_and_places_that_are_not_ours():
    batch = Batch([300, 61], [9, 26], 2, 5, seed=14)
    want = run(batch)
    args = batch.device()
    total, hq = int(batch.cu[-1]), 10
    wide = torch.randn(total + 2, hq + 3, 264, device="cuda").bfloat16()
    wide[1:-1, 2:-1, :256] = args["q"]
    args["q"] = wide[1:-1, 2:-1, :256]
    out = torch.full((total + 4, hq + 2, 272), 7.0, dtype=torch.bfloat16, device="cuda")
    view = out[2:-2, 1:-1, 8:264]
    got = api.mtp_tree_attn_fwd(**args, out=view)
    assert torch.equal(got, want)
    view.fill_(7.0)
    assert (out == 7.0).all()


def test_rows_of_no_sequence_are_left():
    batch = Batch([100, 40], [9, 6], 1, 8, seed=15)
    args = batch.device()
    want = run(batch)
    args["q"] = torch.cat([args["q"], args["q"][:5]])
    args["tree_mask"] = torch.cat([args["tree_mask"], args["tree_mask"][:5]])
    out = torch.full_like(args["q"], 3.0)
    api.mtp_tree_attn_fwd(**args, out=out)
    assert torch.equal(out[:15], want) and (out[15:] == 3.0).all()


@pytest.mark.parametrize("what", ["page", "neg", "long", "qlen", "order", "short"])
def test_sequences_with_errors_get_zeros(what):
    lens, nodes = [100, 300, 40], [5, 9, 6]
    batch = Batch(lens, nodes, 2, 8, seed=16)
    want = run(batch)
    args = batch.device()
    bit = {"page": 4, "neg": 4, "long": 8, "qlen": 1, "order": 1, "short": 2}[what]
    known = True
    if what == "page":
        args["block_tables"][1, 18] = batch.k.shape[0]
    elif what == "neg":
        args["block_tables"][1, 0] = -1
    elif what == "long":
        args["seq_lens"][1] = 16 * batch.bt.shape[1] + 1
    elif what == "short":
        args["seq_lens"][1] = 8
    elif what == "qlen":                            # 70 nodes: more than a word
        batch = Batch([100, 300, 40], [5, 64, 6], 2, 8, seed=16)
        args = batch.device()
        want = run(batch)
        extra = 10
        args["q"] = torch.cat([args["q"][:69], args["q"][:extra], args["q"][69:]])
        args["tree_mask"] = torch.cat([args["tree_mask"][:69], args["tree_mask"][:extra],
                                       args["tree_mask"][69:]])
        args["cu_seqlens_q"][2:] += extra
        want = torch.cat([want[:5], torch.zeros_like(want[:64 + extra]), want[69:]])
    elif what == "order":
        args["cu_seqlens_q"][1] = 30                # past the third's start: two are unknown
        known = False
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(args["q"], 5.0)
    api.mtp_tree_attn_fwd(**args, out=out, status=status)
    assert status.item() & bit
    if not known:
        return
    rows = args["cu_seqlens_q"].tolist()
    assert not out[rows[1]:rows[2]].any()
    assert torch.equal(out[:rows[1]], want[:rows[1]]) and torch.equal(out[rows[2]:], want[rows[2]:])


def test_the_same_bits_again_on_any_stream_and_workspace():
    batch = Batch([9000, 500, 60], [20, 64, 3], 1, 16, seed=17)
    want = run(batch)
    args = batch.device()
    size = api.mtp_tree_attn_workspace_size(3, int(batch.cu[-1]), 16, 1, batch.bt.shape[1])
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")      # NaNs as floats
    assert torch.equal(run(batch, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [api.mtp_tree_attn_fwd(**args, stream=side) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    with pytest.raises(api.MtpAttnError):
        run(batch, workspace=ws[:size - 256])


def test_captured_and_replayed_with_other_lengths():
    """A captured call takes lengths, tables, masks and trees from their buffers at each replay."""
    first = Batch([900, 300], [20, 12], 2, 8, seed=18)
    second = Batch([350, 40], [11, 21], 2, 8, seed=19)
    buf = first.device()
    out = torch.empty_like(buf["q"])
    width, pool = buf["block_tables"].shape[1], buf["k_cache"].shape[0]
    ws = torch.empty(api.mtp_tree_attn_workspace_size(2, 32, 16, 2, width), dtype=torch.uint8,
                     device="cuda")
    api.mtp_tree_attn_fwd(**buf, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.mtp_tree_attn_fwd(**buf, out=out, workspace=ws)
    for batch in (first, second, first):
        want = run(batch)
        new = batch.device()
        for name in ("q", "seq_lens", "cu_seqlens_q", "tree_mask"):
            buf[name].copy_(new[name])
        n = min(width, new["block_tables"].shape[1])
        buf["block_tables"][:, :n] = new["block_tables"][:, :n]
        for name in ("k_cache", "v_cache"):
            buf[name][:new[name].shape[0]] = new[name]
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        if batch is second:                        # the pieces may be cut elsewhere: not the same bits
            check(out, batch)
        else:
            assert torch.equal(out, want)


def test_a_chain_agrees_with_the_verify_attention():
    b = synth.make_batch([3000, 70, 500], [4, 3, 1], 16, 1, seed=20, kv_recipe="unit").to("cuda")
    kd = torch.ones(1, device="cuda")
    want = api.mtp_verify_attn_fwd(b.q, b.k_cache, b.v_cache, b.block_tables, b.seq_lens,
                                   b.cu_seqlens_q, kd, kd, b.softmax_scale)
    parents = torch.tensor([-1, 0, 1, 2, -1, 0, 1, -1], dtype=torch.int32, device="cuda")
    mask = api.mtp_tree_mask(parents, b.cu_seqlens_q)
    got = api.mtp_tree_attn_fwd(b.q, b.k_cache, b.v_cache, b.block_tables, b.seq_lens,
                                b.cu_seqlens_q, mask, kd, kd, b.softmax_scale)
    # each is within its own bound of the exact value: 0.01 std for the verify attention
    # (half an ulp of bf16 on top of either)
    d = (got.float() - want.float()).abs()
    std = want.float().std()
    assert (d <= 0.02 * std + 2.0 ** -7 * want.float().abs()).all()


@pytest.mark.parametrize("nodes", [[1], [2, 64, 33], [5] * 100])
def test_masks_from_parents(nodes):
    rng = np.random.default_rng(21)
    trees = [[-1] + [int(rng.integers(0, i)) for i in range(1, n)] for n in nodes]
    want = [m - (1 << 64) if m >> 63 else m for t in trees for m in oracle.tree.ancestors(t)]
    parents = torch.tensor([p if i else 99 for t in trees for i, p in enumerate(t)],
                           dtype=torch.int32, device="cuda")          # the root's is not read
    cu = torch.tensor(np.cumsum([0] + nodes), dtype=torch.int32, device="cuda")
    assert api.mtp_tree_mask(parents, cu).tolist() == want


def test_masks_of_bad_parents():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    parents = torch.tensor([-1, 0, 5, 2, 0, 0], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    got = api.mtp_tree_mask(parents, cu, status=status)
    assert status.item() == api.ERR_PARENT
    assert got.tolist() == [1, 3, 4, 12, 1, 3]
