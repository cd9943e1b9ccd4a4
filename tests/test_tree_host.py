"""Host-only tests of the draft-tree and cache entry points: refusals before any launch, empty
batches, workspace sizes, the binding's own checks."""
from __future__ import annotations

import pytest
import torch

from paged_fp8_speculative_gb300 import _lib, api

FAKE = 0x10000


def call(name, order, good, **over):
    a = dict(good)
    for k in over:
        assert k in a, k
    a.update(over)
    return getattr(_lib.lib(), name)(*[a[k] for k in order.split()])


ATTN = ("q q_st q_sh k v pages bt max_pages sl cu mask seqs total hq hkv kd vd scale ws ws_bytes out "
        "o_st o_sh status stream")
ATTN_GOOD = dict(q=FAKE, q_st=24 * 256, q_sh=256, k=FAKE, v=FAKE, pages=10, bt=FAKE, max_pages=5,
                 sl=FAKE, cu=FAKE, mask=FAKE, seqs=2, total=90, hq=24, hkv=2, kd=FAKE, vd=FAKE,
                 scale=0.0625, ws=FAKE, ws_bytes=1 << 40, out=FAKE, o_st=24 * 256, o_sh=256,
                 status=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), api.E_ARG), (dict(k=None), api.E_ARG), (dict(mask=None), api.E_ARG),
    (dict(bt=None), api.E_ARG), (dict(out=None), api.E_ARG), (dict(vd=None), api.E_ARG),
    (dict(seqs=-1), api.E_ARG), (dict(total=1), api.E_ARG), (dict(pages=0), api.E_ARG),
    (dict(max_pages=0), api.E_ARG), (dict(q_sh=100), api.E_ARG), (dict(o_st=0), api.E_ARG),
    (dict(q=FAKE + 8), api.E_ARG), (dict(mask=FAKE + 4), api.E_ARG),
    (dict(scale=float("inf")), api.E_ARG), (dict(hkv=0), api.E_ARG),
    (dict(hq=34, hkv=2), api.E_UNSUPPORTED),          # ratio 17
    (dict(hq=25, hkv=2), api.E_UNSUPPORTED),          # not a multiple
    (dict(total=129), api.E_UNSUPPORTED),             # a tree of more than 64 nodes somewhere
    (dict(pages=1 << 32), api.E_UNSUPPORTED),
])
def test_tree_attn_refusals(over, code):
    assert call("mtp_tree_attn_fwd", ATTN, ATTN_GOOD, **over) == code


VERIFY = "rows dtype stride vocab tok par cu seqs total width index count said status stream"
VERIFY_GOOD = dict(rows=FAKE, dtype=0, stride=100, vocab=100, tok=FAKE, par=FAKE, cu=FAKE, seqs=2,
                   total=9, width=64, index=FAKE, count=FAKE, said=FAKE, status=None, stream=None)
SAMPLE = "rows stride q q_stride dtype vocab tok par cu u seqs total width index count said status stream"
SAMPLE_GOOD = dict(VERIFY_GOOD, q=FAKE, q_stride=100, u=FAKE)

COMMON = [
    (dict(rows=None), api.E_ARG), (dict(tok=None), api.E_ARG), (dict(par=None), api.E_ARG),
    (dict(cu=None), api.E_ARG), (dict(index=None), api.E_ARG), (dict(count=None), api.E_ARG),
    (dict(said=None), api.E_ARG), (dict(vocab=0), api.E_ARG), (dict(stride=99), api.E_ARG),
    (dict(width=0), api.E_ARG), (dict(seqs=-1), api.E_ARG), (dict(total=1), api.E_ARG),
    (dict(rows=FAKE + 2), api.E_ARG), (dict(tok=FAKE + 2), api.E_ARG),
    (dict(dtype=3), api.E_UNSUPPORTED), (dict(width=65), api.E_UNSUPPORTED),
    (dict(total=129), api.E_UNSUPPORTED),
    (dict(vocab=(1 << 20) + 1, stride=1 << 21), api.E_UNSUPPORTED),
]


@pytest.mark.parametrize("over,code", COMMON)
def test_verify_refusals(over, code):
    assert call("mtp_tree_verify_greedy", VERIFY, VERIFY_GOOD, **over) == code
    assert call("mtp_tree_verify_sample", SAMPLE, SAMPLE_GOOD, **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(u=None), api.E_ARG), (dict(u=FAKE + 1), api.E_ARG), (dict(q_stride=99), api.E_ARG),
    (dict(q=FAKE + 1), api.E_ARG),
])
def test_sample_refusals(over, code):
    assert call("mtp_tree_verify_sample", SAMPLE, SAMPLE_GOOD, **over) == code


MASK = "par cu seqs total mask status stream"
MASK_GOOD = dict(par=FAKE, cu=FAKE, seqs=2, total=9, mask=FAKE, status=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(par=None), api.E_ARG), (dict(mask=None), api.E_ARG), (dict(mask=FAKE + 4), api.E_ARG),
    (dict(total=1), api.E_ARG), (dict(total=129), api.E_UNSUPPORTED),
])
def test_mask_refusals(over, code):
    assert call("mtp_tree_mask", MASK, MASK_GOOD, **over) == code


CACHE = "k v layers stride pages hkv "
CACHE_GOOD = dict(k=FAKE, v=FAKE, layers=2, stride=10 * 16 * 256, pages=10, hkv=1)
RESIZE = CACHE + "bt max_pages sl rows ref new ws ws_bytes status stream"
RESIZE_GOOD = dict(CACHE_GOOD, bt=FAKE, max_pages=4, sl=FAKE, rows=3, ref=FAKE, new=FAKE + 64, ws=FAKE,
                   ws_bytes=1 << 20, status=None, stream=None)
FORK = CACHE + "bt max_pages sl rows ref src dst pairs ws ws_bytes status stream"
FORK_GOOD = dict(CACHE_GOOD, bt=FAKE, max_pages=4, sl=FAKE, rows=3, ref=FAKE, src=FAKE, dst=FAKE,
                 pairs=2, ws=FAKE, ws_bytes=1 << 20, status=None, stream=None)
COPY = CACHE + "src dst pairs status stream"
COPY_GOOD = dict(CACHE_GOOD, src=FAKE, dst=FAKE, pairs=2, status=None, stream=None)
COMPACT = CACHE + "bt max_pages sl cu seqs total index count width new status stream"
COMPACT_GOOD = dict(CACHE_GOOD, bt=FAKE, max_pages=4, sl=FAKE, cu=FAKE, seqs=2, total=9, index=FAKE,
                    count=FAKE, width=8, new=FAKE + 64, status=None, stream=None)
CALLS = {"mtp_cache_resize": (RESIZE, RESIZE_GOOD), "mtp_cache_fork": (FORK, FORK_GOOD),
         "mtp_cache_copy_pages": (COPY, COPY_GOOD), "mtp_cache_compact": (COMPACT, COMPACT_GOOD)}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("over,code", [
    (dict(k=None), api.E_ARG), (dict(v=None), api.E_ARG), (dict(layers=0), api.E_ARG),
    (dict(pages=0), api.E_ARG), (dict(hkv=0), api.E_ARG), (dict(k=FAKE + 8), api.E_ARG),
    (dict(stride=10 * 16 * 256 - 16), api.E_ARG),     # layers overlap
    (dict(stride=10 * 16 * 256 + 8), api.E_ARG),
    (dict(pages=1 << 32, stride=1 << 45), api.E_UNSUPPORTED),
])
def test_cache_refusals(name, over, code):
    assert call(name, *CALLS[name], **over) == code


@pytest.mark.parametrize("name,over,code", [
    ("mtp_cache_resize", dict(bt=None), api.E_ARG), ("mtp_cache_resize", dict(ref=None), api.E_ARG),
    ("mtp_cache_resize", dict(new=None), api.E_ARG),
    ("mtp_cache_resize", dict(new=FAKE), api.E_ARG),             # seq_lens itself
    ("mtp_cache_resize", dict(rows=8193), api.E_UNSUPPORTED),
    ("mtp_cache_resize", dict(pages=(1 << 22) + 1), api.E_UNSUPPORTED),
    ("mtp_cache_resize", dict(ws=None), api.E_WORKSPACE),
    ("mtp_cache_resize", dict(ws=FAKE + 16), api.E_WORKSPACE),
    ("mtp_cache_resize", dict(ws_bytes=16), api.E_WORKSPACE),
    ("mtp_cache_fork", dict(src=None), api.E_ARG), ("mtp_cache_fork", dict(dst=FAKE + 2), api.E_ARG),
    ("mtp_cache_fork", dict(pairs=4), api.E_ARG), ("mtp_cache_fork", dict(pairs=-1), api.E_ARG),
    ("mtp_cache_fork", dict(ws=None), api.E_WORKSPACE),
    ("mtp_cache_copy_pages", dict(src=None), api.E_ARG),
    ("mtp_cache_copy_pages", dict(pairs=-1), api.E_ARG),
    ("mtp_cache_compact", dict(index=None), api.E_ARG),
    ("mtp_cache_compact", dict(new=FAKE), api.E_ARG),
    ("mtp_cache_compact", dict(width=0), api.E_ARG),
    ("mtp_cache_compact", dict(width=65), api.E_UNSUPPORTED),
    ("mtp_cache_compact", dict(total=1), api.E_ARG),
    ("mtp_cache_compact", dict(max_pages=0), api.E_ARG),
])
def test_cache_refusals_of_one_call(name, over, code):
    assert call(name, *CALLS[name], **over) == code


def test_empty_calls_are_no_ops():
    assert call("mtp_tree_attn_fwd", ATTN, ATTN_GOOD, seqs=0, total=0) == api.OK
    assert call("mtp_tree_verify_greedy", VERIFY, VERIFY_GOOD, seqs=0, total=0) == api.OK
    assert call("mtp_tree_verify_sample", SAMPLE, SAMPLE_GOOD, seqs=0, total=0) == api.OK
    assert call("mtp_tree_mask", MASK, MASK_GOOD, seqs=0, total=0) == api.OK
    assert call("mtp_cache_resize", RESIZE, RESIZE_GOOD, rows=0) == api.OK
    assert call("mtp_cache_fork", FORK, FORK_GOOD, pairs=0) == api.OK
    assert call("mtp_cache_copy_pages", COPY, COPY_GOOD, pairs=0) == api.OK
    assert call("mtp_cache_compact", COMPACT, COMPACT_GOOD, seqs=0, total=0) == api.OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_no_device_is_reported():
    assert call("mtp_tree_attn_fwd", ATTN, ATTN_GOOD) == api.E_DEVICE
    assert call("mtp_tree_verify_greedy", VERIFY, VERIFY_GOOD) == api.E_DEVICE
    assert call("mtp_tree_verify_sample", SAMPLE, SAMPLE_GOOD) == api.E_DEVICE
    assert call("mtp_tree_mask", MASK, MASK_GOOD) == api.E_DEVICE
    for name in CALLS:
        assert call(name, *CALLS[name]) == api.E_DEVICE


def test_workspace_sizes():
    f = api.mtp_cache_workspace_size
    assert f(0, 0) >= 0 and f(100, 7) >= 100 * 8 and f(8192, 7) >= 8192 * 8
    assert f(-1, 7) == 0 and f(8193, 7) == 0 and f(4, -1) == 0
    g = api.mtp_tree_attn_workspace_size
    assert g(2, 9, 24, 0, 5) == 0 and g(2, 9, 25, 2, 5) == 0 and g(-1, 9, 24, 2, 5) == 0


def test_binding_checks():
    cpu = dict(dtype=torch.int32)
    cu, par = torch.tensor([0, 3], **cpu), torch.tensor([-1, 0, 0], **cpu)
    rows = torch.zeros(3, 10)
    with pytest.raises(ValueError, match="parents"):
        api.mtp_tree_mask(par.long(), cu)
    with pytest.raises(ValueError, match="out"):
        api.mtp_tree_mask(par, cu, out=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="draft_tokens"):
        api.mtp_tree_verify_greedy(rows, par[:2], par, cu)
    with pytest.raises(ValueError, match="logits"):
        api.mtp_tree_verify_greedy(rows.double(), par, par, cu)
    with pytest.raises(ValueError, match="logits"):
        api.mtp_tree_verify_greedy(rows.T.contiguous().T, par, par, cu)
    with pytest.raises(ValueError, match="draft_probs"):
        api.mtp_tree_verify_sample(rows, rows[:, :9], par, par, cu, torch.zeros(3))
    with pytest.raises(ValueError, match="uniforms"):
        api.mtp_tree_verify_sample(rows, None, par, par, cu, torch.zeros(2))
    with pytest.raises(ValueError, match="accept_index"):
        api.mtp_tree_verify_greedy(rows, par, par, cu, max_path=4,
                                   accept_index=torch.zeros(1, 5, **cpu))
    kv = torch.zeros(2, 4, 16, 1, 256, dtype=torch.uint8)
    bt, sl, ref = torch.zeros(3, 2, **cpu), torch.zeros(3, **cpu), torch.zeros(4, **cpu)
    with pytest.raises(ValueError, match="k_cache"):
        api.mtp_cache_copy_pages(kv[..., :128], kv[..., :128], par, par)
    with pytest.raises(ValueError, match="contiguous"):
        api.mtp_cache_copy_pages(kv.transpose(1, 2).contiguous().transpose(1, 2),
                                 kv.transpose(1, 2).contiguous().transpose(1, 2), par, par)
    with pytest.raises(ValueError, match="ref_counts"):
        api.mtp_cache_resize(kv, kv, bt, sl, ref[:3], sl)
    with pytest.raises(ValueError, match="new_lens"):
        api.mtp_cache_resize(kv, kv, bt, sl, ref, sl[:2])
    with pytest.raises(ValueError, match="dst"):
        api.mtp_cache_fork(kv, kv, bt, sl, ref, par, par[:2])
    with pytest.raises(ValueError, match="cu_seqlens_q"):
        api.mtp_cache_compact(kv, kv, bt, sl, cu, bt, sl)
    q = torch.zeros(3, 8, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="tree_mask"):
        api.mtp_tree_attn_fwd(q, kv[0], kv[0], bt[:1], sl[:1], cu, torch.zeros(2, dtype=torch.int64),
                              1.0, 1.0, 0.0625)
