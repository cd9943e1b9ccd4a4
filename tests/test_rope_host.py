"""Rotary frequencies and the refusals of the rotary, appending and latent attention calls, on the CPU."""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import pytest
import torch

from paged_fp8_speculative_gb300 import api, rope
from paged_fp8_speculative_gb300._lib import SIGNATURES, lib

FAKE = 1 << 40

# 1 / (2 pi) to 60 digits
TURN = Fraction("0.159154943091895335768883763372514362034459645740456448747667")


def freqs(values):
    return [x % (1 << 64) for x in api.mtp_rope_freqs(values).tolist()]


@pytest.mark.parametrize("value", [0.0, 1.0, 0.1, 1e-4, 3e-7, 1e-12, 2 * math.pi, 6.0, 100.25, 2.0 ** 20,
                                   math.nextafter(2 * math.pi, 0), 1e-300])
def test_freqs_are_turns_rounded(value):
    """Within one unit of 2^-64 turns plus the double's product error, 2^-104 of the value."""
    want = Fraction(value) * TURN * 2 ** 64
    got = freqs([value])[0]
    off = abs(Fraction(got) - want % 2 ** 64)
    off = min(off, 2 ** 64 - off)
    assert off <= 2 + want / 2 ** 100


def test_freqs_order_and_tensors():
    values = [10000.0 ** (-2 * i / 64) for i in range(32)]
    got = freqs(values)
    assert got == freqs(torch.tensor(values, dtype=torch.float64))
    assert got == sorted(got, reverse=True) and api.mtp_rope_freqs([]).shape == (0,)


@pytest.mark.parametrize("value", [-1.0, math.nan, math.inf, 2.0 ** 20 + 1])
def test_freqs_refusals(value):
    with pytest.raises(ValueError):
        api.mtp_rope_freqs([1.0, value])


def test_angles_of_far_positions():
    """position * freq modulo 2^64 against exact arithmetic, to the largest 32-bit position."""
    for f in (1.0, 0.37, 1e-3):
        unit = freqs([f])[0]
        for m in (1, 77, 131071, 10 ** 6, 2 ** 31 - 1, -1, -2 ** 31):
            turns = Fraction((m * unit) % 2 ** 64, 2 ** 64)
            want = (m * Fraction(f) * TURN) % 1
            off = abs(turns - want)
            assert min(off, 1 - off) <= Fraction(abs(m) * 3, 2 ** 64)


def test_inv_freq_plain_and_linear():
    f, s = rope.inv_freq(64)
    assert len(f) == 32 and f[0] == 1.0 and s == 1.0 and f[31] == pytest.approx(10000.0 ** (-62 / 64), rel=1e-15)
    g, _ = rope.inv_freq(64, scaling="linear", factor=4.0)
    assert all(a == b / 4 for a, b in zip(g, f))


def test_inv_freq_ntk_ends():
    f, _ = rope.inv_freq(128)
    g, _ = rope.inv_freq(128, scaling="ntk", factor=8.0)
    assert g[0] == f[0] and g[-1] == pytest.approx(f[-1] / 8.0, rel=1e-12)
    assert rope.inv_freq(2, scaling="ntk", factor=8.0)[0] == [1.0]


@pytest.mark.parametrize("scaling", ["parts", "bands"])
def test_inv_freq_in_parts(scaling):
    f, _ = rope.inv_freq(64)
    g, s = rope.inv_freq(64, scaling=scaling, factor=40.0)
    for a, b in zip(g, f):
        turns = 4096 * b / (2 * math.pi)
        assert b / 40.0 <= a * (1 + 1e-12) and a <= b * (1 + 1e-12)
        if turns > 60:
            assert a == b
        if turns < 0.5:
            assert a == pytest.approx(b / 40.0, rel=1e-12)
    assert s == (pytest.approx(0.1 * math.log(40.0) + 1.0) if scaling == "parts" else 1.0)
    assert rope.inv_freq(64, scaling=scaling, factor=40.0, mscale=1.25)[1] == 1.25


@pytest.mark.parametrize("bad", [dict(rot_dim=0), dict(rot_dim=7), dict(base=1.0), dict(factor=0.5),
                                 dict(scaling="other"), dict(scaling="parts", fast=1.0, slow=1.0),
                                 dict(scaling="bands", original_length=0)])
def test_inv_freq_refusals(bad):
    with pytest.raises(ValueError):
        rope.inv_freq(**{**dict(rot_dim=64), **bad})


# ---- the C entry points' refusals (pointers that are never followed) -------------------------------

NAMES = {
    "mtp_rope_append": "q qt qh k kt kh v vt vh dtype pos freqs rot il ms kc vc pages bt width lens cu seqs total hq hkv "
                       "kd vd out ot oh status stream".split(),
    "mtp_rope_latent_append": "q qt qh c ct r rt dtype pos freqs il ms cache pages bt width lens cu seqs total heads d "
                              "out ot oh status stream".split(),
    "mtp_rope_prefill": "q qt qh k kt kh r rt v vt vh dtype pos freqs il ms total hq hkv qd kd vd q8 k8 v8 stream".split(),
    "mtp_latent_attn_fwd": "q qt qh cache pages bt width lens cu mask seqs total heads d scale ws wsb out ot oh status "
                           "stream".split(),
}
GOOD = {
    "mtp_rope_append": dict(q=FAKE, qt=4096, qh=256, k=FAKE, kt=256, kh=256, v=FAKE, vt=256, vh=256, dtype=1, pos=FAKE,
                            freqs=FAKE, rot=64, il=0, ms=1.0, kc=FAKE, vc=FAKE + 4096, pages=4, bt=FAKE, width=2,
                            lens=FAKE, cu=FAKE, seqs=2, total=3, hq=16, hkv=1, kd=FAKE, vd=FAKE, out=FAKE + (1 << 20),
                            ot=4096, oh=256, status=None, stream=None),
    "mtp_rope_latent_append": dict(q=FAKE, qt=1024, qh=64, c=FAKE, ct=512, r=FAKE, rt=64, dtype=1, pos=FAKE, freqs=FAKE,
                                   il=1, ms=1.0, cache=FAKE, pages=4, bt=FAKE, width=2, lens=FAKE, cu=FAKE, seqs=2,
                                   total=3, heads=16, d=FAKE, out=FAKE + (1 << 20), ot=9216, oh=576, status=None,
                                   stream=None),
    "mtp_rope_prefill": dict(q=FAKE, qt=384, qh=192, k=FAKE, kt=256, kh=128, r=FAKE, rt=64, v=FAKE, vt=256, vh=128,
                             dtype=1, pos=FAKE, freqs=FAKE, il=1, ms=1.0, total=3, hq=2, hkv=2, qd=FAKE, kd=FAKE,
                             vd=FAKE, q8=FAKE, k8=FAKE, v8=FAKE, stream=None),
    "mtp_latent_attn_fwd": dict(q=FAKE, qt=9216, qh=576, cache=FAKE, pages=4, bt=FAKE, width=2, lens=FAKE, cu=FAKE,
                                mask=None, seqs=2, total=3, heads=16, d=FAKE, scale=0.1, ws=FAKE, wsb=1 << 40, out=FAKE,
                                ot=8192, oh=512, status=None, stream=None),
}


def call(name, **over):
    args = {**GOOD[name], **over}
    assert list(GOOD[name]) == NAMES[name] and len(NAMES[name]) == len(SIGNATURES[name][1])
    return getattr(lib(), name)(*[args[k] for k in NAMES[name]])


REFUSED = {
    "mtp_rope_append": [
        dict(seqs=-1), dict(total=-1), dict(hkv=0), dict(hq=-1), dict(rot=-16), dict(dtype=3), dict(ms=math.inf),
        dict(ms=math.nan), dict(seqs=0), dict(q=None), dict(hq=0), dict(freqs=None), dict(kc=None), dict(vc=None),
        dict(vc=FAKE), dict(pos=None), dict(kd=None), dict(vd=None), dict(bt=None), dict(lens=None), dict(cu=None),
        dict(pages=0), dict(width=0), dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(kt=0), dict(kh=-256),
        dict(vt=257), dict(qt=4), dict(out=None), dict(out=FAKE + 8), dict(oh=4), dict(out=FAKE, ot=8192),
        dict(out=FAKE, dtype=2), dict(out=FAKE, oh=512), dict(pos=FAKE + 2), dict(freqs=FAKE + 4), dict(kd=FAKE + 1),
        dict(status=FAKE + 2), dict(cu=FAKE + 2), dict(kc=FAKE + 8)],
    "mtp_rope_latent_append": [
        dict(seqs=-1), dict(total=-1), dict(heads=-1), dict(dtype=-1), dict(ms=math.nan), dict(seqs=0), dict(q=None),
        dict(heads=0), dict(freqs=None), dict(cache=None), dict(pos=None), dict(d=None), dict(bt=None), dict(lens=None),
        dict(cu=None), dict(pages=0), dict(width=0), dict(c=None), dict(r=None), dict(c=FAKE + 8), dict(ct=510),
        dict(rt=0), dict(rt=60), dict(out=None), dict(out=FAKE), dict(out=FAKE + 8), dict(cache=FAKE + 8),
        dict(freqs=FAKE + 4), dict(d=FAKE + 2), dict(qt=0)],
    "mtp_rope_prefill": [
        dict(total=-1), dict(hq=0), dict(hkv=0), dict(dtype=9), dict(ms=math.inf), dict(pos=None), dict(freqs=None),
        dict(qd=None), dict(kd=None), dict(vd=None), dict(q8=None), dict(k8=None), dict(v8=None), dict(q=None),
        dict(k=None), dict(r=None), dict(v=None), dict(qt=4), dict(kh=0), dict(rt=12), dict(vt=-8), dict(q8=FAKE + 8),
        dict(freqs=FAKE + 4), dict(pos=FAKE + 1)],
    "mtp_latent_attn_fwd": [
        dict(seqs=-1), dict(total=-1), dict(heads=0), dict(pages=-1), dict(width=-1), dict(seqs=0), dict(total=1),
        dict(q=None), dict(cache=None), dict(bt=None), dict(lens=None), dict(cu=None), dict(d=None), dict(out=None),
        dict(pages=0), dict(width=0), dict(scale=math.inf), dict(scale=math.nan), dict(qt=0), dict(qh=4), dict(ot=-8),
        dict(oh=12), dict(q=FAKE + 8), dict(cache=FAKE + 8), dict(out=FAKE + 2), dict(bt=FAKE + 2), dict(lens=FAKE + 1),
        dict(cu=FAKE + 2), dict(mask=FAKE + 4), dict(d=FAKE + 2), dict(status=FAKE + 2)],
}
UNSUPPORTED = {
    "mtp_rope_append": [dict(rot=24), dict(rot=272), dict(pages=1 << 31), dict(width=1 << 28), dict(hq=65536),
                        dict(hkv=65536)],
    "mtp_rope_latent_append": [dict(pages=1 << 31), dict(width=1 << 28), dict(heads=65536)],
    "mtp_rope_prefill": [dict(hq=3), dict(hq=65536)],
    "mtp_latent_attn_fwd": [dict(heads=129), dict(total=129), dict(pages=1 << 31), dict(width=(1 << 27) - 4)],
}


@pytest.mark.parametrize("name", sorted(REFUSED))
def test_refusals(name):
    for over in REFUSED[name]:
        assert call(name, **over) == api.E_ARG, over
    for over in UNSUPPORTED[name]:
        assert call(name, **over) == api.E_UNSUPPORTED, over
    # nothing but the pointers themselves is wrong (or, without a device, that there is none)
    assert call(name) == api.E_DEVICE


def test_empty_calls():
    for name in ("mtp_rope_append", "mtp_rope_latent_append", "mtp_rope_prefill"):
        assert call(name, total=0) == api.OK
    assert call("mtp_latent_attn_fwd", seqs=0, total=0) == api.OK


def test_no_rotation_needs_no_freqs():
    assert call("mtp_rope_append", rot=0, freqs=None) == api.E_DEVICE
    assert call("mtp_rope_append", q=None, hq=0, out=None) == api.E_DEVICE


# ---- the binding's refusals ------------------------------------------------------------------------


def append_args(**over):
    t, hq, hkv = 3, 4, 2
    a = dict(q=torch.zeros(t, hq, 256, dtype=torch.bfloat16), k=torch.zeros(t, hkv, 256, dtype=torch.bfloat16),
             v=torch.zeros(t, hkv, 256, dtype=torch.bfloat16), positions=torch.zeros(t, dtype=torch.int32),
             freqs=torch.zeros(32, dtype=torch.int64), k_cache=torch.zeros(5, 16, hkv, 256, dtype=torch.uint8),
             v_cache=torch.zeros(5, 16, hkv, 256, dtype=torch.uint8), block_tables=torch.zeros(2, 2, dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32), cu_seqlens_q=torch.zeros(3, dtype=torch.int32),
             k_descale=torch.ones(1), v_descale=torch.ones(1))
    return {**a, **over}


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(3, 4, 256)), dict(k=torch.zeros(3, 2, 128, dtype=torch.bfloat16)),
    dict(v=torch.zeros(2, 2, 256, dtype=torch.bfloat16)), dict(v=torch.zeros(3, 1, 256, dtype=torch.bfloat16)),
    dict(positions=torch.zeros(3, dtype=torch.int64)), dict(positions=torch.zeros(2, dtype=torch.int32)),
    dict(freqs=torch.zeros(32)), dict(freqs=torch.zeros(129, dtype=torch.int64)),
    dict(k_cache=torch.zeros(5, 16, 1, 256, dtype=torch.uint8)), dict(v_cache=torch.zeros(4, 16, 2, 256, dtype=torch.uint8)),
    dict(block_tables=torch.zeros(3, 2, dtype=torch.int32)), dict(seq_lens=torch.zeros(3, dtype=torch.int32)),
    dict(k_descale=torch.ones(2)), dict(k_descale=torch.ones(1, dtype=torch.float64)),
    dict(q_out=torch.zeros(3, 4, 256)), dict(q_out=torch.zeros(3, 2, 256, dtype=torch.bfloat16)),
    dict(q=None, q_out=torch.zeros(3, 4, 256, dtype=torch.bfloat16)), dict(q=1), dict(mscale="x"),
    dict(q=torch.zeros(3, 4, 512, dtype=torch.bfloat16)[..., ::2])])
def test_binding_append_refusals(over):
    with pytest.raises(ValueError):
        api.mtp_rope_append(**append_args(**over))


def test_binding_refuses_cpu_tensors():
    with pytest.raises(api.MtpAttnError) as e:
        api.mtp_rope_append(**append_args())
    assert e.value.code == api.E_DEVICE


def latent_args(**over):
    a = dict(q=torch.zeros(3, 4, 576, dtype=torch.bfloat16), cache=torch.zeros(5, 16, 576, dtype=torch.uint8),
             block_tables=torch.zeros(2, 2, dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32),
             cu_seqlens_q=torch.zeros(3, dtype=torch.int32), descale=torch.ones(1), softmax_scale=0.1)
    return {**a, **over}


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(3, 4, 576)), dict(q=torch.zeros(3, 4, 512, dtype=torch.bfloat16)),
    dict(cache=torch.zeros(5, 16, 1, 576, dtype=torch.uint8)), dict(cache=torch.zeros(5, 16, 576)),
    dict(cache=torch.zeros(5, 16, 640, dtype=torch.uint8)[..., :576]), dict(tree_mask=torch.zeros(3, dtype=torch.int32)),
    dict(tree_mask=torch.zeros(2, dtype=torch.int64)), dict(out=torch.zeros(3, 4, 576, dtype=torch.bfloat16)),
    dict(out=torch.zeros(3, 4, 512)), dict(descale=torch.ones(2)), dict(softmax_scale=None),
    dict(cu_seqlens_q=torch.zeros(4, dtype=torch.int32))])
def test_binding_latent_refusals(over):
    with pytest.raises(ValueError):
        api.mtp_latent_attn_fwd(**latent_args(**over))


@pytest.mark.parametrize("over", [
    dict(q_rope=torch.zeros(3, 4, 64)), dict(latent=torch.zeros(3, 576, dtype=torch.bfloat16)),
    dict(k_rope=torch.zeros(2, 64, dtype=torch.bfloat16)), dict(freqs=torch.zeros(31, dtype=torch.int64)),
    dict(q_out=torch.zeros(3, 4, 576, dtype=torch.bfloat16)), dict(q_rope=None, q_out=torch.zeros(3, 4, 64, dtype=torch.bfloat16))])
def test_binding_latent_append_refusals(over):
    a = dict(q_rope=torch.zeros(3, 4, 64, dtype=torch.bfloat16), latent=torch.zeros(3, 512, dtype=torch.bfloat16),
             k_rope=torch.zeros(3, 64, dtype=torch.bfloat16), positions=torch.zeros(3, dtype=torch.int32),
             freqs=torch.zeros(32, dtype=torch.int64), cache=torch.zeros(5, 16, 576, dtype=torch.uint8),
             block_tables=torch.zeros(2, 2, dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32),
             cu_seqlens_q=torch.zeros(3, dtype=torch.int32), descale=torch.ones(1))
    with pytest.raises(ValueError):
        api.mtp_rope_latent_append(**{**a, **over})


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(3, 2, 128, dtype=torch.bfloat16)), dict(k=torch.zeros(3, 2, 192, dtype=torch.bfloat16)),
    dict(v=torch.zeros(3, 1, 128, dtype=torch.bfloat16)), dict(k_rope=torch.zeros(3, 2, 64, dtype=torch.bfloat16)),
    dict(q_out=torch.zeros(3, 2, 192)), dict(k_out=torch.zeros(3, 2, 128, dtype=torch.uint8)),
    dict(v_out=torch.zeros(3, 2, 256, dtype=torch.uint8)[..., :128])])
def test_binding_prefill_refusals(over):
    a = dict(q=torch.zeros(3, 2, 192, dtype=torch.bfloat16), k=torch.zeros(3, 2, 128, dtype=torch.bfloat16),
             k_rope=torch.zeros(3, 64, dtype=torch.bfloat16), v=torch.zeros(3, 2, 128, dtype=torch.bfloat16),
             positions=torch.zeros(3, dtype=torch.int32), freqs=torch.zeros(32, dtype=torch.int64),
             q_descale=torch.ones(1), k_descale=torch.ones(1), v_descale=torch.ones(1))
    with pytest.raises(ValueError):
        api.mtp_rope_prefill(**{**a, **over})
