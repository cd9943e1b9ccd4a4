"""What stands before and beside the attention calls of a step, as cases to be measured.

The operators:

* ``prefill``  rotary positions on the part of each head that carries them, and everything rounded
               to the e4m3 codes that the varlen prefill attention reads (q and k of 192, v of 128);
* ``append``   new tokens into the paged e4m3 K/V cache: rotary positions on q and k, k and v rounded
               and written through the block table;
* ``lappend``  the same for a cache of one latent vector (512, and 64 rotated) a token;
* ``latent``   attention of 1 to 64 new tokens a sequence over such a cache (the absorbed form: keys
               and values are the same 576 codes of a token, all heads share them).

``own`` chooses between the plain torch form (false) and the library's calls (true).
"""
import math
import random

import torch

own = False

PAGE = 16
DIM = 256                  # a head of the K/V cache
LATENT, ROPE = 512, 64     # a token of the latent cache
NOPE, VDIM = 128, 128      # a prefill head: 128 + 64 rotated, and its values
NODES = 64                 # most new tokens of one sequence in the latent attention
TOP = 448.0                # the largest e4m3 value
DEV = "cuda"


# ---- cases -------------------------------------------------------------------------------------


def listed():
    return [
        # a short prompt on a rank with 16 of the heads: the latency of a call
        dict(name="prefill_short", op="prefill", tokens=300, hq=16, hkv=16, interleaved=True,
             scaling="none", dtype="bfloat16"),
        # the prefill benchmark's 12288 tokens and 96 heads, far positions by interpolation
        dict(name="prefill_12k", op="prefill", tokens=12288, hq=96, hkv=96, interleaved=True,
             scaling="parts", dtype="bfloat16"),
        # one user, the last token and three drafted ones
        dict(name="append_one", op="append", lens="300", nodes="4", hkv=1, ratio=16, rot=256,
             interleaved=False, chain=True, scaling="none", dtype="bfloat16"),
        # a full batch with draft trees: positions by depth, a quarter of the head rotated
        dict(name="append_trees", op="append", lens="2027*64", nodes="26*64", hkv=2, ratio=16,
             rot=64, interleaved=True, chain=False, scaling="none", dtype="bfloat16"),
        # two prompts whole, all heads: the bytes of q count
        dict(name="append_prompts", op="append", lens="8191,8192", nodes="8191,8192", hkv=8,
             ratio=8, rot=256, interleaved=False, chain=True, scaling="linear",
             dtype="bfloat16"),
        # one user, four tokens, 16 heads
        dict(name="lappend_one", op="lappend", lens="300", nodes="4", heads=16,
             interleaved=True, chain=True, scaling="none", dtype="bfloat16"),
        # a chunk of 12288 prompt tokens and a batch that decodes beside it, all heads
        dict(name="lappend_mixed", op="lappend", lens="35000*64,14336", nodes="4*64,12288",
             heads=128, interleaved=True, chain=True, scaling="parts", dtype="bfloat16"),
        # one user, a short prompt, four tokens: the latency of a call
        dict(name="latent_one", op="latent", lens="300", nodes="4", heads=16, chain=True),
        # the verify benchmark's batch, 64 query rows a sequence: reading the cache
        dict(name="latent_16x35k", op="latent", lens="35000*16", nodes="4*16", heads=16,
             chain=True),
        # single tokens of all 128 heads: bound by the products
        dict(name="latent_heads", op="latent", lens="35000*16", nodes="1*16", heads=128,
             chain=True),
        # the draft-extend mix: contexts over the whole range, one to four tokens
        dict(name="latent_ragged", op="latent", lens="6,105000,431,27011,2290,63,9001,52345",
             nodes="4,2,1,3,4,3,1,2", heads=64, chain=True),
        # the widest draft trees: 1024 query rows a sequence
        dict(name="latent_trees", op="latent", lens="8191*8", nodes="64*8", heads=16,
             chain=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _ints(case, name):
    """The numbers of a case's text: "7,9" is [7, 9], "5*3" is [5, 5, 5]."""
    out = []
    for part in case[name].split(","):
        x, _, times = part.partition("*")
        out += [int(x)] * int(times or 1)
    return out


def _text(numbers):
    return ",".join(str(x) for x in numbers)


def draw(rng):
    op = rng.choice(["prefill", "append", "lappend", "latent", "latent"])
    scaling = rng.choice(["none", "none", "linear", "parts"])
    dtype = rng.choice(["bfloat16", "bfloat16", "bfloat16", "float16", "float32"])
    wide = 2 if dtype == "float32" else 1
    if op == "prefill":
        hkv = rng.choice([1, 2, 8, 16, 24, 96])
        hq = hkv * rng.choice([1, 1, 2, 4]) if hkv < 24 else hkv
        return dict(op=op, tokens=_log(rng, 1, min(20000, 1_100_000 // (hq + hkv) // wide)), hq=hq,
                    hkv=hkv, interleaved=rng.random() < 0.7, scaling=scaling, dtype=dtype)
    seqs = _log(rng, 1, 128)
    if op in ("append", "lappend"):
        c = dict(op=op, interleaved=rng.random() < 0.5, chain=rng.random() < 0.5, scaling=scaling,
                 dtype=dtype)
        if op == "append":
            c["hkv"], c["ratio"] = rng.choice([1, 1, 2, 3, 8]), rng.choice([1, 3, 8, 8, 16])
            c["rot"] = rng.choice([32, 64, 96, 128, 256, 256])
            room = 16383 * 80 // (c["hkv"] * (c["ratio"] + 2)) // wide
        else:
            c["heads"] = rng.choice([1, 8, 16, 20, 64, 128])
            room = 12544 * 136 // (c["heads"] + 8) // wide
        top = _log(rng, 1, 12288 if c["chain"] else NODES)
        hi, kept = _log(rng, 1, 35000), 560_000 // c.get("hkv", 1)
        lens, nodes = [], []
        for _ in range(seqs):
            n = rng.randint(1, min(top, room))
            ln = n + _log(rng, 1, hi)
            if n > room or ln > kept:
                break
            room, kept = room - n, kept - ln
            lens.append(ln)
            nodes.append(n)
            if room < 1:
                break
        if not lens:
            lens, nodes = [65], [4]
        return dict(c, lens=_text(lens), nodes=_text(nodes))
    heads = rng.choice([1, 5, 8, 16, 16, 32, 64, 128, 128])
    top, hi = _log(rng, 1, NODES), _log(rng, 64, 105000)
    lens, nodes, keys, pairs = [], [], 0, 0
    for _ in range(seqs):
        n = rng.randint(1, top)
        ln = n + _log(rng, 1, hi)
        # no dearer than the largest listed cases: cache bytes, and products of rows and keys
        if keys + ln > 560_000 or pairs + ln * n * heads > 67_000_000 or ln * n * heads > 27_000_000:
            break
        keys, pairs = keys + ln, pairs + ln * n * heads
        lens.append(ln)
        nodes.append(n)
    if not lens:
        lens, nodes = [rng.randint(65, 2000)], [rng.randint(1, 64)]
    return dict(op=op, lens=_text(lens), nodes=_text(nodes), heads=heads, chain=rng.random() < 0.6)


def work(case):
    op = case["op"]
    if op == "latent":
        seen = keys = 0
        for ln, n, p in zip(_ints(case, "lens"), _ints(case, "nodes"), _parents(case)):
            keys += ln
            seen += n * (ln - n) + sum(_depths(p)) + n
        rows = sum(_ints(case, "nodes")) * case["heads"]
        return {"bytes": keys * (LATENT + ROPE) + rows * (2 * LATENT + ROPE) * 2,
                "flops": 2 * seen * case["heads"] * (2 * LATENT + ROPE)}
    size = 4 if case["dtype"] == "float32" else 2
    if op == "prefill":
        hq, hkv, t = case["hq"], case["hkv"], case["tokens"]
        codes = hq * (NOPE + ROPE) + hkv * (NOPE + ROPE + VDIM)
        read = hq * (NOPE + ROPE) + hkv * (NOPE + VDIM) + ROPE
        return {"bytes": t * (read * size + codes), "flops": t * (3 * (hq + 1) * ROPE + codes)}
    t = sum(_ints(case, "nodes"))
    if op == "append":
        hkv = case["hkv"]
        hq = hkv * case["ratio"]
        return {"bytes": t * ((hq + 2 * hkv) * DIM * size + hq * DIM * 2 + 2 * hkv * DIM),
                "flops": t * (3 * (hq + hkv) * case["rot"] + 2 * hkv * DIM)}
    return {"bytes": t * ((LATENT + ROPE * (1 + case["heads"])) * size + case["heads"] * ROPE * 2 +
                          LATENT + ROPE),
            "flops": t * (3 * (case["heads"] + 1) * ROPE + LATENT + ROPE)}


# ---- inputs ------------------------------------------------------------------------------------


def _parents(case):
    """The new tokens' links, parents before children: a chain, or a tree that branches."""
    trees = []
    rng = random.Random(12345)
    for n in _ints(case, "nodes"):
        trees.append([-1] + [i - 1 if case["chain"] else
                             rng.randint(max(0, (i - 1) // 4 - 1), max(0, (i - 1) // 4))
                             for i in range(1, n)])
    return trees


def _depths(parents):
    out = []
    for p in parents:
        out.append(out[p] + 1 if p >= 0 else 0)
    return out


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _normal(g, *shape, dtype="bfloat16"):
    out = torch.empty(shape, dtype=getattr(torch, dtype), device=DEV)
    flat, step = out.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV)
    return out


def _codes(g, *shape):
    """Cache contents: unit normal values rounded to e4m3, as uint8."""
    return _normal(g, *shape, dtype="float8_e4m3fn").view(torch.uint8)


def _inv_freq(rot, scaling):
    """Radians a position for each rotated pair, and the factor on sines and cosines: as they are,
    all of them slowed down for contexts four times as long, or only those that turn seldom within
    the trained length of 4096 (between 1 and 32 turns, in part)."""
    inv = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [f / 4.0 for f in inv], 1.0
    if scaling == "parts":
        def keep(f):
            return min(1.0, max(0.0, (4096 * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)))
        return [f * keep(f) + f / 40.0 * (1.0 - keep(f)) for f in inv], 0.1 * math.log(40.0) + 1.0
    return inv, 1.0


def _paged(s, case, g, *row):
    """Block tables and lengths of the case's sequences; returns the pool's shape."""
    lens, nodes = _ints(case, "lens"), _ints(case, "nodes")
    per = [-(-ln // PAGE) for ln in lens]
    pool = sum(per) + 3
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    bt = torch.full((len(lens), max(per)), -1, dtype=torch.int32, device=DEV)
    at, cu = 0, [0]
    for b, n in enumerate(per):
        bt[b, :n] = perm[at:at + n]
        at += n
        cu.append(cu[-1] + nodes[b])
    s.update(bt=bt, lens=_i32(lens), cu=_i32(cu), first=cu)
    return (pool, PAGE) + row


def _rotary(s, case, rot):
    inv, s["mscale"] = _inv_freq(rot, case["scaling"])
    s["inv"] = torch.tensor(inv, dtype=torch.float64, device=DEV)
    if own:
        from paged_fp8_speculative_gb300 import api
        s["freqs"] = api.mtp_rope_freqs(inv, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(1_000_003 * seed + 29)
    s = dict(case=case)
    op = case["op"]
    if op == "prefill":
        t, hq, hkv, dt = case["tokens"], case["hq"], case["hkv"], case["dtype"]
        s["q"] = _normal(g, t, hq, NOPE + ROPE, dtype=dt)
        # one projection gives the keys' unrotated part and the values, another the shared part
        kv = _normal(g, t, hkv, NOPE + VDIM, dtype=dt)
        s["k"], s["v"] = kv[..., :NOPE], kv[..., NOPE:]
        s["k_rope"] = _normal(g, t, LATENT + ROPE, dtype=dt)[:, LATENT:]
        s["positions"] = _i32(list(range(t))) + 1000 * (seed % 100)
        s["qd"], s["kd"], s["vd"] = (torch.full((1,), x, device=DEV) for x in (0.03, 0.0171, 0.02))
        _rotary(s, case, ROPE)
        return s
    if op == "latent":
        heads = case["heads"]
        s["cache"] = _codes(g, *_paged(s, case, g, LATENT + ROPE))
        s["q"] = _normal(g, s["first"][-1], heads, LATENT + ROPE)
        s["descale"] = torch.full((1,), 0.75, device=DEV)
        s["scale"] = 1.5 / math.sqrt(NOPE + ROPE)
        s["mask"] = None
        if not case["chain"]:
            bits = []
            for p in _parents(case):
                words = []
                for i, up in enumerate(p):
                    words.append((words[up] if up >= 0 else 0) | 1 << i)
                bits += [w - (1 << 64) if w >> 63 else w for w in words]
            s["mask"] = torch.tensor(bits, dtype=torch.int64, device=DEV)
        return s
    starts = [ln - n for ln, n in zip(_ints(case, "lens"), _ints(case, "nodes"))]
    s["positions"] = _i32([a + d for a, p in zip(starts, _parents(case)) for d in _depths(p)])
    t, dt = len(s["positions"]), case["dtype"]
    s["kd"], s["vd"] = torch.full((1,), 0.0171, device=DEV), torch.full((1,), 0.02, device=DEV)
    if op == "append":
        hkv, hq = case["hkv"], case["hkv"] * case["ratio"]
        shape = _paged(s, case, g, hkv, DIM)
        s["k_cache"], s["v_cache"] = _codes(g, *shape), _codes(g, *shape)
        # q, k and v as one projection leaves them
        qkv = _normal(g, t, hq + 2 * hkv, DIM, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.empty(t, hq, DIM, dtype=torch.bfloat16, device=DEV)
        _rotary(s, case, case["rot"])
        return s
    heads = case["heads"]
    s["cache"] = _codes(g, *_paged(s, case, g, LATENT + ROPE))
    # the projections' own layouts; the rotated part of q goes beside the absorbed one
    both = _normal(g, t, LATENT + ROPE, dtype=dt)
    s["latent"], s["k_rope"] = both[:, :LATENT], both[:, LATENT:]
    s["q_rope"] = _normal(g, t, heads, NOPE + ROPE, dtype=dt)[..., NOPE:]
    s["q_out"] = torch.empty(t, heads, LATENT + ROPE, dtype=torch.bfloat16, device=DEV)[..., LATENT:]
    _rotary(s, case, ROPE)
    return s


# ---- the plain forms ---------------------------------------------------------------------------


def _rotate(x, s, interleaved):
    """Rotary positions on the first 2 * len(inv) of the last axis of x [tokens, heads, ..]."""
    angle = s["positions"].double()[:, None] * s["inv"]
    c = (torch.cos(angle) * s["mscale"]).float()[:, None]
    d = (torch.sin(angle) * s["mscale"]).float()[:, None]
    rot = 2 * c.shape[-1]
    y = x.float().clone()
    if interleaved:
        a, b = x[..., 0:rot:2].float(), x[..., 1:rot:2].float()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * d, b * c + a * d
    else:
        a, b = x[..., :rot // 2].float(), x[..., rot // 2:rot].float()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * d, b * c + a * d
    return y


def _round(x, descale):
    return (x.float() / descale).clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _places(s):
    """The page and the row in it of every new token."""
    cu = s["cu"].long()
    at = torch.arange(s["first"][-1], device=DEV)
    seq = torch.searchsorted(cu[1:], at, right=True)
    slot = s["lens"].long()[seq] - cu[seq + 1] + at
    return s["bt"][seq, slot // PAGE].long(), slot % PAGE


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "prefill":
        q, k, kr = s["q"], s["k"], s["k_rope"]
        kr = _rotate(kr[:, None], s, case["interleaved"]).expand(-1, k.shape[1], -1)
        q = torch.cat([q[..., :NOPE].float(), _rotate(q[..., NOPE:], s, case["interleaved"])], -1)
        return (_round(q, s["qd"]), _round(torch.cat([k.float(), kr], -1), s["kd"]),
                _round(s["v"], s["vd"]))
    if op == "append":
        page, row = _places(s)
        s["q_out"].copy_(_rotate(s["q"], s, case["interleaved"]))
        k = _round(_rotate(s["k"], s, case["interleaved"]), s["kd"])
        s["k_cache"][page, row] = k.view(torch.uint8)
        s["v_cache"][page, row] = _round(s["v"], s["vd"]).view(torch.uint8)
        return s["q_out"], s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn)
    if op == "lappend":
        page, row = _places(s)
        s["q_out"].copy_(_rotate(s["q_rope"], s, case["interleaved"]))
        kr = _rotate(s["k_rope"][:, None], s, case["interleaved"])[:, 0]
        both = _round(torch.cat([s["latent"].float(), kr], -1), s["kd"])
        s["cache"][page, row] = both.view(torch.uint8)
        return s["q_out"], s["cache"].view(torch.float8_e4m3fn)
    heads = case["heads"]
    out = torch.empty(s["q"].shape[0], heads, LATENT, dtype=torch.bfloat16, device=DEV)
    for b, ln in enumerate(_ints(case, "lens")):
        q0, q1 = s["first"][b], s["first"][b + 1]
        n = q1 - q0
        at = torch.arange(ln, device=DEV)
        keys = s["cache"][s["bt"][b, at // PAGE].long(), at % PAGE].view(torch.float8_e4m3fn).float()
        score = s["q"][q0:q1].reshape(n * heads, -1).float() @ keys.T
        score = (score * (s["descale"] * s["scale"])).view(n, heads, ln)
        node = torch.arange(n, device=DEV)
        if s["mask"] is None:
            see = node[None] <= node[:, None]
        else:
            see = (s["mask"][q0:q1, None] >> node[None]) & 1 == 1
        score[:, :, ln - n:].masked_fill_(~see[:, None], -math.inf)
        p = torch.exp(score - score.amax(-1, keepdim=True)).view(n * heads, ln)
        o = (p @ keys[:, :LATENT]) / p.sum(-1, keepdim=True) * s["descale"]
        out[q0:q1] = o.view(n, heads, LATENT)
    return out


# ---- the library's calls -----------------------------------------------------------------------


def run(s):
    if not own:
        return _plain(s)
    from paged_fp8_speculative_gb300 import api
    case = s["case"]
    op = case["op"]
    if op == "latent":
        return api.mtp_latent_attn_fwd(s["q"], s["cache"], s["bt"], s["lens"], s["cu"], s["descale"],
                                       s["scale"], tree_mask=s["mask"])
    how = dict(mscale=s["mscale"], interleaved=case["interleaved"])
    if op == "prefill":
        q, k, v = api.mtp_rope_prefill(s["q"], s["k"], s["k_rope"], s["v"], s["positions"],
                                       s["freqs"], s["qd"], s["kd"], s["vd"], **how)
        return q, k, v
    if op == "append":
        api.mtp_rope_append(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["k_cache"],
                            s["v_cache"], s["bt"], s["lens"], s["cu"], s["kd"], s["vd"],
                            q_out=s["q_out"], **how)
        return s["q_out"], s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn)
    api.mtp_rope_latent_append(s["q_rope"], s["latent"], s["k_rope"], s["positions"], s["freqs"],
                               s["cache"], s["bt"], s["lens"], s["cu"], s["kd"], q_out=s["q_out"],
                               **how)
    return s["q_out"], s["cache"].view(torch.float8_e4m3fn)


# ---- the definitions in 64 bits ----------------------------------------------------------------


def _turned(x, s, interleaved):
    """Rotary positions as products of complex numbers; x [tokens, heads, rotated]."""
    x = x.double()
    half = x.shape[-1] // 2
    pair = x.unflatten(-1, (half, 2)) if interleaved else x.unflatten(-1, (2, half)).transpose(-1, -2)
    turn = torch.polar(torch.full_like(s["inv"], s["mscale"]).expand(x.shape[0], -1).contiguous(),
                       torch.outer(s["positions"].double(), s["inv"]))
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
    return z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)


def _clipped(x, descale):
    return (x.double() / descale.double()).clamp(-TOP, TOP)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefill":
        il = case["interleaved"]
        q, k = s["q"].double(), s["k"].double()
        q[..., NOPE:] = _turned(q[..., NOPE:], s, il)
        kr = _turned(s["k_rope"][:, None], s, il).repeat(1, k.shape[1], 1)
        return (_clipped(q, s["qd"]), _clipped(torch.cat([k, kr], -1), s["kd"]),
                _clipped(s["v"], s["vd"]))
    if op == "latent":
        heads, out = case["heads"], []
        for b, (ln, n) in enumerate(zip(_ints(case, "lens"), _ints(case, "nodes"))):
            q0 = s["first"][b]
            pages = s["bt"][b, :-(-ln // PAGE)].long()
            keys = s["cache"][pages].flatten(0, 1)[:ln].view(torch.float8_e4m3fn).double()
            keys *= s["descale"].double()
            for i in range(n):
                score = s["q"][q0 + i].double() @ keys.T * s["scale"]
                word = (1 << (i + 1)) - 1 if s["mask"] is None else int(s["mask"][q0 + i])
                dark = [ln - n + j for j in range(n) if not word >> j & 1]
                score[:, dark] = -math.inf
                out.append(torch.softmax(score, -1) @ keys[:, :LATENT])
        return torch.stack(out)
    lens, nodes = _ints(case, "lens"), _ints(case, "nodes")
    slot = torch.tensor([b * s["bt"].shape[1] * PAGE + ln - n + i
                         for b, (ln, n) in enumerate(zip(lens, nodes)) for i in range(n)], device=DEV)
    place = s["bt"].view(-1).long()[slot // PAGE] * PAGE + slot % PAGE
    il = case["interleaved"]

    def with_rows(cache, rows):
        out = cache.view(torch.float8_e4m3fn).double().flatten(0, 1)
        out[place] = rows
        return out.view(cache.shape)

    if op == "append":
        q, k, rot = s["q"].double(), s["k"].double(), case["rot"]
        q[..., :rot], k[..., :rot] = _turned(q[..., :rot], s, il), _turned(k[..., :rot], s, il)
        return (q, with_rows(s["k_cache"], _clipped(k, s["kd"])),
                with_rows(s["v_cache"], _clipped(s["v"], s["vd"])))
    rows = torch.cat([s["latent"].double(), _turned(s["k_rope"][:, None], s, il)[:, 0]], -1)
    return _turned(s["q_rope"], s, il), with_rows(s["cache"], _clipped(rows, s["kd"]))
