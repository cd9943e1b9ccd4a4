"""What a speculative-decoding step does around the verify attention, as cases to be measured.

The operators:

* ``attn``    attention of a tree of drafted tokens over the paged e4m3 cache;
* ``greedy``  the walk down the draft tree that follows the target's largest logits;
* ``sample``  the walk by rejection sampling from the target's and the drafter's probabilities;
* ``compact`` the accepted tokens' keys and values moved to where the sequence goes on;
* ``pages``   a step of a paged cache's book-keeping: rows retired and trimmed, rows forked,
              pages handed out for the next tree.

``own`` chooses between the plain torch form (false) and the library's calls (true).
"""
import math
import random

import torch

own = False

PAGE = 16
DIM = 256
NODES = 64           # most tree nodes of one sequence
DEV = "cuda"


# ---- cases -------------------------------------------------------------------------------------


def listed():
    return [
        # one user, a short prompt, a small tree: the latency of a call
        dict(name="attn_small", op="attn", lens="300", nodes="8", hkv=1, ratio=8),
        # the verify benchmark's batch with a tree of eight tokens: reading the cache
        dict(name="attn_16x35k", op="attn", lens="35000*16", nodes="8*16", hkv=1, ratio=16),
        # the draft-extend mix: contexts over the whole range, trees of one to sixteen tokens
        dict(name="attn_ragged", op="attn", lens="6,105000,431,27011,2290,63,9001,52345",
             nodes="5,16,1,9,13,16,3,7", hkv=1, ratio=16),
        # the widest trees: 1024 query rows a KV head, bound by the products
        dict(name="attn_wide", op="attn", lens="8191*8", nodes="64*8", hkv=2, ratio=16),
        # one user, a chain of three drafted tokens, a small vocabulary
        dict(name="sample_chain", op="sample", nodes="4", vocab=32000, drafter=True, chain=True,
             dtype="float32"),
        # a full batch with trees drawn from the drafter's distributions
        dict(name="sample_tree", op="sample", nodes="26*64", vocab=131072, drafter=True,
             chain=False, dtype="float32"),
        # one user, greedy, an odd vocabulary (rows that start at any address)
        dict(name="greedy_one", op="greedy", nodes="8", vocab=50257, chain=True, dtype="float32"),
        # a full batch, greedy, logits as the model leaves them
        dict(name="greedy_batch", op="greedy", nodes="16*64", vocab=131072, chain=False,
             dtype="bfloat16"),
        # one user's accepted path in one layer's cache
        dict(name="compact_one", op="compact", lens="1001", nodes="8", hkv=1, layers=1),
        # a full batch, all the layers of a stack at once
        dict(name="compact_batch", op="compact", lens="203*64", nodes="26*64", hkv=2,
             layers=16),
        # a handful of sequences in a small pool
        dict(name="pages_small", op="pages", rows=4, forks=1, lens_hi=300, pool=512, room=4,
             layers=1),
        # parallel sampling: half of the rows are forked anew from the other half
        dict(name="pages_batch", op="pages", rows=256, forks=128, lens_hi=1500, pool=16384,
             room=26, layers=4),
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
    op = rng.choice(["attn", "attn", "greedy", "sample", "compact", "pages"])
    if op == "attn":
        hkv = rng.choice([1, 1, 2, 3, 4, 8])
        ratio = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 16])
        seqs, top, hi = _log(rng, 1, 64), _log(rng, 1, NODES), _log(rng, 64, 105000)
        keys = 0
        lens, nodes = [], []
        for _ in range(seqs):
            n = rng.randint(1, top)
            ln = n + _log(rng, 1, hi)
            # no dearer than the largest listed cases: cache bytes and products, and the plain
            # form's padded arrays
            pad = (len(lens) + 1) * max(lens + [ln]) * hkv
            if ((keys + ln) * hkv > 560_000 or (keys + ln) * hkv * top * ratio > 134_000_000
                    or pad > 840_000 or pad * top * ratio > 215_000_000):
                break
            keys += ln
            lens.append(ln)
            nodes.append(n)
        if not lens:
            lens, nodes = [rng.randint(65, 2000)], [rng.randint(1, 64)]
        return dict(op="attn", lens=_text(lens), nodes=_text(nodes), hkv=hkv, ratio=ratio)
    if op in ("greedy", "sample"):
        vocab = _log(rng, 500, 131072)
        wide = {"greedy": 134e6, "sample": 218e6}[op] / vocab
        seqs = min(_log(rng, 1, 64), max(1, int(wide)))
        top = max(1, min(_log(rng, 1, NODES), int(wide / seqs)))
        c = dict(op=op, nodes=_text(rng.randint(1, top) for _ in range(seqs)), vocab=vocab,
                 chain=rng.random() < 0.4)
        if op == "sample":
            c["drafter"] = rng.random() < 0.7
            c["dtype"] = rng.choice(["float32", "float32", "bfloat16"])
        else:
            c["dtype"] = rng.choice(["float32", "bfloat16", "float16"])
        return c
    if op == "compact":
        layers, hkv = _log(rng, 1, 16), rng.choice([1, 2, 3])
        seqs, top = _log(rng, 1, 64), rng.randint(2, 40)
        nodes = [rng.randint(1, top) for _ in range(seqs)]
        most = max(2, min(200, 33_000 // (seqs * layers * hkv) * 16))
        return dict(op="compact", lens=_text(n + rng.randint(0, most) for n in nodes),
                    nodes=_text(nodes), hkv=hkv, layers=layers)
    rows = 2 * _log(rng, 1, 128)
    forks = rng.randint(1, rows // 2)
    hi = _log(rng, 20, 1500)
    pool = min(16384, rows * ((hi + NODES) // PAGE + 2) + rng.randint(0, 500))
    hi = max(1, min(hi, (pool // rows - 2) * PAGE - NODES))
    return dict(op="pages", rows=rows, forks=forks, lens_hi=hi, pool=pool,
                room=rng.randint(1, NODES), layers=rng.randint(1, 4))


def work(case):
    op = case["op"]
    if op == "attn":
        hq = case["hkv"] * case["ratio"]
        seen = keys = 0
        for ln, n, p in zip(_ints(case, "lens"), _ints(case, "nodes"), _parents(case, 0)):
            keys += ln
            seen += n * (ln - n) + sum(len(_path(p, i)) for i in range(n))
        rows = sum(_ints(case, "nodes")) * hq
        pages = sum(-(-ln // PAGE) for ln in _ints(case, "lens"))
        return {"bytes": keys * case["hkv"] * DIM * 2 + rows * DIM * 4 + 4 * pages,
                "flops": 4 * seen * hq * DIM}
    if op in ("greedy", "sample"):
        # sampling: the row of each sequence's last node (and the drafter's); greedy: the rows
        # of the nodes on the way too, the drafter being right about two times in three
        size = {"float32": 4, "bfloat16": 2, "float16": 2}[case["dtype"]]
        if op == "sample":
            rows = len(_ints(case, "nodes")) * (2 if case["drafter"] else 1)
        else:
            rows = sum(0.65 ** d for t in _parents(case, 0)
                       for d in range(max(len(_path(t, i)) for i in range(len(t)))))
        rows = int(rows)
        return {"bytes": rows * case["vocab"] * size, "flops": rows * case["vocab"]}
    if op == "compact":
        # about a third of the tree is kept, read and written once
        kept = sum(max(0, n // 3) for n in _ints(case, "nodes"))
        return {"bytes": kept * case["layers"] * case["hkv"] * DIM * 2 * 2 + 64, "flops": 0}
    # a scan of the pool's counts for free pages in the two calls that hand pages out, the
    # forked rows' last pages copied, and the tables of the rows that change
    pages = case["rows"] * (case["lens_hi"] // PAGE) // 2
    copies = case["forks"] * case["layers"] * PAGE * DIM * 2 * 2
    return {"bytes": 8 * case["pool"] + copies + 8 * pages, "flops": 0}


# ---- inputs ------------------------------------------------------------------------------------


def _parents(case, seed):
    """The draft trees' links, parents before children: a chain, or a tree that branches."""
    rng = random.Random(12345 + 97 * seed)
    trees = []
    for n in _ints(case, "nodes"):
        back = 1 if case.get("chain") else 4
        trees.append([-1] + [rng.randint(max(0, (i - 1) // back - 1), max(0, (i - 1) // back))
                             if back > 1 else i - 1 for i in range(1, n)])
    return trees


def _path(parents, i):
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out[::-1]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _codes(shape, g):
    """Cache contents: unit normal values rounded to e4m3."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat, step = out.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV).to(torch.float8_e4m3fn)
    return out


def _cu(nodes):
    cu = [0]
    for n in nodes:
        cu.append(cu[-1] + n)
    return cu


def _tables(lens, g, spare=0):
    """Shuffled pages for sequences of these lengths: (block tables, pages in the pool)."""
    per = [-(-ln // PAGE) for ln in lens]
    pool = sum(per) + spare
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    bt = torch.full((len(lens), max(per)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(per):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, pool


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(1_000_003 * seed + 17)
    s = dict(case=case)
    op = case["op"]
    if op == "attn":
        hkv, ratio = case["hkv"], case["ratio"]
        cu = _cu(_ints(case, "nodes"))
        s["bt"], pool = _tables(_ints(case, "lens"), g, spare=3)
        s["k"] = _codes((pool, PAGE, hkv, DIM), g)
        s["v"] = _codes((pool, PAGE, hkv, DIM), g)
        s["q"] = torch.randn(cu[-1], hkv * ratio, DIM, generator=g, device=DEV).bfloat16()
        s["lens"], s["cu"] = _i32(_ints(case, "lens")), _i32(cu)
        bits = []
        for p in _parents(case, seed):
            for i in range(len(p)):
                word = sum(1 << j for j in _path(p, i))
                bits.append(word - (1 << 64) if word >> 63 else word)
        s["mask"] = torch.tensor(bits, dtype=torch.int64, device=DEV)
        s["kd"] = torch.full((1,), 0.75, device=DEV)
        s["vd"] = torch.full((1,), 1.25, device=DEV)
        s["scale"] = 2.0 / math.sqrt(DIM)
        # where each sequence's rows stand, for the plain form's padded arrays
        s["row_seq"] = torch.cat([torch.full((n,), b, device=DEV) for b, n in enumerate(_ints(case, "nodes"))])
        s["row_at"] = torch.cat([torch.arange(n, device=DEV) for n in _ints(case, "nodes")])
        return s
    if op in ("greedy", "sample"):
        vocab, dtype = case["vocab"], getattr(torch, case["dtype"])
        trees = _parents(case, seed)
        cu = _cu(_ints(case, "nodes"))
        total, seqs = cu[-1], len(trees)
        s["cu"] = _i32(cu)
        s["parents"] = _i32([p for t in trees for p in t])
        up = torch.tensor([cu[b] + max(0, p) for b, t in enumerate(trees) for p in t], device=DEV)
        logits = torch.randn(total, vocab, generator=g, device=DEV)
        logits *= 3.0
        if op == "greedy":
            s["logits"] = logits.to(dtype)
            # a drafter that is right about two times in three
            top = s["logits"].float().argmax(-1)[up]
            other = torch.randint(0, vocab, (total,), generator=g, device=DEV)
            right = torch.rand(total, generator=g, device=DEV) < 0.65
            s["tokens"] = torch.where(right, top, other).to(torch.int32)
        else:
            s["p"] = torch.softmax(logits, -1).to(dtype)
            logits += torch.randn(total, vocab, generator=g, device=DEV)
            q = torch.softmax(logits, -1)
            s["q"] = q.to(dtype) if case["drafter"] else None
            # each node's token is drawn from its parent's row (by the largest of q over
            # exponential noise, so that one pass over the rows draws them all)
            noise = torch.empty(1, vocab, device=DEV)
            tok = torch.empty(total, dtype=torch.int64, device=DEV)
            for i in range(0, total, 64):
                noise = torch.empty(min(64, total - i), vocab, device=DEV).exponential_(generator=g)
                tok[i:i + 64] = (q[up[i:i + 64]] / noise).argmax(-1)
            s["tokens"] = tok.to(torch.int32)
            s["u"] = torch.rand(total, generator=g, device=DEV)
        del logits
        # the padded node grid of the plain form: [sequence, node] -> packed row, or the root's
        at = torch.arange(NODES, device=DEV)[None, :]
        n = torch.tensor(_ints(case, "nodes"), device=DEV)[:, None]
        first = torch.tensor(cu[:-1], device=DEV)[:, None]
        s["grid"] = first + torch.where(at < n, at, torch.zeros_like(at))
        s["live"] = at < n
        s["first"] = first[:, 0]
        # loop bounds of the plain form: the deepest path, the most children of a node
        s["depth"] = max(len(_path(t, i)) - 1 for t in trees for i in range(len(t)))
        s["most"] = max([t.count(i) for t in trees for i in range(len(t))])
        return s
    if op == "compact":
        cu = _cu(_ints(case, "nodes"))
        trees = _parents(case, seed)
        s["bt"], pool = _tables(_ints(case, "lens"), g, spare=2)
        shape = (case["layers"], pool, PAGE, case["hkv"], DIM)
        s["k"], s["v"] = _codes(shape, g), _codes(shape, g)
        s["lens"], s["cu"] = _i32(_ints(case, "lens")), _i32(cu)
        rng = random.Random(seed)
        index, count = [], []
        for t in trees:
            path = _path(t, rng.randrange(len(t)))
            index.append(path + [-1] * (NODES - len(path)))
            count.append(len(path) - 1)
        s["index"], s["count"] = _i32(index), _i32(count)
        s["new"] = torch.zeros(len(trees), dtype=torch.int32, device=DEV)
        return s
    # pages: `rows` sequences, the last `forks` of which are forks that the pass retires and
    # forks anew from the first ones; every row ends with the room for its next tree
    rng = random.Random(seed)
    rows, forks, room = case["rows"], case["forks"], case["room"]
    lens = [rng.randint(1, case["lens_hi"]) for _ in range(rows)]
    lens[rows - forks:] = lens[:forks]
    held = [ln + room for ln in lens]
    width = -(-(case["lens_hi"] + room) // PAGE)
    pool = case["pool"]
    bt = torch.full((rows, width), -1, dtype=torch.int32)
    ref = torch.zeros(pool, dtype=torch.int32)
    free = list(range(pool))
    rng.shuffle(free)
    for b in range(rows):
        whole = lens[b] // PAGE
        for j in range(-(-held[b] // PAGE)):
            if b >= rows - forks and j < whole:
                page = int(bt[b - (rows - forks), j])
            else:
                page = free.pop()
            bt[b, j] = page
            ref[page] += 1
    s["bt"], s["ref"], s["lens"] = bt.to(DEV), ref.to(DEV), _i32(held)
    keep = list(lens)
    keep[rows - forks:] = [0] * forks
    s["keep"], s["held"] = _i32(keep), _i32(held)
    s["src"], s["dst"] = _i32(list(range(forks))), _i32(list(range(rows - forks, rows)))
    shape = (case["layers"], pool, PAGE, 1, DIM)
    s["k"], s["v"] = _codes(shape, g), _codes(shape, g)
    return s


# ---- one pass ----------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"attn": _attn, "greedy": _greedy, "sample": _sample, "compact": _compact,
            "pages": _pages}[op](state)


def _own(op, s):
    from paged_fp8_speculative_gb300 import api
    if "ws" not in s and op in ("attn", "pages"):        # kept for the calls that follow
        if op == "attn":
            nbytes = api.mtp_tree_attn_workspace_size(s["lens"].numel(), s["q"].shape[0],
                                                      s["q"].shape[1], s["k"].shape[2],
                                                      s["bt"].shape[1])
        else:
            nbytes = api.mtp_cache_workspace_size(*s["bt"].shape)
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    if op == "attn":
        return api.mtp_tree_attn_fwd(s["q"], s["k"], s["v"], s["bt"], s["lens"], s["cu"], s["mask"],
                                     s["kd"], s["vd"], s["scale"], workspace=s["ws"])
    if op == "greedy":
        return api.mtp_tree_verify_greedy(s["logits"], s["tokens"], s["parents"], s["cu"])
    if op == "sample":
        return api.mtp_tree_verify_sample(s["p"], s["q"], s["tokens"], s["parents"], s["cu"], s["u"])
    if op == "compact":
        api.mtp_cache_compact(s["k"], s["v"], s["bt"], s["lens"], s["cu"], s["index"], s["count"],
                              new_seq_lens=s["new"])
        return s["k"], s["v"], s["new"]
    pool = (s["k"], s["v"], s["bt"], s["lens"], s["ref"])
    api.mtp_cache_resize(*pool, s["keep"], workspace=s["ws"])
    api.mtp_cache_fork(*pool, s["src"], s["dst"], workspace=s["ws"])
    api.mtp_cache_resize(*pool, s["held"], workspace=s["ws"])
    return pool


def _rows(cache, *index):
    return cache.view(torch.uint8)[index].view(cache.dtype)


def _attn(s):
    """Scores of every (row, key) pair of the padded batch in 32 bits, softmax, product."""
    c = s["case"]
    hkv, ratio = c["hkv"], c["ratio"]
    seqs, width = s["bt"].shape
    most = max(_ints(c, "nodes"))
    pages = s["bt"].clamp_min(0).long()
    k = _rows(s["k"], pages).reshape(seqs, width * PAGE, hkv, DIM).permute(0, 2, 3, 1).float()
    q = torch.zeros(seqs, most, hkv, ratio, DIM, device=DEV)
    q[s["row_seq"], s["row_at"]] = s["q"].float().view(-1, hkv, ratio, DIM)
    q = q.permute(0, 2, 1, 3, 4).reshape(seqs, hkv, most * ratio, DIM)
    sc = torch.matmul(q, k)
    del k
    sc *= s["scale"] * s["kd"]
    word = torch.zeros(seqs, most, dtype=torch.int64, device=DEV)
    word[s["row_seq"], s["row_at"]] = s["mask"]
    # a key before the tree is seen by every row, a node of the tree by the rows whose bit is set
    key = torch.arange(width * PAGE, device=DEV)
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    node = key[None, :] - (s["lens"].long() - n)[:, None]
    bit = (word[:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1
    seen = (node < 0)[:, None, :] | ((node < n[:, None])[:, None, :] & (bit == 1))
    seen = seen[:, None, :, None, :].expand(seqs, 1, most, ratio, width * PAGE)
    sc.view(seqs, hkv, most, ratio, -1).masked_fill_(~seen, -math.inf)
    top = sc.amax(-1, keepdim=True)
    sc -= torch.where(top == -math.inf, torch.zeros_like(top), top)
    sc.exp_()
    total = sc.sum(-1, keepdim=True)
    v = _rows(s["v"], pages).reshape(seqs, width * PAGE, hkv, DIM).permute(0, 2, 1, 3).float()
    o = torch.matmul(sc, v) / torch.where(total > 0, total, torch.ones_like(total)) * s["vd"]
    o = o.view(seqs, hkv, most, ratio, DIM).permute(0, 2, 1, 3, 4)[s["row_seq"], s["row_at"]]
    return o.reshape(-1, hkv * ratio, DIM).bfloat16()


def _grid(s):
    """Tokens and parents on the padded [sequence, node] grid; no node is a child of -2."""
    tokens = s["tokens"].long()[s["grid"]]
    parents = s["parents"].long()[s["grid"]]
    parents = torch.where(s["live"], parents, torch.full_like(parents, -2))
    return tokens, parents


def _emit(path, tokens, count, last):
    """(accepted nodes behind the root's 0, their number, the accepted tokens and the next)."""
    at = torch.arange(NODES, device=DEV)[None, :]
    kept = torch.where(at <= count[:, None], path, torch.full_like(path, -1))
    took = torch.gather(tokens, 1, kept.clamp_min(0).roll(-1, 1))
    out = torch.where(at < count[:, None], took, torch.full_like(took, -1))
    out = torch.where(at == count[:, None], last[:, None], out)
    return kept.to(torch.int32), count.to(torch.int32), out.to(torch.int32)


def _greedy(s):
    top = s["logits"].float().argmax(-1)
    tokens, parents = _grid(s)
    seqs = tokens.shape[0]
    cur = torch.zeros(seqs, dtype=torch.int64, device=DEV)
    count = torch.zeros_like(cur)
    path = torch.zeros(seqs, NODES, dtype=torch.int64, device=DEV)
    for d in range(s["depth"]):
        want = top[s["first"] + cur]
        child = (parents == cur[:, None]) & (tokens == want[:, None])
        found = child.any(1) & (count == d)
        cur = torch.where(found, child.int().argmax(1), cur)
        count = count + found.long()
        path[:, d + 1] = cur
    return _emit(path, tokens, count, top[s["first"] + cur])


def _residual(s, row, scale, dead):
    """What is left of the target's rows: p - scale * q, or p without the tokens in `dead`, in 64 bits."""
    p = s["p"][row].double()
    if s["q"] is not None:
        return (p - scale[:, None] * s["q"][row].double()).clamp_min(0)
    return torch.where(dead, torch.zeros_like(p), p)


def _sample(s):
    """Each node's children are tried in order: child x is taken if u q(x) Z < w(x), where w is
    what the target's row has left and Z its sum (1 before the first refusal); a refusal takes
    Z q from w.  Without a drafter's rows q is 1 at the child's own token.  Where no child is
    left, the next token is drawn from w by its running sum."""
    tokens, parents = _grid(s)
    seqs, vocab = tokens.shape[0], s["p"].shape[1]
    u = s["u"].double()[s["grid"]]
    with_q = s["q"] is not None
    cur = torch.zeros(seqs, dtype=torch.int64, device=DEV)
    count = torch.zeros_like(cur)
    path = torch.zeros(seqs, NODES, dtype=torch.int64, device=DEV)
    live = torch.ones(seqs, dtype=torch.bool, device=DEV)
    scale = torch.zeros(seqs, dtype=torch.float64, device=DEV)
    dead = torch.zeros(seqs, 1 if with_q else vocab, dtype=torch.bool, device=DEV)
    order = torch.arange(NODES, device=DEV)[None, :]
    for d in range(s["depth"]):
        row = s["first"] + cur
        left = torch.ones(seqs, dtype=torch.float64, device=DEV)
        tried = torch.zeros_like(cur)            # children before this one have been refused
        moved = torch.zeros_like(live)
        here = cur
        if not with_q:
            dead = dead & ~live[:, None]
        scale = torch.where(live, torch.zeros_like(scale), scale)
        for _ in range(s["most"]):
            child = (parents == here[:, None]) & (order >= tried[:, None])
            there = child.any(1) & live & ~moved
            i = child.int().argmax(1)
            x = torch.gather(tokens, 1, i[:, None])[:, 0]
            coin = torch.gather(u, 1, i[:, None])[:, 0]
            p = s["p"][row, x].double()
            if with_q:
                q = s["q"][row, x].double()
                w = (p - scale * q).clamp_min(0)
                take = coin * q * left < w
            else:
                gone = torch.gather(dead, 1, x[:, None])[:, 0]
                w = torch.where(gone, torch.zeros_like(p), p)
                take = coin * left < w
            take = take & there
            drop = there & ~take
            if with_q:
                scale = torch.where(drop, scale + left, scale)
                rest = _residual(s, row, scale, dead).sum(-1)
                left = torch.where(drop, rest, left)
            else:
                left = torch.where(drop, left - w, left)
                dead = dead.scatter(1, x[:, None], (torch.gather(dead, 1, x[:, None])[:, 0] | drop)[:, None])
            tried = torch.where(drop, i + 1, tried)
            cur = torch.where(take, i, cur)
            moved = moved | take
        count = count + moved.long()
        path[:, d + 1] = cur
        live = live & moved
    scale = torch.where(live, torch.zeros_like(scale), scale)     # a leaf: nothing was refused
    if not with_q:
        dead = dead & ~live[:, None]
    row = s["first"] + cur
    w = _residual(s, row, scale, dead)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, s["p"][row].double())
    run_ = w.cumsum(-1)
    last = (run_ <= u[:, :1] * run_[:, -1:]).sum(-1)
    last = torch.where(run_[:, -1] > 0, last, torch.full_like(last, -1))
    return _emit(path, tokens, count, last)


def _compact(s):
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    start = (s["lens"].long() - n)[:, None]
    at = torch.arange(NODES, device=DEV)[None, :]
    kept = at <= s["count"].long()[:, None]
    zero = torch.zeros_like(s["index"].long())
    src = start + torch.where(kept, s["index"].long(), zero)
    dst = start + torch.where(kept, at, zero)
    seq = torch.arange(src.shape[0], device=DEV)[:, None]
    sp, dp = s["bt"][seq, src // PAGE].long(), s["bt"][seq, dst // PAGE].long()
    for cache in (s["k"], s["v"]):
        raw = cache.view(torch.uint8)
        raw[:, dp, dst % PAGE] = raw[:, sp, src % PAGE]
    s["new"].copy_(start[:, 0] + 1 + s["count"].long())
    return s["k"], s["v"], s["new"]


def _take_free(ref, want):
    """The lowest free pages for the places that `want` marks, in the places' order; -1 if the
    pool cannot serve them all."""
    order = torch.sort((ref > 0).to(torch.int32), stable=True).indices
    rank = (want.reshape(-1).long().cumsum(0) - 1).reshape(want.shape)
    fits = want.sum() <= (ref == 0).sum()
    page = order[rank.clamp(0, ref.numel() - 1)].to(torch.int32)
    return torch.where(want & fits, page, torch.full_like(page, -1)), fits


def _copy_pages(s, src, dst, on):
    """Pages src -> dst in every layer, where `on`; the others copy page 0 onto itself."""
    held = torch.where(on, src, torch.zeros_like(src)).long()
    to = torch.where(on, dst, torch.zeros_like(dst)).long()
    for cache in (s["k"], s["v"]):
        raw = cache.view(torch.uint8)
        # page 0 may also be a real target: rows that copy nothing write what that will hold
        data = raw[:, held]
        into0 = on & (to == 0)
        first = torch.where(into0.any(), held[into0.int().argmax()], torch.zeros_like(held[0]))
        data = torch.where(on[None, :, None, None, None], data, raw[:, first][:, None])
        raw[:, to] = data


def _resize(s, new):
    bt, ref, lens = s["bt"], s["ref"], s["lens"]
    at = torch.arange(bt.shape[1], device=DEV)[None, :]
    old_p, new_p = (lens[:, None] + PAGE - 1) // PAGE, (new[:, None] + PAGE - 1) // PAGE
    drop = (at >= new_p) & (at < old_p)
    ref.index_add_(0, bt.clamp_min(0).reshape(-1).long(), -drop.reshape(-1).to(torch.int32))
    bt.masked_fill_(drop, -1)
    kept = torch.minimum(lens, new)
    tail = ((kept - 1).clamp_min(0) // PAGE).long()[:, None]
    page = torch.gather(bt, 1, tail)[:, 0]
    part = (kept % PAGE != 0) & (ref[page.clamp_min(0).long()] > 1)
    want = ((at >= old_p) & (at < new_p)) | ((at == tail) & part[:, None])
    got, fits = _take_free(ref, want)
    part = part & fits
    _copy_pages(s, page, torch.gather(got, 1, tail)[:, 0], part)
    ref.index_add_(0, page.clamp_min(0).long(), -part.to(torch.int32))
    ref.index_add_(0, got.clamp_min(0).reshape(-1).long(), (got >= 0).reshape(-1).to(torch.int32))
    bt.copy_(torch.where(got >= 0, got, bt))
    lens.copy_(torch.where(fits, new, kept))


def _fork(s, src, dst):
    bt, ref, lens = s["bt"], s["ref"], s["lens"]
    src, dst = src.long(), dst.long()
    at = torch.arange(bt.shape[1], device=DEV)[None, :]
    n = lens[src]
    part = n % PAGE != 0
    whole = (n // PAGE)[:, None]
    share = at < whole
    got, fits = _take_free(ref, (at == whole) & part[:, None])
    row = torch.where(share, bt[src], got)
    at_tail = (n // PAGE).clamp_max(bt.shape[1] - 1).long()[:, None]
    _copy_pages(s, torch.gather(bt[src], 1, at_tail)[:, 0], torch.gather(got, 1, at_tail)[:, 0],
                part & fits)
    ref.index_add_(0, row.clamp_min(0).reshape(-1).long(),
                   ((row >= 0) & fits).reshape(-1).to(torch.int32))
    bt[dst] = torch.where(fits, row, bt[dst])
    lens[dst] = torch.where(fits, n, lens[dst])


def _pages(s):
    _resize(s, s["keep"])
    _fork(s, s["src"], s["dst"])
    _resize(s, s["held"])
    return s["k"], s["v"], s["bt"], s["lens"], s["ref"]


# ---- 64 bits -----------------------------------------------------------------------------------


def exact(case, seed):
    op = case["op"]
    if op in ("compact", "pages"):
        return None                    # moved codes and counts: nothing is rounded
    s = prepare(case, seed)
    if op == "attn":
        hkv, ratio = case["hkv"], case["ratio"]
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        cu = _cu(_ints(case, "nodes"))
        for b, (ln, n) in enumerate(zip(_ints(case, "lens"), _ints(case, "nodes"))):
            pos = torch.arange(ln, device=DEV)
            page = s["bt"][b].long()[pos // PAGE]
            see = torch.ones(n, ln, dtype=torch.bool, device=DEV)
            words = s["mask"][cu[b]:cu[b + 1]]
            for j in range(n):
                see[:, ln - n + j] = ((words >> j) & 1).bool()
            for h in range(hkv):
                key = _rows(s["k"], page, pos % PAGE)[:, h].double() * s["kd"].double()
                val = _rows(s["v"], page, pos % PAGE)[:, h].double() * s["vd"].double()
                q = s["q"][cu[b]:cu[b + 1], h * ratio:(h + 1) * ratio].double().reshape(n * ratio, DIM)
                logit = q @ key.T * s["scale"]
                logit[~see.repeat_interleave(ratio, 0)] = -math.inf
                out[cu[b]:cu[b + 1], h * ratio:(h + 1) * ratio] = \
                    (torch.softmax(logit, -1) @ val).reshape(n, ratio, DIM)
        return out
    cu = _cu(_ints(case, "nodes"))
    index = torch.full((len(_ints(case, "nodes")), NODES), -1, dtype=torch.int32)
    said = torch.full_like(index, -1)
    count = torch.zeros(len(_ints(case, "nodes")), dtype=torch.int32)
    tokens, parents = s["tokens"].tolist(), s["parents"].tolist()
    us = s["u"].tolist() if op == "sample" else None
    for b, n in enumerate(_ints(case, "nodes")):
        at, path = 0, [0]
        tok, par = tokens[cu[b]:cu[b + 1]], parents[cu[b]:cu[b + 1]]
        while True:
            sons = [i for i in range(1, n) if par[i] == at]
            nxt = None
            if op == "greedy":
                row = s["logits"][cu[b] + at].double()
                last = int((row == row.max()).nonzero()[0, 0])
                nxt = next((i for i in sons if tok[i] == last), None)
            else:
                w = s["p"][cu[b] + at].double()
                q = s["q"][cu[b] + at].double() if s["q"] is not None else None
                mass = 1.0
                for i in sons:
                    qi = q if q is not None else None
                    qx = float(q[tok[i]]) if q is not None else 1.0
                    if us[cu[b] + i] * qx * mass < float(w[tok[i]]):
                        nxt = i
                        break
                    if qi is not None:
                        w = (w - mass * qi).clamp_min(0)
                        mass = float(w.sum())
                    else:
                        mass -= float(w[tok[i]])
                        w = w.clone()
                        w[tok[i]] = 0
                if nxt is None:
                    if not float(w.sum()) > 0:
                        w = s["p"][cu[b] + at].double()
                    acc = torch.cumsum(w, 0)
                    last = int((acc > us[cu[b]] * float(acc[-1])).nonzero()[0, 0])
            if nxt is None:
                break
            at = nxt
            path.append(at)
        index[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        count[b] = len(path) - 1
        said[b, :len(path)] = torch.tensor([tok[i] for i in path[1:]] + [last], dtype=torch.int32)
    return index.to(DEV), count.to(DEV), said.to(DEV)
