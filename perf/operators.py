"""The operators of the attention layers beside the recurrent ones, as measured cases.

An attention layer of a decode loop with drafts keeps its keys and values in pages.
Four operators work on them, each in its plain form (elementary torch operations in
fp32) and through the package's entry points:

* stage   -- per-head RMSNorm of queries and keys, position rotation, keys and values
             written to their pages;
* verify  -- attention of a block of drafted tokens (a chain or a tree) over the pages;
* accept  -- the accepted path of a tree moved to the front of the draft's rows in every
             layer's cache, and the new lengths;
* pages   -- fork of sequences (shared full pages, copied last page), room reserved for
             the next draft, release.

``own`` selects which of the two ``run`` computes.
"""
import math

import numpy as np
import torch

own = False

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------- cases
def _stage(name, B, T, Hq, Hkv, d, rot, style, page, lo, hi, dl, dtype, packed):
    return dict(name=name, op="stage", B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, rot=rot, style=style, page=page,
                len_lo=lo, len_hi=hi, draft_lo=dl, dtype=dtype, packed=packed)


def _verify(name, B, T, Hq, Hkv, d, page, lo, hi, dl, tree, dtype):
    return dict(name=name, op="verify", B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, page=page, len_lo=lo, len_hi=hi,
                draft_lo=dl, tree=tree, dtype=dtype)


def _accept(name, B, T, Hkv, d, page, layers, lo, hi, dtype):
    return dict(name=name, op="accept", B=B, T=T, Hkv=Hkv, d=d, page=page, layers=layers, len_lo=lo,
                len_hi=hi, dtype=dtype)


def _pages(name, sources, forks, T, Hkv, d, page, layers, lo, hi, dtype):
    return dict(name=name, op="pages", sources=sources, forks=forks, T=T, Hkv=Hkv, d=d, page=page,
                layers=layers, len_lo=lo, len_hi=hi, dtype=dtype)


def listed():
    return [
        # the decode sweep's block (B 32, T 16, 16 heads of 128): one step's queries, keys and values
        _stage("stage block", 32, 16, 16, 2, 128, 128, "half", 16, 900, 8000, 16, "bf16", True),
        # prompts of ragged lengths entering the cache, wide heads of which a quarter is rotated
        _stage("stage prompts", 6, 4096, 16, 2, 256, 64, "half", 64, 0, 0, 1500, "bf16", True),
        # one user, one token: the call's latency
        _verify("verify one token", 1, 1, 16, 2, 128, 16, 700, 700, 1, "chain", "bf16"),
        # the decode sweep's block over ragged contexts
        _verify("verify chains", 32, 16, 16, 2, 128, 16, 900, 8000, 16, "chain", "bf16"),
        # wide trees of up to 48 drafted tokens, several row tiles per key head
        _verify("verify trees", 12, 48, 32, 4, 128, 64, 1500, 6000, 31, "tree", "bf16"),
        # one user with a very long context: the work is split along the keys
        _verify("verify long", 1, 16, 16, 2, 128, 64, 131001, 131001, 16, "tree", "bf16"),
        # many users, wide heads, short drafts: the most keys and values
        _verify("verify many", 128, 8, 16, 2, 256, 32, 500, 3500, 5, "tree", "bf16"),
        # full precision at the small head size, odd lengths
        _verify("verify fp32", 5, 7, 12, 3, 64, 16, 333, 2100, 3, "tree", "fp32"),
        # one decode step's accept over the attention layers of a small stack
        _accept("accept block", 32, 16, 2, 128, 16, 6, 900, 4000, "bf16"),
        # wide trees, many sequences and layers
        _accept("accept trees", 96, 64, 4, 128, 64, 12, 300, 700, "bf16"),
        # one conversation continued four ways
        _pages("fork one", 1, 4, 16, 2, 128, 16, 6, 1001, 1001, "bf16"),
        # parallel samples of several prompts over a whole stack
        _pages("fork many", 16, 64, 16, 2, 128, 64, 24, 700, 2100, "bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["stage", "verify", "verify", "accept", "pages"])
        d = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 2, 3, 4, 8])
        G = rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
        page = rng.choice([16, 16, 32, 64, 128])
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        if 3072 in (Hkv * G * d, Hkv * (G + 2) * d, Hkv * d, Hkv * G, page * d):
            continue
        if op == "stage":
            B, T = spread(1, 64), spread(1, 4096)
            lo = spread(1, 2000)
            c = _stage("", B, T, Hkv * G, Hkv, d, rng.choice([d, d // 2, d // 4]), rng.choice(["half", "pairs"]),
                       page, lo, lo + spread(1, 2000), rng.randint((T + 1) // 2, T), dtype, rng.random() < 0.5)
            most = 0.37e9
        elif op == "verify":
            B, T = spread(1, 128), rng.randint(1, 64)
            lo = spread(1, 20000)
            hi = lo + spread(1, 8000)
            c = _verify("", B, T, Hkv * G, Hkv, d, page, lo, hi, rng.randint((T + 1) // 2, T),
                        rng.choice(["chain", "tree"]), dtype)
            most = 0.5e9
            if c["dtype"] == "fp32" and work(c)["flops"] > 6e9:
                continue
        elif op == "accept":
            lo = spread(1, 1000)
            c = _accept("", spread(1, 96), rng.randint(2, 64), min(Hkv, 4), min(d, 128), page, rng.randint(1, 12),
                        lo, lo + spread(1, 400), dtype)
            most = 0.4e9
        else:
            lo = spread(1, 1500)
            src = spread(1, 16)
            c = _pages("", src, src * rng.randint(1, 4), rng.randint(1, 64), min(Hkv, 4), min(d, 128), page,
                       rng.randint(1, 24), lo, lo + spread(1, 600), dtype)
            most = 0.4e9
        if 3072 in c.values() or _cache_bytes(c) > 1.6e9 or work(c)["bytes"] > most or work(c)["flops"] > 30e9:
            continue
        del c["name"]
        return c


def _fill(n, lo, hi, k):
    """n whole numbers spread over [lo, hi], the same for every seed."""
    return [lo + int((hi - lo + 0.999) * ((i * 0.6180339887 + 0.37 * k) % 1.0)) if hi > lo else lo for i in range(n)]


def _lens(c):
    return _fill(c["sources"] if c["op"] == "pages" else c["B"], c["len_lo"], c["len_hi"], 1)


def _drafts(c):
    return _fill(c["B"], c["draft_lo"], c["T"], 2)


def _paths(c):
    return [min(c["T"], max(0, p)) for p in _fill(c["B"], 0, c["T"], 3)]


def _size(c):
    return 2 if c["dtype"] == "bf16" else 4


def _max_pages(c):
    return -(-(c["len_hi"] + c["T"]) // c["page"])


def _n_page(c):
    n = sum(-(-(x + c["T"]) // c["page"]) for x in _lens(c)) + 3
    if c["op"] == "pages":
        n += c["forks"] * (2 + -(-c["T"] // c["page"]))
    return n


def _cache_bytes(c):
    return 2 * c.get("layers", 1) * _n_page(c) * c["Hkv"] * c["page"] * c["d"] * _size(c)


def work(c):
    e, d, lens = _size(c), c["d"], _lens(c)
    if c["op"] == "stage":
        n = sum(_drafts(c))
        return {"bytes": 2 * n * (c["Hq"] + 2 * c["Hkv"]) * d * e + 4 * n, "flops": 10 * n * (c["Hq"] + c["Hkv"]) * d}
    if c["op"] == "verify":
        keys = [x + y for x, y in zip(lens, _drafts(c))]
        rows = [y * c["Hq"] for y in _drafts(c)]
        return {"bytes": sum(2 * k * c["Hkv"] * d * e for k in keys) + sum(r * (2 * d * e + 4) for r in rows),
                "flops": sum(4 * r * k * d for r, k in zip(rows, keys))}
    if c["op"] == "accept":
        row = c["layers"] * 2 * c["Hkv"] * d * e
        return {"bytes": 2 * row * sum(max(0, p - 1) for p in _paths(c)) + 8 * sum(_paths(c)) + 12 * c["B"], "flops": 0}
    page = c["layers"] * 2 * c["Hkv"] * c["page"] * d * e
    src = [i % c["sources"] for i in range(c["forks"])]
    tails = sum(1 for i in src if lens[i] % c["page"])
    shared = sum(lens[i] // c["page"] for i in src)
    new = sum(-(-(lens[i] + c["T"]) // c["page"]) - lens[i] // c["page"] for i in src)
    # fork: the shared entries read, written and counted up; reserve and release: entries, counts, free list
    return {"bytes": 2 * tails * page + 4 * (shared * (1 + 1 + 2 + 1 + 2) + new * (1 + 1 + 1 + 1 + 2 + 1)), "flops": 0}


# ------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _pool(c, g, owned, lens, n_slot, spread_v=1.0):
    """Keys and values of every page and the pool's bookkeeping: sequence i owns owned[i]
    pages of a random order, the rest are free."""
    n_page, mp, L = _n_page(c), _max_pages(c), c.get("layers", 1)
    shape = (L, n_page, c["Hkv"], c["page"], c["d"])
    dt = TORCH[c["dtype"]]
    order = torch.randperm(n_page, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n_slot, mp), -1, dtype=torch.int32, device="cuda")
    own_t = torch.tensor(owned, dtype=torch.int64, device="cuda")
    first = torch.cumsum(own_t, 0) - own_t
    col = torch.arange(mp, device="cuda")[None]
    rows = order[(first[:, None] + col).clamp(max=n_page - 1)]
    table[:len(owned)] = torch.where(col < own_t[:, None], rows, table[:len(owned)])
    used = sum(owned)
    ref = torch.zeros(n_page, dtype=torch.int32, device="cuda")
    ref[order[:used].long()] = 1
    free = torch.zeros(n_page, dtype=torch.int32, device="cuda")
    free[:n_page - used] = order[used:]
    zeros = [0] * (n_slot - len(owned))
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(k=_randn(g, *shape, scale=1.4, dtype=dt), v=_randn(g, *shape, scale=spread_v, dtype=dt),
                block_table=table, seq_len=torch.tensor(lens + zeros, **i32),
                n_owned=torch.tensor(owned + zeros, **i32), ref=ref, free_list=free,
                free_count=torch.tensor([n_page - used], **i32))


def _parents(c, g):
    """Parents of T drafted tokens per sequence: token 0 is the root, each other token hangs
    from one of the few before it (drafts of several candidates per step)."""
    B, T = c["B"], c["T"]
    t = torch.arange(T, device="cuda")
    back = 1 + (torch.rand(B, T, generator=g, device="cuda") * 4).long()
    return torch.where(t == 0, -1, (t - back).clamp(min=0)).to(torch.int32)


def _ancestors(parents):
    """[B, T, T] truth values (u is t or an ancestor of t) and depths [B, T]."""
    B, T = parents.shape
    m = torch.zeros(B, T, T, dtype=torch.bool, device=parents.device)
    depth = torch.zeros(B, T, dtype=torch.int64, device=parents.device)
    rows = torch.arange(B, device=parents.device)
    for t in range(T):
        p = parents[:, t].long()
        has = p >= 0
        m[:, t] = m[rows, p.clamp(min=0)] & has[:, None]
        m[:, t, t] = True
        depth[:, t] = torch.where(has, depth[rows, p.clamp(min=0)] + 1, 0)
    return m, depth


def _bits(m):
    """[B, T, T] truth values -> one 64-bit word per row (bit u = column u)."""
    w = torch.ones(m.shape[-1], dtype=torch.int64, device=m.device) << torch.arange(m.shape[-1], device=m.device)
    return (m.to(torch.int64) * w).sum(-1)


def _tables(c, max_pos):
    """cos | sin of each position, fp32 [max_pos, rot], from 64-bit angles."""
    h = c["rot"] // 2
    f = 10000.0 ** (-torch.arange(h, dtype=torch.float64, device="cuda") / h)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt, lens = TORCH[c["dtype"]], _lens(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case=dict(c))
    if c["op"] in ("stage", "verify"):
        B, T, Hq, Hkv, d = (c[n] for n in ("B", "T", "Hq", "Hkv", "d"))
        owned = [-(-(x + T) // c["page"]) for x in lens]
        s["t"] = t = _pool(c, g, owned, lens, B)
        s["draft_len"] = torch.tensor(_drafts(c), **i32)
        max_pos = c["len_hi"] + T
        if c["op"] == "stage":
            s["q_weight"], s["k_weight"] = 1 + _randn(g, d, scale=0.2), 1 + _randn(g, d, scale=0.2)
            width = [Hq * d, Hkv * d, Hkv * d]
            scale = torch.exp2(2 * torch.rand(B, T, 1, generator=g, device="cuda") - 1)
            if c["packed"]:                                # the output of one projection
                qkv = (_randn(g, B, T, sum(width)) * scale).to(dt)
                parts = qkv.split(width, -1)
            else:
                parts = [(_randn(g, B, T, w) * scale).to(dt) for w in width]
            s["q"], s["k"], s["v"] = (p.unflatten(-1, (-1, d)) for p in parts)
            s["cos_sin"] = _tables(c, max_pos)
            s["q_out"] = torch.zeros(B, T, Hq, d, dtype=dt, device="cuda")
            s["pos"] = (t["seq_len"][:, None] + torch.arange(T, **i32)).contiguous()
        else:
            s["q"] = _randn(g, B, T, Hq, d, scale=1.4, dtype=dt)
            if c["tree"] == "tree":
                m, _ = _ancestors(_parents(c, g))
                s["tree"], s["seen"] = _bits(m), m
            else:
                s["tree"], s["seen"] = None, torch.ones(T, T, dtype=torch.bool, device="cuda").tril()[None]
            s["out"] = torch.zeros(B, T, Hq, d, dtype=dt, device="cuda")
            s["lse"] = torch.zeros(B, T, Hq, device="cuda")
        if own:
            import speculative_decode_recurrent_gb300 as lib
            cache = lib.PagedCache(_page_dims(lib, c, B), t)
            dims = lib.AttnDims(B=B, T=T, Hq=Hq, scale=d ** -0.5)
            if c["op"] == "stage":
                rope = lib.RopeDims(rot=c["rot"], style=lib.ROPE_PAIRS if c["style"] == "pairs" else lib.ROPE_HALF,
                                    max_pos=max_pos, eps=1e-6)
                s["layer"] = lib.AttnLayer(dims, cache, 0, rope, s["q_weight"], s["k_weight"], s["cos_sin"])
            else:
                s["layer"] = lib.AttnLayer(dims, cache, 0)
    elif c["op"] == "accept":
        owned = [-(-(x + c["T"]) // c["page"]) for x in lens]
        s["t"] = t = _pool(c, g, owned, lens, c["B"])
        # the accepted path: token 0, then ever later tokens of the draft
        r = torch.rand(c["B"], c["T"], generator=g, device="cuda")
        take = torch.tensor(_paths(c), device="cuda")
        r[:, 0] = -1.0
        rank = r.argsort(1).argsort(1)
        s["path"] = torch.where(rank < take[:, None], torch.arange(c["T"], device="cuda"), c["T"]).sort(1)[0].to(torch.int32)
        s["accepted"] = take.to(torch.int32)
        s["new_len"] = torch.zeros_like(t["seq_len"])
        if own:
            import speculative_decode_recurrent_gb300 as lib
            s["cache"] = lib.PagedCache(_page_dims(lib, c, c["B"]), t)
    else:
        owned = [-(-x // c["page"]) for x in lens]
        n_slot = c["sources"] + c["forks"]
        s["t"] = _pool(c, g, owned, lens, n_slot)
        s["src"] = (torch.arange(c["forks"], **i32) % c["sources"]).contiguous()
        s["dst"] = torch.arange(c["sources"], n_slot, **i32)
        s["copies"] = torch.zeros(c["forks"], 2, **i32)
        if own:
            import speculative_decode_recurrent_gb300 as lib
            s["cache"] = lib.PagedCache(_page_dims(lib, c, n_slot), s["t"])
    return s


def _page_dims(lib, c, n_slot):
    return lib.PageDims(n_slot=n_slot, max_pages=_max_pages(c), n_page=_n_page(c), page=c["page"],
                        n_layer=c.get("layers", 1), Hkv=c["Hkv"], d=c["d"],
                        dtype=lib.DTYPE_BF16 if c["dtype"] == "bf16" else lib.DTYPE_F32)


# ------------------------------------------------------------------- plain forms
def _rotate(y, cs, rot, style):
    h = rot // 2
    cos, sin = cs[..., :h], cs[..., h:]
    if style == "half":
        a, b = y[..., :h], y[..., h:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _norm(x, w, eps=1e-6):
    x = x.float()
    return x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w


def _rows(t, T, page, slots=None):
    """Page and row within it of the T tokens past each sequence's length."""
    p = t["seq_len"].long()[:, None] + torch.arange(T, device="cuda")
    return t["block_table"].long().gather(1, p // page), p % page


def _plain_stage(s):
    c, t = s["case"], s["t"]
    cs = s["cos_sin"][s["pos"].long()][:, :, None]
    live = (torch.arange(c["T"], device="cuda") < s["draft_len"][:, None])[..., None, None]
    dt = TORCH[c["dtype"]]
    q = _rotate(_norm(s["q"], s["q_weight"]), cs, c["rot"], c["style"]).to(dt)
    k = _rotate(_norm(s["k"], s["k_weight"]), cs, c["rot"], c["style"]).to(dt)
    s["q_out"].copy_(torch.where(live, q, torch.zeros_like(q)))
    pg, off = _rows(t, c["T"], c["page"])
    kc, vc = t["k"][0], t["v"][0]
    kc[pg, :, off] = torch.where(live, k, kc[pg, :, off])
    vc[pg, :, off] = torch.where(live, s["v"], vc[pg, :, off])
    return {"q": s["q_out"], "k": kc, "v": vc}


def _plain_verify(s):
    c, t = s["case"], s["t"]
    B, T, Hq, Hkv, d, G = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], c["Hq"] // c["Hkv"]
    tab = t["block_table"].long().clamp(min=0)
    k = t["k"][0][tab].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    v = t["v"][0][tab].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    n = k.shape[2]
    q = s["q"].float().reshape(B, T, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, T * G, d)
    x = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    j = torch.arange(n, device="cuda") - t["seq_len"][:, None]          # < 0: committed, else draft token
    live = torch.arange(T, device="cuda") < s["draft_len"][:, None]
    seen = s["seen"].expand(B, T, T).gather(2, j.clamp(0, T - 1)[:, None].expand(B, T, n))
    seen = torch.where((j < 0)[:, None], True, seen & (j < s["draft_len"][:, None])[:, None]) & live[..., None]
    seen = seen[:, None, :, None].expand(B, Hkv, T, G, n).reshape(B, Hkv, T * G, n)
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / l.clamp(min=1e-37)
    lse = (m + torch.log(l)).reshape(B, Hkv, T, G).transpose(1, 2).reshape(B, T, Hq)
    o = o.reshape(B, Hkv, T, G, d).transpose(1, 2).reshape(B, T, Hq, d)
    return {"out": o.to(TORCH[c["dtype"]]), "lse": lse}


def _plain_accept(s):
    c, t = s["case"], s["t"]
    pg, off = _rows(t, c["T"], c["page"])
    at = s["path"].long().clamp(max=c["T"] - 1)
    take = (torch.arange(c["T"], device="cuda") < s["accepted"][:, None])[..., None, None, None]
    for x in (t["k"], t["v"]):
        x[:, pg, :, off] = torch.where(take, x[:, pg.gather(1, at), :, off.gather(1, at)], x[:, pg, :, off])
    s["new_len"].copy_(t["seq_len"] + s["accepted"])
    return {"k": t["k"], "v": t["v"], "len": s["new_len"]}


def _take_pages(t, need):
    """Which rows get their pages (in order, while there are some), how many lie before
    each row, and the new free count."""
    incl = torch.cumsum(need, 0)
    ok = (need == 0) | (incl <= t["free_count"])
    give = torch.where(ok, need, 0)
    return ok, give, incl - need


def _plain_fork(s):
    c, t = s["case"], s["t"]
    src, dst, page = s["src"].long(), s["dst"].long(), c["page"]
    ln = t["seq_len"].long()[src]
    full = ln // page
    ok, give, before = _take_pages(t, (ln % page > 0).long())
    new = t["free_list"].long()[(t["free_count"] - 1 - before).clamp(min=0).long()]
    col = torch.arange(t["block_table"].shape[1], device="cuda")[None]
    old = t["block_table"].long()[src]
    shared = (col < full[:, None]) & ok[:, None]
    tail = (col == full[:, None]) & (give > 0)[:, None]
    t["block_table"][dst] = torch.where(shared, old, torch.where(tail, new[:, None], t["block_table"].long()[dst])).to(torch.int32)
    t["ref"].index_add_(0, old.clamp(min=0).flatten(), shared.flatten().to(torch.int32))
    t["ref"].index_add_(0, new, give.to(torch.int32))
    t["free_count"] -= give.sum().to(torch.int32)
    t["seq_len"][dst] = torch.where(ok, ln, t["seq_len"].long()[dst]).to(torch.int32)
    t["n_owned"][dst] = torch.where(ok, full + give, t["n_owned"].long()[dst]).to(torch.int32)
    last = old.gather(1, full.clamp(max=old.shape[1] - 1)[:, None])[:, 0]
    pair = torch.stack([torch.where(give > 0, last, -1), torch.where(give > 0, new, -1)], 1)
    s["copies"].copy_(pair)
    # the last pages' keys and values, in every layer; a row without one rewrites a page it shares
    a, b = torch.where(give > 0, last, old[:, 0]), torch.where(give > 0, new, old[:, 0])
    for x in (t["k"], t["v"]):
        x[:, b] = x[:, a]


def _plain_reserve(s):
    c, t = s["case"], s["t"]
    rows, page = s["dst"].long(), c["page"]
    own_n = t["n_owned"].long()[rows]
    need = ((t["seq_len"].long()[rows] + c["T"] + page - 1) // page - own_n).clamp(min=0)
    _, give, before = _take_pages(t, need)
    col = torch.arange(t["block_table"].shape[1], device="cuda")[None]
    k = before[:, None] + col - own_n[:, None]
    new = t["free_list"].long()[(t["free_count"] - 1 - k).clamp(0, t["free_list"].numel() - 1).long()]
    get = (col >= own_n[:, None]) & (col < (own_n + give)[:, None])
    t["block_table"][rows] = torch.where(get, new, t["block_table"].long()[rows]).to(torch.int32)
    t["ref"].index_add_(0, new.flatten(), get.flatten().to(torch.int32))
    t["free_count"] -= give.sum().to(torch.int32)
    t["n_owned"][rows] = (own_n + give).to(torch.int32)


def _plain_release(s):
    t = s["t"]
    rows = s["dst"].long()
    tab = t["block_table"].long()[rows]
    col = torch.arange(tab.shape[1], device="cuda")[None]
    mine = (col < t["n_owned"].long()[rows][:, None]).flatten()
    pg = tab.clamp(min=0).flatten()
    t["ref"].index_add_(0, pg, -mine.to(torch.int32))
    n = t["ref"].numel()
    order = torch.arange(1, pg.numel() + 1, device="cuda")
    gone = mine & (t["ref"][pg] == 0)
    last = torch.zeros(n, dtype=torch.int64, device="cuda").scatter_reduce(0, pg, torch.where(gone, order, 0), "amax")
    win = gone & (last[pg] == order)
    at = torch.where(win, t["free_count"].long() + torch.cumsum(win.long(), 0) - 1, n)
    more = torch.cat([t["free_list"], t["free_list"][:1]]).scatter(0, at, pg.to(torch.int32))
    t["free_list"].copy_(more[:n])
    t["free_count"] += win.sum().to(torch.int32)
    t["seq_len"][rows] = 0
    t["n_owned"][rows] = 0


def _pool_state(s):
    t = s["t"]
    return {n: t[n] for n in ("k", "v", "block_table", "seq_len", "n_owned", "ref", "free_list", "free_count")} | {"copies": s["copies"]}


def run(s):
    op, t = s["case"]["op"], s["t"]
    if not own:
        if op == "stage":
            return _plain_stage(s)
        if op == "verify":
            return _plain_verify(s)
        if op == "accept":
            return _plain_accept(s)
        _plain_fork(s)
        _plain_reserve(s)
        _plain_release(s)
        return _pool_state(s)
    if op == "stage":
        s["layer"].stage(s["q"], s["k"], s["v"], s["q_out"], pos=s["pos"], draft_len=s["draft_len"])
        return {"q": s["q_out"], "k": t["k"][0], "v": t["v"][0]}
    if op == "verify":
        s["layer"].verify(s["q"], s["out"], lse=s["lse"], tree=s["tree"], draft_len=s["draft_len"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "accept":
        s["cache"].accept(s["accepted"], path=s["path"], new_len=s["new_len"])
        return {"k": t["k"], "v": t["v"], "len": s["new_len"]}
    s["cache"].fork(s["src"], s["dst"], s["copies"])
    s["cache"].reserve(s["dst"], s["case"]["T"])
    s["cache"].release(s["dst"])
    return _pool_state(s)


# ------------------------------------------------------------------ 64-bit values
def _np(x):
    return x.detach().cpu().double().numpy()


def _exact_rows(x, w, pos, c):
    """x [T, H, d] normalised per head, weighted, and turned by its position's angle; the
    angles' cosines and sines are the tables' (inputs)."""
    cos, sin = pos[:, None, :c["rot"] // 2], pos[:, None, c["rot"] // 2:]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * w
    r = y.copy()
    if c["style"] == "half":
        i = np.arange(c["rot"] // 2)
        j = i + c["rot"] // 2
    else:
        i = np.arange(0, c["rot"], 2)
        j = i + 1
    r[..., i] = y[..., i] * cos - y[..., j] * sin
    r[..., j] = y[..., j] * cos + y[..., i] * sin
    return r


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    t = s["t"]
    tab, ln = t["block_table"].cpu().numpy(), t["seq_len"].cpu().numpy()
    page, op = c["page"], c["op"]
    if op == "stage":
        q, k, v, cs = _np(s["q"]), _np(s["k"]), _np(s["v"]), _np(s["cos_sin"])
        kc, vc, out = _np(t["k"][0]), _np(t["v"][0]), np.zeros_like(q)
        wq, wk = _np(s["q_weight"]), _np(s["k_weight"])
        for b, n in enumerate(_drafts(c)):
            rows = cs[ln[b]:ln[b] + n]
            out[b, :n] = _exact_rows(q[b, :n], wq, rows, c)
            at = ln[b] + np.arange(n)
            kc[tab[b, at // page], :, at % page] = _exact_rows(k[b, :n], wk, rows, c)
            vc[tab[b, at // page], :, at % page] = v[b, :n]
        return {"q": out, "k": kc, "v": vc}
    if op == "verify":
        if work(c)["flops"] > 60e9:
            return None
        B, T, Hq, Hkv, d = (c[n] for n in ("B", "T", "Hq", "Hkv", "d"))
        G = Hq // Hkv
        seen = s["seen"].expand(B, T, T).cpu().numpy()
        out, lse = np.zeros((B, T, Hq, d)), np.full((B, T, Hq), -np.inf)
        for b, n in enumerate(_drafts(c)):
            m = ln[b] + n
            pages = torch.as_tensor(tab[b, :-(-m // page)].astype(np.int64), device="cuda")
            k, v = (_np(t[x][0][pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :m]) for x in ("k", "v"))
            q = _np(s["q"][b, :n])
            mask = np.ones((n, m), dtype=bool)
            mask[:, ln[b]:] = seen[b, :n, :n]
            mask = np.repeat(mask, G, 0)                                 # rows (t, g)
            for h in range(Hkv):
                x = q[:, h * G:(h + 1) * G].reshape(n * G, d) @ k[h].T / math.sqrt(d)
                x = np.where(mask, x, -np.inf)
                top = x.max(1, keepdims=True)
                np.subtract(x, top, out=x)
                e = np.exp(x, out=x)
                den = e.sum(1, keepdims=True)
                out[b, :n, h * G:(h + 1) * G] = (e @ v[h] / den).reshape(n, G, d)
                lse[b, :n, h * G:(h + 1) * G] = (top + np.log(den)).reshape(n, G)
        return {"out": out, "lse": lse}
    if op == "accept":
        k, v = t["k"].clone(), t["v"].clone()
        path = s["path"].cpu().numpy()
        for b, p in enumerate(_paths(c)):
            a, z = ln[b] + path[b, :p].astype(np.int64), ln[b] + np.arange(p)
            for x in (k, v):
                was = x[:, tab[b, a // page].tolist(), :, (a % page).tolist()].clone()
                x[:, tab[b, z // page].tolist(), :, (z % page).tolist()] = was
        return {"k": k, "v": v, "len": None}
    # sequences are forked one by one; the pages they take come off the end of the free list
    free = t["free_list"][:int(t["free_count"])].tolist()
    for a in s["src"].tolist():
        if ln[a] % page:
            new = free.pop()
            for x in (t["k"], t["v"]):
                x[:, new] = x[:, int(tab[a, ln[a] // page])]
    return {"k": t["k"], "v": t["v"], "block_table": None, "seq_len": None, "n_owned": None, "ref": None,
            "free_list": None, "free_count": None, "copies": None}
