"""What comes before the decode loop and what closes each of its steps, as measured cases.

Four operators, each in its plain form (elementary torch operations) and through the
package's entry points:

* advance -- the gated delta rule over committed tokens (a prompt, a chunk of one, a single
             token): outputs of every token, the checkpoint moved on in place;
* conv    -- the short causal convolution before it, over the same tokens, and its ring;
* chunk   -- attention of a chunk of new tokens over a paged cache that holds them already;
* sample  -- drafted tokens (a chain or a tree) verified against the target's probabilities
             with given random numbers: the accepted path and the next token.

``own`` selects which of the two ``run`` computes.
"""
import math

import torch

own = False

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------- cases
def _advance(name, B, T, lo, H, Hk, dk, dv, fresh, dtype):
    return dict(name=name, op="advance", B=B, T=T, len_lo=lo, H=H, Hk=Hk, dk=dk, dv=dv, fresh=fresh, dtype=dtype)


def _conv(name, B, T, lo, D, W, silu, fresh, dtype):
    return dict(name=name, op="conv", B=B, T=T, len_lo=lo, D=D, W=W, silu=silu, fresh=fresh, dtype=dtype)


def _chunk(name, B, T, lo, Hq, Hkv, d, page, past_lo, past_hi, dtype):
    return dict(name=name, op="chunk", B=B, T=T, len_lo=lo, Hq=Hq, Hkv=Hkv, d=d, page=page, past_lo=past_lo,
                past_hi=past_hi, dtype=dtype)


def _sample(name, B, T, lo, V, shape, drafter):
    return dict(name=name, op="sample", B=B, T=T, len_lo=lo, V=V, shape=shape, drafter=drafter)


def listed():
    return [
        # one user, one token without a draft: the call's latency
        _advance("advance one token", 1, 1, 1, 16, 16, 128, 128, "none", "bf16"),
        # prompts of ragged lengths entering the decode sweep's layer (16 heads of 128), some slots new
        _advance("advance prompts", 8, 2048, 700, 16, 16, 128, 128, "some", "bf16"),
        # one user with a long prompt: few independent rows, a long axis
        _advance("advance long", 1, 8192, 8192, 16, 16, 128, 128, "all", "bf16"),
        # full precision at the small head size, two value heads per key head, odd lengths
        _advance("advance fp32", 5, 333, 61, 6, 3, 64, 64, "some", "fp32"),
        # the convolution of the same prompts: q, k and v of 16 heads side by side
        _conv("conv prompts", 8, 2048, 700, 6144, 4, True, "some", "bf16"),
        # a short last chunk, odd channel count, another width
        _conv("conv tail", 2, 65, 33, 200, 3, False, "none", "fp32"),
        # prompts from their first token, ragged (16 query heads, 2 key heads of 128)
        _chunk("chunk prompts", 4, 4096, 2500, 16, 2, 128, 64, 0, 0, "bf16"),
        # a chunk added to a long conversation: few rows, the work is split along the keys
        _chunk("chunk long", 1, 256, 256, 16, 2, 128, 64, 60001, 60001, "bf16"),
        # full precision at the small head size, odd lengths, small pages
        _chunk("chunk fp32", 3, 150, 67, 12, 3, 64, 16, 5, 700, "fp32"),
        # one user, a short chain of drafted tokens: the call's latency
        _sample("sample one chain", 1, 8, 8, 32768, "chain", "dist"),
        # the decode sweep's block over a large vocabulary
        _sample("sample chains", 32, 16, 16, 131072, "chain", "dist"),
        # wide trees of several candidates per step, odd vocabulary
        _sample("sample trees", 12, 48, 31, 65537, "tree", "dist"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["advance", "advance", "conv", "chunk", "chunk", "sample", "sample"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        T = spread(1, 8192)
        fresh = rng.choice(["none", "some", "all"])
        if op == "advance":
            Hk = rng.choice([1, 2, 4, 5, 8, 16])
            c = _advance("", spread(1, 32), T, rng.randint(max(1, T // 3), T), Hk * rng.choice([1, 1, 2, 3]), Hk,
                         rng.choice([64, 128, 128]), rng.choice([64, 128, 128]), fresh, dtype)
            n = sum(_lens(c)) * c["H"]
            if n > 8 * 2048 * 16 or c["H"] > 32 or (dtype == "fp32" and n * T > 4e7):
                continue
        elif op == "conv":
            c = _conv("", spread(1, 32), T, rng.randint(max(1, T // 3), T), 8 * rng.randint(1, 1024), rng.randint(1, 4),
                      rng.random() < 0.7, fresh, dtype)
            if sum(_lens(c)) * c["D"] > 8 * 2048 * 6144:
                continue
        elif op == "chunk":
            Hkv, G = rng.choice([1, 2, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
            lo = rng.choice([0, spread(1, 20000)])
            c = _chunk("", spread(1, 16), T, rng.randint(max(1, T // 2), T), Hkv * G, Hkv,
                       rng.choice([64, 128, 128, 256]), rng.choice([16, 16, 32, 64, 128]), lo,
                       lo + rng.choice([0, spread(1, 8000)]), dtype)
            if T < 2 or work(c)["flops"] > (2e11 if dtype == "bf16" else 1e10) or _cache_bytes(c) > 1.6e9:
                continue
            if c["B"] * T * c["Hq"] * c["d"] > 1.5e8:
                continue
        else:
            V = spread(2, 200000)
            T = rng.randint(2, 64)
            c = _sample("", spread(1, 64), T, rng.randint((T + 1) // 2, T), V, rng.choice(["chain", "chain", "tree"]),
                        rng.choice(["dist", "dist", "point"]))
            if c["B"] * T * V > 32 * 16 * 131072:
                continue
        del c["name"]
        return c


def _fill(n, lo, hi, k):
    """n whole numbers spread over [lo, hi], the same for every seed."""
    return [lo + int((hi - lo + 0.999) * ((i * 0.6180339887 + 0.37 * k) % 1.0)) if hi > lo else lo for i in range(n)]


def _lens(c):
    n = _fill(c["B"], c["len_lo"], c["T"], 2)
    n[0] = c["T"]
    return n


def _past(c):
    return _fill(c["B"], c["past_lo"], c["past_hi"], 1)


def _fresh(c):
    return [int(c["fresh"] == "all" or (c["fresh"] == "some" and i % 3 != 1)) for i in range(c["B"])]


def _size(c):
    return 2 if c["dtype"] == "bf16" else 4


def _max_pages(c):
    return -(-(c["past_hi"] + c["T"]) // c["page"])


def _n_page(c):
    return sum(-(-(x + y) // c["page"]) for x, y in zip(_past(c), _lens(c))) + 3


def _cache_bytes(c):
    return 2 * _n_page(c) * c["Hkv"] * c["page"] * c["d"] * _size(c)


def work(c):
    op, lens = c["op"], _lens(c)
    n = sum(lens)
    if op == "advance":
        state = 4 * c["H"] * c["dk"] * c["dv"]
        token = 2 * c["Hk"] * c["dk"] * _size(c) + c["H"] * (c["dv"] * (_size(c) + 4) + 8)
        # S k, S q, the rank-one update and the decay
        return {"bytes": n * token + state * (2 * c["B"] - sum(_fresh(c))), "flops": 7 * n * c["H"] * c["dk"] * c["dv"]}
    if op == "conv":
        ring = 2 * (c["W"] - 1) * c["B"] * c["D"] * _size(c)
        return {"bytes": 2 * n * c["D"] * _size(c) + ring + 4 * c["D"] * (c["W"] + 1), "flops": 2 * n * c["D"] * (c["W"] + 2)}
    if op == "chunk":
        e, d = _size(c), c["d"]
        seen = sum(y * x + y * (y + 1) // 2 for x, y in zip(_past(c), lens))
        keys = n + sum(_past(c))
        return {"bytes": 2 * keys * c["Hkv"] * d * e + n * c["Hq"] * (2 * d * e + 4), "flops": 4 * seen * c["Hq"] * d}
    # one row of the target's and the drafter's probabilities per sequence, a few numbers per token
    rows = 2 if c["drafter"] == "dist" else 1
    return {"bytes": 4 * (rows * c["B"] * c["V"] + n * (rows + 3)), "flops": 3 * c["B"] * c["V"]}


# ------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _slots(c, g):
    """One slot more than there are sequences, in a random order."""
    return torch.randperm(c["B"] + 1, generator=g, device="cuda")[:c["B"]].to(torch.int32)


def _prepare_advance(c, g, s):
    B, T, H, Hk, dk, dv = (c[n] for n in ("B", "T", "H", "Hk", "dk", "dv"))
    dt = TORCH[c["dtype"]]
    unit = torch.nn.functional.normalize
    s["q"] = unit(_randn(g, B, T, Hk, dk), dim=-1).to(dt)
    s["k"] = unit(_randn(g, B, T, Hk, dk), dim=-1).to(dt)
    s["v"] = _randn(g, B, T, H, dv, dtype=dt)
    s["g"] = -torch.nn.functional.softplus(_randn(g, B, T, H))
    s["beta"] = torch.sigmoid(_randn(g, B, T, H))
    s["slots"] = _slots(c, g)
    s["state"] = _randn(g, B + 1, H, dv, dk, scale=0.1)
    s["len"], s["fresh"] = _i32(_lens(c)), _i32(_fresh(c))
    s["out"] = torch.zeros(B, T, H, dv, device="cuda")
    if own:
        import speculative_decode_recurrent_gb300 as lib
        cap = 31 + 16
        dims = lib.Dims(B=B, H=H, dk=dk, dv=dv, T=16, cap=cap, threshold=32, n_slot=B + 1,
                        in_dtype=lib.DTYPE_BF16 if c["dtype"] == "bf16" else lib.DTYPE_F32, scale=dk ** -0.5)
        init = dict(state=s["state"], state_idx=s["slots"], buf_len=_i32([0] * (B + 1)))
        for n, d in (("buf_k", dk), ("buf_v", dv)):
            init[n] = torch.zeros(B + 1, H, cap, d, dtype=dt, device="cuda")
        for n in ("buf_g", "buf_beta"):
            init[n] = torch.zeros(B + 1, H, cap, device="cuda")
        s["layer"] = lib.ReplayLayer(dims, init)
        s["workspace"] = s["layer"].advance_workspace(T, Hk)


def _prepare_conv(c, g, s):
    B, T, D, W = c["B"], c["T"], c["D"], c["W"]
    dt, cap = TORCH[c["dtype"]], c["W"] - 1 + 16
    s["x"] = _randn(g, B, T, D, dtype=dt)
    s["weight"], s["bias"] = _randn(g, D, W, scale=W ** -0.5), _randn(g, D, scale=0.1)
    s["slots"] = _slots(c, g)
    s["ring"] = _randn(g, B + 1, cap, D, dtype=dt)
    s["pos"] = torch.randint(0, cap, (B + 1,), generator=g, device="cuda", dtype=torch.int32)
    s["len"], s["fresh"] = _i32(_lens(c)), _i32(_fresh(c))
    s["y"] = torch.zeros(B, T, D, dtype=dt, device="cuda")
    if own:
        import speculative_decode_recurrent_gb300 as lib
        code = lib.DTYPE_BF16 if c["dtype"] == "bf16" else lib.DTYPE_F32
        dims = lib.ConvDims(B=B, D=D, W=W, T=16, cap=cap, n_slot=B + 1, in_dtype=code, out_dtype=code,
                            act=lib.CONV_ACT_SILU if c["silu"] else lib.CONV_ACT_NONE)
        s["layer"] = lib.ConvLayer(dims, {n: s[m] for n, m in (("ring", "ring"), ("pos", "pos"), ("state_idx", "slots"),
                                                               ("weight", "weight"), ("bias", "bias"))})


def _prepare_chunk(c, g, s):
    B, T, Hq, Hkv, d, page = (c[n] for n in ("B", "T", "Hq", "Hkv", "d", "page"))
    dt, past, lens, n_page, mp = TORCH[c["dtype"]], _past(c), _lens(c), _n_page(c), _max_pages(c)
    owned = [-(-(x + y) // page) for x, y in zip(past, lens)]
    order = torch.randperm(n_page, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(owned):
        table[b, :n] = order[at:at + n]
        at += n
    ref = torch.zeros(n_page, dtype=torch.int32, device="cuda")
    ref[order[:at].long()] = 1
    free = torch.zeros(n_page, dtype=torch.int32, device="cuda")
    free[:n_page - at] = order[at:]
    shape = (1, n_page, Hkv, page, d)
    s["t"] = dict(k=_randn(g, *shape, scale=1.4, dtype=dt), v=_randn(g, *shape, dtype=dt), block_table=table,
                  seq_len=_i32(past), n_owned=_i32(owned), ref=ref, free_list=free, free_count=_i32([n_page - at]))
    s["q"] = _randn(g, B, T, Hq, d, scale=1.4, dtype=dt)
    s["len"] = _i32(lens)
    s["out"] = torch.zeros(B, T, Hq, d, dtype=dt, device="cuda")
    s["lse"] = torch.zeros(B, T, Hq, device="cuda")
    if own:
        import speculative_decode_recurrent_gb300 as lib
        cache = lib.PagedCache(lib.PageDims(n_slot=B, max_pages=mp, n_page=n_page, page=page, n_layer=1, Hkv=Hkv, d=d,
                                            dtype=lib.DTYPE_BF16 if c["dtype"] == "bf16" else lib.DTYPE_F32), s["t"])
        s["layer"] = lib.AttnLayer(lib.AttnDims(B=B, T=T, Hq=Hq, scale=d ** -0.5), cache, 0)


def _prepare_sample(c, g, s):
    B, T, V = c["B"], c["T"], c["V"]
    t = torch.arange(T, device="cuda")
    if c["shape"] == "tree":
        back = 1 + (torch.rand(B, T, generator=g, device="cuda") * 4).long()
        parent = torch.where(t == 0, -1, (t - back).clamp(min=0)).to(torch.int32)
        s["parent"] = parent
    else:
        parent = (t - 1).to(torch.int32).expand(B, T)
        s["parent"] = None
    # the drafter's logits are the target's with some noise
    z = _randn(g, B, T, V, scale=2.5)
    s["probs"] = torch.softmax(z, -1)
    zq = z.add_(_randn(g, B, T, V, scale=0.5))
    draft = torch.softmax(zq, -1)
    # token t is drawn from the drafter's probabilities after its parent
    tokens = torch.zeros(B, T, dtype=torch.int64, device="cuda")
    rows = torch.arange(B, device="cuda")
    for i in range(T):
        p = draft[rows, parent[:, i].long().clamp(min=0)].cumsum(-1)
        r = torch.rand(B, 1, generator=g, device="cuda") * p[:, -1:]
        tokens[:, i] = (p <= r).sum(-1).clamp(max=V - 1)
    s["tokens"] = tokens.to(torch.int32)
    s["draft"] = draft if c["drafter"] == "dist" else None
    s["u"] = torch.rand(B, T, generator=g, device="cuda")
    s["len"] = _i32(_lens(c))
    s["accepted"], s["next"] = _i32([0] * B), _i32([0] * B)
    s["path"] = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    if own:
        import speculative_decode_recurrent_gb300 as lib
        s["sampler"] = lib.DraftSampler(lib.DraftDims(B=B, T=T, V=V))


def prepare(case, seed):
    s = dict(case=dict(case))
    {"advance": _prepare_advance, "conv": _prepare_conv, "chunk": _prepare_chunk, "sample": _prepare_sample}[case["op"]](
        case, _gen(seed), s)
    return s


# ------------------------------------------------------------------- plain forms
def _plain_advance(s):
    c = s["case"]
    rep, slots = c["H"] // c["Hk"], s["slots"].long()
    q = s["q"].float().repeat_interleave(rep, 2) * c["dk"] ** -0.5
    k = s["k"].float().repeat_interleave(rep, 2)
    v = s["v"].float()
    live = torch.arange(c["T"], device="cuda") < s["len"][:, None]
    alpha = torch.where(live[..., None], s["g"].exp(), torch.ones_like(s["g"]))
    beta = torch.where(live[..., None], s["beta"], torch.zeros_like(s["beta"]))
    S = torch.where(s["fresh"][:, None, None, None] != 0, torch.zeros_like(s["state"][slots]), s["state"][slots])
    for t in range(c["T"]):
        S = S * alpha[:, t, :, None, None]
        kt = k[:, t, :, None]
        u = (v[:, t] - (S * kt).sum(-1)) * beta[:, t, :, None]
        S = S + u[..., None] * kt
        s["out"][:, t] = (S * q[:, t, :, None]).sum(-1)
    s["out"].masked_fill_(~live[..., None, None], 0.0)
    s["state"][slots] = S
    return {"out": s["out"], "state": s["state"]}


def _plain_conv(s):
    c = s["case"]
    T, W, cap, slots, n = c["T"], c["W"], s["ring"].shape[1], s["slots"].long(), s["len"].long()
    pos, back = s["pos"][slots].long(), torch.arange(W - 1, 0, -1, device="cuda")
    window = s["ring"][slots[:, None], (pos[:, None] - back) % cap].float()              # oldest first
    window = torch.where(s["fresh"][:, None, None] != 0, torch.zeros_like(window), window)
    x = torch.cat([window, s["x"].float()], 1)                                            # [B, W - 1 + T, D]
    y = s["bias"].expand(c["B"], T, -1).clone()
    for j in range(W):
        y += x[:, j:j + T] * s["weight"][:, j]
    if c["silu"]:
        y = y / (1 + torch.exp(-y))
    live = torch.arange(T, device="cuda") < n[:, None]
    s["y"].copy_(torch.where(live[..., None], y, torch.zeros_like(y)))
    end = (pos + n) % cap
    if W > 1:
        last = x.gather(1, (n[:, None] + torch.arange(W - 1, device="cuda"))[..., None].expand(-1, -1, c["D"]))
        s["ring"][slots[:, None], (end[:, None] - back) % cap] = last.to(s["ring"].dtype)
    s["pos"][slots] = end.to(torch.int32)
    return {"y": s["y"], "ring": s["ring"], "pos": s["pos"]}


def _plain_chunk(s):
    c, t = s["case"], s["t"]
    Hkv, d, G, page = c["Hkv"], c["d"], c["Hq"] // c["Hkv"], c["page"]
    for b, (past, n) in enumerate(zip(_past(c), _lens(c))):
        m = past + n
        ids = t["block_table"][b, :-(-m // page)].long()
        k, v = (t[x][0][ids].transpose(0, 1).reshape(Hkv, -1, d)[:, :m].float() for x in ("k", "v"))
        step = max(1, 4_000_000 // m)                        # rows of tokens at a time: the scores stay small
        for i in range(0, n, step):
            w = min(step, n - i)
            q = s["q"][b, i:i + w].float().reshape(w, Hkv, G, d).permute(1, 2, 0, 3)          # [Hkv, G, w, d]
            x = torch.matmul(q, k[:, None].transpose(2, 3)) * d ** -0.5
            x.masked_fill_(torch.arange(m, device="cuda") > past + i + torch.arange(w, device="cuda")[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            den = p.sum(-1, keepdim=True)
            s["out"][b, i:i + w] = (torch.matmul(p, v[:, None]) / den).permute(2, 0, 1, 3).reshape(w, -1, d).to(s["out"].dtype)
            s["lse"][b, i:i + w] = (top + torch.log(den))[..., 0].permute(2, 0, 1).reshape(w, -1)
        s["out"][b, n:] = 0
        s["lse"][b, n:] = -math.inf
    return {"out": s["out"], "lse": s["lse"]}


def _plain_sample(s):
    """Node by node in the order of the tokens, for all sequences at once.  At a node with the
    target's probabilities p and the drafter's q, after k rejected children the rest is
    r = max(p - c q, 0) with c the sum of the rests' masses so far (1 for r = p); a child x is
    accepted where u q(x) mass(r) < r(x)."""
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    rows, dev = torch.arange(B, device="cuda"), dict(device="cuda")
    p, u = s["probs"], s["u"].double()
    parent = s["parent"].long() if s["parent"] is not None else (torch.arange(T, **dev) - 1).expand(B, T)
    cur = torch.zeros(B, dtype=torch.int64, **dev)
    cnt = torch.where(s["len"] > 0, 1, 0).long()
    path = torch.where(torch.arange(T, **dev)[None] == 0, 0, -1).expand(B, T).contiguous()
    mass = torch.ones(B, dtype=torch.float64, **dev)
    r = p[:, 0].double().clamp(min=0)
    taken = torch.zeros(B, dtype=torch.float64, **dev)                   # c
    for t in range(1, T):
        x = s["tokens"][:, t].long()
        child = (parent[:, t] == cur) & (t < s["len"]) & (mass > 0)
        q = s["draft"][rows, cur].double() if s["draft"] is not None else None
        qx = q[rows, x] if q is not None else 1.0
        ok = child & (u[:, t] * qx * mass < r[rows, x])
        no = child & ~ok
        if q is not None:
            taken_no = taken + mass
            r_no = (p[rows, cur].double().clamp(min=0) - taken_no[:, None] * q).clamp(min=0)
            mass_no = r_no.sum(-1)
        else:
            taken_no = taken
            mass_no = mass - r[rows, x]
            r_no = r.scatter(1, x[:, None], 0.0)
        cur = torch.where(ok, t, cur)
        path[rows, cnt.clamp(max=T - 1)] = torch.where(ok, t, path[rows, cnt.clamp(max=T - 1)])
        cnt = cnt + ok
        r = torch.where(ok[:, None], p[:, t].double().clamp(min=0), torch.where(no[:, None], r_no, r))
        mass = torch.where(ok, 1.0, torch.where(no, mass_no, mass))
        taken = torch.where(ok, 0.0, torch.where(no, taken_no, taken))
    # a rest without mass: the target's own probabilities
    r = torch.where((r.sum(-1) > 0)[:, None], r, p[rows, cur].double().clamp(min=0))
    acc = r.cumsum(-1)
    over = acc > u[:, :1] * acc[:, -1:]
    last = V - 1 - (r.flip(-1) > 0).to(torch.uint8).argmax(-1)
    nxt = torch.where(over.any(-1), over.to(torch.uint8).argmax(-1), last)
    s["accepted"].copy_(cnt)
    s["next"].copy_(nxt)
    s["path"].copy_(path)
    return {"accepted": s["accepted"], "next": s["next"], "path": s["path"]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"advance": _plain_advance, "conv": _plain_conv, "chunk": _plain_chunk, "sample": _plain_sample}[op](s)
    if op == "advance":
        s["layer"].advance(s["q"], s["k"], s["v"], s["g"], s["beta"], s["out"], chunk_len=s["len"], fresh=s["fresh"],
                           workspace=s["workspace"])
        return {"out": s["out"], "state": s["state"]}
    if op == "conv":
        s["layer"].advance(s["x"], s["y"], chunk_len=s["len"], fresh=s["fresh"])
        return {"y": s["y"], "ring": s["ring"], "pos": s["pos"]}
    if op == "chunk":
        s["layer"].chunk(s["q"], s["out"], lse=s["lse"], chunk_len=s["len"])
        return {"out": s["out"], "lse": s["lse"]}
    s["sampler"].accept(s["tokens"], s["probs"], s["u"], s["accepted"], s["next"], draft=s["draft"], parent=s["parent"],
                        path=s["path"], draft_len=s["len"])
    return {"accepted": s["accepted"], "next": s["next"], "path": s["path"]}


# ------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    c = case
    if c["op"] == "sample":                                  # whole numbers only
        return None
    s = prepare(case, seed)
    lens = _lens(c)
    if c["op"] == "advance":
        # S_t = a_t S_{t-1} (I - b_t k k^T) + b_t v k^T,  o_t = S_t q_t / sqrt(d), sequence by sequence
        out, state = torch.zeros_like(s["out"], dtype=torch.float64), s["state"].double()
        rep = c["H"] // c["Hk"]
        eye = torch.eye(c["dk"], dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            slot = int(s["slots"][b])
            S = state[slot] * (0.0 if _fresh(c)[b] else 1.0)
            q, k = (s[x][b, :n].double().repeat_interleave(rep, 1) for x in ("q", "k"))
            v, a, be = s["v"][b, :n].double(), s["g"][b, :n].double().exp(), s["beta"][b, :n].double()
            if n * c["H"] <= 1 << 14:
                for t in range(n):
                    kk = torch.einsum("hi,hj->hij", k[t], k[t])
                    S = a[t, :, None, None] * torch.einsum("hvi,hij->hvj", S, eye - be[t, :, None, None] * kk)
                    S = S + be[t, :, None, None] * torch.einsum("hv,hi->hvi", v[t], k[t])
                    out[b, t] = torch.einsum("hvi,hi->hv", S, q[t])
            else:
                # the same, 32 tokens at a time: with G the sums of g, u_t = b_t (v_t - e^{G_t} S k_t
                # - sum_{s<t} e^{G_t - G_s} (k_t.k_s) u_s), by elimination
                lg = s["g"][b, :n].double()
                for i in range(0, n, 32):
                    w = min(32, n - i)
                    G = lg[i:i + w].cumsum(0).t()                                             # [H, w]
                    K, Q, V = (x[i:i + w].transpose(0, 1) for x in (k, q, v))                 # [H, w, d]
                    D = torch.exp((G[:, :, None] - G[:, None]).tril()).tril()
                    B_ = be[i:i + w].t()[..., None]
                    A = (K @ K.transpose(1, 2) * D).tril(-1) * B_
                    rhs = B_ * (V - G.exp()[..., None] * (K @ S.transpose(1, 2)))
                    u = torch.zeros_like(rhs)
                    for t in range(w):
                        u[:, t] = rhs[:, t] - (A[:, t:t + 1, :t] @ u[:, :t])[:, 0] if t else rhs[:, 0]
                    o = G.exp()[..., None] * (Q @ S.transpose(1, 2)) + (Q @ K.transpose(1, 2) * D) @ u
                    out[b, i:i + w] = o.transpose(0, 1)
                    S = G[:, -1].exp()[:, None, None] * S + (u * D[:, -1, :, None]).transpose(1, 2) @ K
            out[b, :n] *= c["dk"] ** -0.5
            state[slot] = S
        return {"out": out, "state": state}
    if c["op"] == "conv":
        ring, y = s["ring"].double(), torch.zeros_like(s["y"], dtype=torch.float64)
        cap, W = ring.shape[1], c["W"]
        for b, n in enumerate(lens):
            slot, pos = int(s["slots"][b]), int(s["pos"][int(s["slots"][b])])
            old = [torch.zeros(c["D"], dtype=torch.float64, device="cuda") if _fresh(c)[b] else ring[slot, (pos - j) % cap].clone()
                   for j in range(W - 1, 0, -1)]
            x = torch.stack(old + list(s["x"][b, :n].double())) if n + W > 1 else None
            z = (x.unfold(0, W, 1) * s["weight"].double()).sum(-1) + s["bias"].double()
            y[b, :n] = z * torch.sigmoid(z) if c["silu"] else z
            for j in range(1, W):
                ring[slot, (pos + n - j) % cap] = x[W - 1 + n - j]
        return {"y": y, "ring": ring, "pos": None}
    t, d, G = s["t"], c["d"], c["Hq"] // c["Hkv"]
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    lse = torch.full_like(s["lse"], -math.inf, dtype=torch.float64)
    for b, (past, n) in enumerate(zip(_past(c), lens)):
        m = past + n
        row = torch.arange(m, device="cuda")
        ids = t["block_table"][b].long()[row // c["page"]]
        for h in range(c["Hq"]):
            k, v = (t[x][0][ids, h // G, row % c["page"]].double() for x in ("k", "v"))
            for i in range(0, n, 1024):
                w = min(1024, n - i)
                x = s["q"][b, i:i + w, h].double() @ k.t() / math.sqrt(d)
                x = torch.where(row[None] <= past + i + torch.arange(w, device="cuda")[:, None], x, -math.inf)
                lse[b, i:i + w, h] = torch.logsumexp(x, -1)
                out[b, i:i + w, h] = torch.exp(x - lse[b, i:i + w, h, None]) @ v
    return {"out": out, "lse": lse}
