"""Decode steps of a small hybrid stack under speculation: recurrent (GDN) layers and an
attention layer, with synthetic projections and drafts.

Each step drafts a chain of T tokens per sequence.  A recurrent layer verifies it over its
checkpoint and buffer; the attention layer stages the chain's keys and values in its pages and
attends over them and the context.  Accepting p tokens moves two lengths.  Between the steps a
sequence is forked and one is released.  A second attention cache then verifies a token tree and
commits one of its paths.

    python examples/hybrid_decode.py            # needs a GB300
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decode_recurrent_gb300 as lib  # noqa: E402

B, T, H, D, HKV, PAGE, SLOTS = 3, 8, 4, 128, 2, 16, 6


def angles(max_pos, rot):
    """cos | sin of each position: fp32 [max_pos, rot], from 64-bit angles."""
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def unit(x):
    return torch.nn.functional.normalize(x, dim=-1)


def recurrent_layer(g):
    n = SLOTS
    dims = lib.Dims(B=B, H=H, dk=D, dv=D, T=T, cap=32 - 1 + T, threshold=32, n_slot=n, in_dtype=lib.DTYPE_BF16,
                    scale=D ** -0.5)
    cap = dims.cap
    init = dict(state=torch.zeros(n, H, D, D), state_idx=torch.arange(B, dtype=torch.int32),
                buf_k=torch.zeros(n, H, cap, D, dtype=torch.bfloat16), buf_v=torch.zeros(n, H, cap, D, dtype=torch.bfloat16),
                buf_g=torch.zeros(n, H, cap), buf_beta=torch.zeros(n, H, cap), buf_len=torch.zeros(n, dtype=torch.int32))
    return lib.ReplayLayer(dims, init)


def attention(cache, g, tokens):
    rope = lib.RopeDims(rot=64, style=lib.ROPE_HALF, max_pos=512, eps=1e-6)
    w = (1 + 0.1 * torch.randn(2, D, generator=g)).cuda()
    return lib.AttnLayer(lib.AttnDims(B=B, T=tokens, Hq=H, scale=D ** -0.5), cache, 0, rope, w[0], w[1],
                         angles(512, 64), state_idx=torch.arange(B, dtype=torch.int32, device="cuda"))


def page_cache():
    return lib.PagedCache(lib.PageDims(n_slot=SLOTS, max_pages=32, n_page=96, page=PAGE, n_layer=1, Hkv=HKV, d=D,
                                       dtype=lib.DTYPE_BF16))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(steps=6, seed=1):
    """The hybrid loop.  Returns the lengths of the attention cache, the committed tokens per
    sequence, and the caches and last outputs (for the tests)."""
    g = torch.Generator().manual_seed(seed)
    cache = page_cache()
    gdn, attn = recurrent_layer(g), attention(cache, g, T)
    rows = i32(range(B))
    w_qkv = (torch.randn(H * D, (H + 2 * HKV) * D, generator=g) * (H * D) ** -0.5).bfloat16().cuda()
    out = torch.empty(B, T, H, D, device="cuda")
    q_rot, att = (torch.empty(B, T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    committed = [0] * B
    for step in range(steps):
        # the recurrent layer verifies the draft
        x = {n: torch.randn(B, T, H, D, generator=g) for n in ("q", "k", "v")}
        q, k, v = unit(x["q"]).bfloat16().cuda(), unit(x["k"]).bfloat16().cuda(), x["v"].bfloat16().cuda()
        gate = (-torch.rand(B, T, H, generator=g)).cuda()
        beta = torch.rand(B, T, H, generator=g).cuda()
        gdn.verify(q, k, v, gate, beta, out)
        # the attention layer on its outputs: one projection, its three parts used in place
        qkv = (out.bfloat16().flatten(2) @ w_qkv).split([H * D, HKV * D, HKV * D], -1)
        qa, ka, va = (p.unflatten(-1, (-1, D)) for p in qkv)
        cache.reserve(rows, T)
        attn.stage(qa, ka, va, q_rot)
        attn.verify(q_rot, att)
        # the first p tokens of each draft are accepted: two lengths move
        p = torch.randint(0, T + 1, (B,), generator=g).tolist()
        gdn.accept(i32(p))
        gdn.flush()
        cache.accept(i32(p), state_idx=rows, T=T)
        committed = [a + b for a, b in zip(committed, p)]
        if step == 2:                                       # a continuation of sequence 0, given up again later
            cache.fork(i32([0]), i32([B]), torch.empty(1, 2, dtype=torch.int32, device="cuda"))
        if step == 4:
            cache.release(i32([B]))
    torch.cuda.synchronize()
    return dict(cache=cache, gdn=gdn, committed=committed, lengths=cache.seq_len.tolist(), att=att, q=q_rot,
                status=int(cache.status.item()) | int(gdn.status.item()))


def run_tree(seed=2):
    """One step with a token tree: context staged as a first block, then a tree of T tokens, of
    which the path to its deepest token is committed."""
    g = torch.Generator().manual_seed(seed)
    cache = page_cache()
    context = 40
    first, layer = attention(cache, g, context), attention(cache, g, T)
    rows = i32(range(B))

    def block(n):
        return [torch.randn(B, n, h, D, generator=g).bfloat16().cuda() for h in (H, HKV, HKV)]

    cache.reserve(rows, context + T)
    first.stage(*block(context), torch.empty(B, context, H, D, dtype=torch.bfloat16, device="cuda"))
    cache.seq_len[:B] = context
    parent = torch.tensor([[-1, 0, 0, 1, 1, 3, 2, 5]] * B, dtype=torch.int32)
    tree = torch.empty(B, T, dtype=torch.int64, device="cuda")
    pos = torch.empty(B, T, dtype=torch.int32, device="cuda")
    layer.build_tree(parent.cuda(), tree, pos)
    q, out = (torch.empty(B, T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    layer.stage(*block(T), q, pos=pos)
    layer.verify(q, out, tree=tree)
    path = i32([[0, 1, 3, 5, 7, 0, 0, 0]] * B)              # tokens 0 -> 1 -> 3 -> 5 -> 7
    staged = cache.k.clone()
    cache.accept(i32([5] * B), path=path, state_idx=rows)
    torch.cuda.synchronize()
    return dict(cache=cache, staged=staged, out=out, q=q, tree=tree, pos=pos, context=context, path=path,
                status=int(cache.status.item()))


if __name__ == "__main__":
    r = run()
    print("lengths", r["lengths"], "committed", r["committed"], "status", r["status"])
    t = run_tree()
    print("tree: lengths", t["cache"].seq_len[:B].tolist(), "status", t["status"])
