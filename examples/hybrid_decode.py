"""Decode steps of a small hybrid stack under speculation: recurrent (GDN) layers and an
attention layer, with synthetic projections and drafts.

Each step drafts a chain of T tokens per sequence.  A recurrent layer verifies it over its
checkpoint and buffer; the attention layer stages the chain's keys and values in its pages and
attends over them and the context.  Accepting p tokens moves two lengths.  Between the steps a
sequence is forked and one is released.  A second attention cache then verifies a token tree and
commits one of its paths.  At last a stack of a convolution, a recurrent and an attention layer takes
prompts in chunks, then decodes: drafts of a bigram table, verified, accepted by speculative sampling.

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


def norm_weights(g):
    return (1 + 0.1 * torch.randn(2, D, generator=g)).cuda()


def attention(cache, g, tokens, w=None):
    rope = lib.RopeDims(rot=64, style=lib.ROPE_HALF, max_pos=512, eps=1e-6)
    w = norm_weights(g) if w is None else w
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


V, W, PART, C = 97, 4, 100, 3 * H * D                       # vocabulary, convolution width, tokens of a prompt's chunk, channels


class Stack:
    """A convolution over the channels of q, k and v, a recurrent layer, an attention layer and a head, with random weights."""

    def __init__(self, g):
        def weight(n, m):
            return (torch.randn(n, m, generator=g) * n ** -0.5).bfloat16().cuda()

        self.embed = torch.randn(V, C, generator=g).bfloat16().cuda()
        self.gate = (-torch.rand(V, H, generator=g)).cuda()
        self.beta = torch.rand(V, H, generator=g).cuda()
        self.w_qkv, self.w_out = weight(H * D, (H + 2 * HKV) * D), weight(H * D, V)
        self.drafter = torch.randn(V, V, generator=g).softmax(-1).cuda()
        dims = lib.ConvDims(B=B, D=C, W=W, T=T, cap=W - 1 + T, n_slot=SLOTS, act=lib.CONV_ACT_SILU, in_dtype=lib.DTYPE_BF16,
                            out_dtype=lib.DTYPE_BF16)
        self.conv = lib.ConvLayer(dims, dict(ring=torch.zeros(SLOTS, dims.cap, C, dtype=torch.bfloat16),
                                             pos=torch.zeros(SLOTS, dtype=torch.int32),
                                             state_idx=torch.arange(B, dtype=torch.int32),
                                             weight=0.5 * torch.randn(C, W, generator=g)))
        self.gdn, self.cache = recurrent_layer(g), page_cache()
        w = norm_weights(g)                                 # one layer, for chunks of a prompt and for drafts
        self.part, self.block = (attention(self.cache, g, n, w) for n in (PART, T))

    def mixed(self, tokens, y):
        """q, k, v, log-decays and update rates from the convolution's outputs."""
        q, k, v = (x.unflatten(-1, (H, D)) for x in y.split(H * D, -1))
        return unit(q.float()).bfloat16(), unit(k.float()).bfloat16(), v, self.gate[tokens], self.beta[tokens]

    def projected(self, out):
        qkv = (out.bfloat16().flatten(2) @ self.w_qkv).split([H * D, HKV * D, HKV * D], -1)
        return [p.unflatten(-1, (-1, D)) for p in qkv]

    def probs(self, att):
        return (att.flatten(2) @ self.w_out).float().softmax(-1)

    def prompt(self, tokens, n, fresh):
        """A chunk of n[b] committed tokens; the target's distribution after the last of them."""
        y = torch.empty(B, PART, C, dtype=torch.bfloat16, device="cuda")
        self.conv.advance(self.embed[tokens], y, chunk_len=n, fresh=fresh)
        out = torch.empty(B, PART, H, D, device="cuda")
        self.gdn.advance(*self.mixed(tokens, y), out, chunk_len=n, fresh=fresh)
        q, att = (torch.empty(B, PART, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.cache.reserve(i32(range(B)), PART)
        self.part.stage(*self.projected(out), q, draft_len=n)
        self.part.chunk(q, att, chunk_len=n)
        self.cache.seq_len[:B] += n
        return self.probs(att)[torch.arange(B, device="cuda"), (n - 1).clamp(min=0).long()]

    def verify(self, tokens):
        """The target's distributions after each token of a block."""
        y = torch.empty(B, T, C, dtype=torch.bfloat16, device="cuda")
        self.conv.verify(self.embed[tokens], y)
        out = torch.empty(B, T, H, D, device="cuda")
        self.gdn.verify(*(x.contiguous() for x in self.mixed(tokens, y)), out)
        q, att = (torch.empty(B, T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.cache.reserve(i32(range(B)), T)
        self.block.stage(*self.projected(out), q)
        self.block.verify(q, att)
        return self.probs(att), q, att

    def accept(self, p):
        self.conv.accept(p)
        self.gdn.accept(p)
        self.gdn.flush()
        self.cache.accept(p, state_idx=i32(range(B)), T=T)


def run_prompt(lens=(150, 70, 1), rounds=5, seed=3):
    """Prompts of the given lengths in chunks, then rounds of speculative decoding.  Returns the stack, each sequence's
    committed tokens and what each round's sampling took and gave (for the tests)."""
    g = torch.Generator().manual_seed(seed)
    s = Stack(g)
    prompts = torch.randint(0, V, (B, -(-max(lens) // PART) * PART), generator=g)
    first = torch.empty(B, V, device="cuda")
    for at in range(0, max(lens), PART):
        n = i32([min(max(x - at, 0), PART) for x in lens])
        p = s.prompt(prompts[:, at:at + PART].cuda(), n, fresh=i32([at == 0] * B))
        first = torch.where((n > 0)[:, None], p, first)
    # the first token after the prompt: a block of one, nothing to accept
    one = lib.DraftSampler(lib.DraftDims(B=B, T=1, V=V))
    sampler = lib.DraftSampler(lib.DraftDims(B=B, T=T, V=V))
    taken, cur = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    one.accept(torch.zeros(B, 1, dtype=torch.int32, device="cuda"), first[:, None].contiguous(), torch.rand(B, 1, generator=g).cuda(),
               taken, cur)
    committed = [prompts[b, :n].tolist() for b, n in enumerate(lens)]
    log = []
    for _ in range(rounds):
        tokens = cur[:, None]
        for _ in range(T - 1):                              # the drafter's chain
            q = s.drafter[tokens[:, -1].long()].cpu()
            tokens = torch.cat([tokens, torch.multinomial(q, 1, generator=g).int().cuda()], 1)
        draft = s.drafter[tokens.long()]                    # row t: what token t + 1 was drawn from
        probs, q_rot, att = s.verify(tokens)
        u = torch.rand(B, T, generator=g).cuda()
        cur = torch.empty_like(cur)
        before = s.cache.seq_len.tolist()
        sampler.accept(tokens, probs, u, taken, cur, draft=draft)
        s.accept(taken)
        log.append(dict(tokens=tokens, probs=probs, draft=draft, u=u, taken=taken.tolist(), next=cur.tolist(), q=q_rot, att=att,
                        lengths=before))
        for b, n in enumerate(log[-1]["taken"]):
            committed[b] += tokens[b, :n].tolist()
    s.gdn.flush(force=True)
    torch.cuda.synchronize()
    status = [x.status.item() for x in (s.conv, s.gdn, s.cache, one, sampler)]
    return dict(stack=s, committed=committed, log=log, status=max(status))


if __name__ == "__main__":
    r = run()
    print("lengths", r["lengths"], "committed", r["committed"], "status", r["status"])
    t = run_tree()
    print("tree: lengths", t["cache"].seq_len[:B].tolist(), "status", t["status"])
    p = run_prompt()
    print("prompts: lengths", [len(x) for x in p["committed"]], "accepted", [x["taken"] for x in p["log"]], "status", p["status"])
