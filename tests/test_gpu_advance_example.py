"""The example's prompts and decode rounds: convolution, recurrence, attention and sampling as they are used together."""
import os
import sys

import numpy as np
import pytest
import torch

import advance_ref as A
import attn_ref as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def rows(cache, x, slot, n):
    pos = torch.arange(n)
    ids = cache.block_table[slot].cpu()[pos // cache.d.page].long()
    return R.f64(x[0].cpu()[ids, :, pos % cache.d.page])


@pytest.mark.parametrize("lens", [(150, 70, 1), (230, 100, 101)])
def test_prompt_then_decode(cuda_ok, lens):
    import hybrid_decode as ex
    r = ex.run_prompt(lens)
    s = r["stack"]
    assert r["status"] == 0 and len(r["log"]) == 5
    # the sampling's decisions are those of its definition, from the same numbers
    for x in r["log"]:
        for b in range(ex.B):
            path, nxt, near = A.sample(x["tokens"][b].tolist(), list(range(-1, ex.T - 1)), R.f64(x["probs"][b]),
                                       R.f64(x["draft"][b]), R.f64(x["u"][b]), ex.T)
            assert near > 1e-9 and (x["taken"][b], x["next"][b]) == (len(path), nxt)
    assert sum(sum(x["taken"]) for x in r["log"]) > 5 * ex.B         # (some drafts were accepted)
    for a, b in zip(r["log"], r["log"][1:]):
        assert b["tokens"][:, 0].tolist() == a["next"]
    # every layer's state is that of the committed tokens in a row
    assert s.cache.seq_len[:ex.B].tolist() == [len(t) for t in r["committed"]]
    w = R.f64(s.conv.t["weight"])
    for b, t in enumerate(r["committed"]):
        x = R.f64(s.embed[t])
        y, window, _ = A.conv(np.zeros((ex.W - 1, ex.C)), x, w, np.zeros(ex.C), True)
        p, cap = int(s.conv.t["pos"][b]), s.conv.d.cap
        assert p == len(t) % cap
        for j in range(1, ex.W):
            assert (R.f64(s.conv.t["ring"][b, (p - j) % cap]) == window[ex.W - 1 - j]).all()
        y = torch.from_numpy(y).cuda().bfloat16()
        q, k, v, g, beta = s.mixed(torch.tensor(t), y)
        _, S, norm, eff = A.advance(np.zeros((ex.H, ex.D, ex.D)), *(R.f64(z) for z in (q, k, v, g, beta)), ex.D ** -0.5)
        # k and v of both sides are off by a rounding to bf16 each at most (2^-8, in y and again in k): a step's update
        # beta (v - S k) k^T by 2 * 2^-8 of v, of S and, with k's second factor, of both: 8 * 2^-8 of the norms
        # (a token missed or taken twice is off by a whole update)
        tol = A.advance_bound(norm, eff, ex.D, True) + 2.0 ** -5 * norm * eff
        assert np.abs(R.f64(s.gdn.t["state"][b]) - S).max() <= tol
    # the last block's attention over the cache's rows
    x = r["log"][-1]
    for b in range(ex.B):
        ln = x["lengths"][b]
        k, v = rows(s.cache, s.cache.k, b, ln + ex.T), rows(s.cache, s.cache.v, b, ln + ex.T)
        o, e, At, St = R.attention(R.f64(x["q"][b]), k, v, [(2 << i) - 1 for i in range(ex.T)], ln, ex.D ** -0.5)
        to, _ = R.verify_bounds(At, St, e, ln + ex.T, ex.D, True)
        assert (np.abs(R.f64(x["att"][b]) - o) <= to).all(), b


def test_decode_continues_a_prompt_like_a_longer_prompt(cuda_ok):
    """The committed tokens of prompt and rounds as one prompt: the same states, but for the roundings to bf16 between
    the layers."""
    import hybrid_decode as ex
    r = ex.run_prompt((150, 70, 1))
    s = ex.Stack(torch.Generator().manual_seed(3))
    n = [len(t) for t in r["committed"]]
    for at in range(0, max(n), ex.PART):
        part = torch.zeros(ex.B, ex.PART, dtype=torch.long)
        m = [min(max(x - at, 0), ex.PART) for x in n]
        for b in range(ex.B):
            part[b, :m[b]] = torch.tensor(r["committed"][b][at:at + ex.PART])
        s.prompt(part.cuda(), ex.i32(m), fresh=ex.i32([at == 0] * ex.B))
    torch.cuda.synchronize()
    assert int(s.cache.status.item()) | int(s.gdn.status.item()) | int(s.conv.status.item()) == 0
    assert s.cache.seq_len[:ex.B].tolist() == n
    for b in range(ex.B):
        a, c = R.f64(r["stack"].gdn.t["state"][b]), R.f64(s.gdn.t["state"][b])
        assert np.abs(a - c).max() <= 2.0 ** -6 * np.abs(c).max()
        # keys are of norm about sqrt(d) after the norm; a value's entry is off by its inputs' roundings
        for x, y in ((r["stack"].cache.k, s.cache.k), (r["stack"].cache.v, s.cache.v)):
            x, y = rows(r["stack"].cache, x, b, n[b]), rows(s.cache, y, b, n[b])
            assert np.sqrt(((x - y) ** 2).mean()) <= 2.0 ** -6 * np.sqrt((y ** 2).mean())
