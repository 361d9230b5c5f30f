"""The example that runs the recurrent and the attention operators together."""
import os
import sys

import numpy as np
import pytest
import torch

import attn_ref as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def _rows(cache, x, slot, n):
    pos = torch.arange(n)
    ids = cache.block_table[slot].cpu()[pos // cache.d.page].long()
    return R.f64(x[0].cpu()[ids, :, pos % cache.d.page])


def test_hybrid_decode(cuda_ok):
    import hybrid_decode as ex
    r = ex.run()
    cache = r["cache"]
    assert r["status"] == 0
    assert r["lengths"][:ex.B] == r["committed"] and r["lengths"][ex.B:] == [0] * (ex.SLOTS - ex.B)
    # the fork was released: every page is free or held once
    owned = int(cache.n_owned.sum())
    assert int(cache.free_count) == cache.d.n_page - owned and int(cache.ref.sum()) == owned
    # the last step's outputs from the cache (its accepted rows are still where they were staged)
    for b in range(ex.B):
        n = ex.T
        ln = _last_context(r, b)
        k, v = _rows(cache, cache.k, b, ln + n), _rows(cache, cache.v, b, ln + n)
        o, e, A, S = R.attention(R.f64(r["q"][b]), k, v, [(2 << t) - 1 for t in range(n)], ln, ex.D ** -0.5)
        to, _ = R.verify_bounds(A, S, e, ln + n, ex.D, True)
        assert (np.abs(R.f64(r["att"][b]) - o) <= to).all(), b


def _last_context(r, b):
    """Committed tokens of sequence b before the last step's accept: the buffer of the recurrent
    layer and the cache move by the same counts, so the last count follows from the draws."""
    import hybrid_decode as ex
    g = torch.Generator().manual_seed(1)
    torch.randn(2, ex.D, generator=g)
    torch.randn(ex.H * ex.D, (ex.H + 2 * ex.HKV) * ex.D, generator=g)
    for _ in range(6):
        for _ in range(3):
            torch.randn(ex.B, ex.T, ex.H, ex.D, generator=g)
        torch.rand(ex.B, ex.T, ex.H, generator=g)
        torch.rand(ex.B, ex.T, ex.H, generator=g)
        p = torch.randint(0, ex.T + 1, (ex.B,), generator=g).tolist()
    return r["committed"][b] - p[b]


def test_tree_step(cuda_ok):
    import hybrid_decode as ex
    t = ex.run_tree()
    cache, n, ln = t["cache"], ex.T, t["context"]
    assert t["status"] == 0 and cache.seq_len[:ex.B].tolist() == [ln + 5] * ex.B
    assert t["pos"][0].tolist() == [ln + x for x in (0, 1, 1, 2, 2, 3, 2, 4)]
    words = [int(w) for w in t["tree"][0].tolist()]
    assert words == R.ancestors([-1, 0, 0, 1, 1, 3, 2, 5], n)[0]
    for b in range(ex.B):
        before = _rows(cache, t["staged"], b, ln + n)       # the keys as they were staged
        v_now = _rows(cache, cache.k, b, ln + 5)
        np.testing.assert_array_equal(v_now[:ln], before[:ln])
        np.testing.assert_array_equal(v_now[ln:], before[ln + np.array([0, 1, 3, 5, 7])])
