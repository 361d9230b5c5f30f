"""The verify over contexts of thousands of tokens, within bounds that a wrong page of values exceeds
(attn_bounds.py; test_attn_bounds.py shows that it does)."""
import numpy as np
import pytest
import torch

import attn_bounds
import attn_ref as R
from test_gpu_attn import BF, F32, VerifyRun

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


# lengths, drafts, T, query and key heads, head size, page
CASES = [
    ([40007], [16], 16, 16, 2, 128, 64, BF),                 # one unit per head over all CTAs
    ([12345, 1, 64, 3000], [5, 5, 5, 5], 5, 8, 1, 128, 16, BF),
    ([30000, 17, 9000, 20011], [5, 5, 0, 3], 5, 8, 4, 64, 64, BF),
    ([14000, 17, 0, 20011], [40, 40, 0, 17], 40, 32, 4, 128, 64, BF),     # pairs of row tiles
    ([30000, 63, 64, 52000], [7, 7, 1, 2], 7, 16, 2, 256, 64, BF),        # one group
    ([5000, 4999, 2113], [33, 64, 1], 64, 12, 2, 64, 32, BF),
    ([20011], [3], 3, 4, 2, 128, 64, F32),
    ([3000, 777], [5, 4], 5, 12, 3, 64, 16, F32),
]


@pytest.mark.parametrize("marks", [True, False])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_verify_long_contexts(i, marks):
    lens, drafts, T, Hq, Hkv, d, page, dtype = CASES[i]
    r = VerifyRun(lens, drafts, T, Hq, Hkv, d, page, dtype, seed=600 + i)
    c = r.case
    if marks:
        for b, (ln, n) in enumerate(zip(lens, drafts)):
            v = attn_bounds.page_marks(ln + n, Hkv, d, page, c.g).to(dtype)
            at = torch.arange(ln + n)
            ids = c.block_table[int(c.state_idx[b])][at // page].long()
            c.v[0][ids, :, at % page] = v
        r.cache.v.copy_(c.v)
    r.call()
    assert int(r.cache.status.item()) == 0 and r.out_ok() and r.lse_ok()
    out, lse = R.f64(r.out), R.f64(r.lse)
    for b, n in enumerate(drafts):
        k, v = (c.rows(x, b, lens[b] + n) for x in (c.k, c.v))
        o, e, A, S = R.attention(R.f64(r.q[b, :n]), k, v, [(2 << t) - 1 for t in range(n)], lens[b], r.scale)
        bound = attn_bounds.verify_bounds(o, A, S, lens[b] + n, d, dtype == BF)
        err = np.abs(out[b, :n] - o)
        assert (err <= bound).all(), (b, float((err / bound).max()))
        _, te = R.verify_bounds(A, S, e, lens[b] + n, d, dtype == BF)
        assert (np.abs(lse[b, :n] - e) <= te).all(), b
        assert (out[b, n:] == 0).all() and np.isneginf(lse[b, n:]).all(), b
