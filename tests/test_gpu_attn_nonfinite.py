"""Draft values that are not finite, in every way in which the tensor-core verify lays its work
out: several row tiles per key head (taken in pairs, singly, or without rows in use), several of
them in turn on one CTA, draft rows over one or two tiles of keys.

A row's output in a column is the plain form's over the finite values, plus the infinities and NaN
of the tokens that it sees there; bounds as in attn_ref.verify_bounds.
"""
import numpy as np
import pytest
import torch

import attn_ref as R
from test_gpu_attn import BF, F32, VerifyRun

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def _batch(B, T, lo, hi):
    """Ragged lengths in a mixed order, and drafts of which some leave whole row tiles unused."""
    lens = [lo + (hi - lo) * ((b * 37) % B) // B for b in range(B)]
    return lens, [(T, T // 3, 3, 2 * T // 3, T // 2 - 1, T - 7, 1, T // 3 + 1, 0)[b % 9] for b in range(B)]


# batch, draft, heads, head size, page, lengths.  In the first five, CTAs (of 152) go from a single row
# tile of an odd number of tiles to a pair of row tiles whose draft tile they hold.
CASES = [
    (40, 48, 16, 2, 128, 16, 0, 300, BF),
    (40, 40, 24, 2, 64, 64, 0, 400, BF),
    (30, 64, 16, 2, 128, 64, 0, 260, BF),
    (16, 64, 40, 2, 64, 16, 3, 200, BF),
    (24, 40, 32, 4, 128, 64, 0, 2000, BF),                   # a unit's beginning and end count as work
    (9, 50, 9, 3, 256, 16, 0, 300, BF),                      # one group
    (20, 16, 16, 2, 128, 32, 0, 900, BF),                    # one row tile: the groups alternate
    (9, 20, 8, 2, 64, 16, 0, 200, F32),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_verify_non_finite_drafts(i):
    B, T, Hq, Hkv, d, page, lo, hi, dtype = CASES[i]
    lens, drafts = _batch(B, T, lo, hi)
    g = torch.Generator().manual_seed(500 + i)
    par = R.random_parents(B, T, g, width=6)
    words = [R.ancestors(par[b], T)[0] for b in range(B)]
    r = VerifyRun(lens, drafts, T, Hq, Hkv, d, page, dtype, words=words, seed=510 + i)
    c, G = r.case, Hq // Hkv
    odd = np.zeros((B, T, Hkv, d))                           # the non-finite values by draft token
    for b, n in enumerate(drafts):
        if b % 5 == 4:
            continue                                         # some sequences without any
        for t, col, y in ((n - 1, b % d, np.inf), (n // 2, (7 * b + 1) % d, -np.inf), (n // 3, d - 1, np.nan),
                          (1, (3 * b) % d, np.inf)):
            if 0 <= t < n:
                odd[b, t, b % Hkv, col] = y
                p, row = c.cell(b, lens[b] + t)
                c.v[:, p, b % Hkv, row, col] = y
    r.cache.v.copy_(c.v)
    r.call()
    assert int(r.cache.status.item()) == 0 and r.out_ok() and r.lse_ok()
    out, lse = R.f64(r.out), R.f64(r.lse)
    for b, n in enumerate(drafts):
        k, v = (c.rows(x, b, lens[b] + n) for x in (c.k, c.v))
        v = np.where(np.isfinite(v), v, 0.0)
        o, e, A, S = R.attention(R.f64(r.q[b, :n]), k, v, words[b], lens[b], r.scale)
        to, te = R.verify_bounds(A, S, e, lens[b] + n, d, dtype == BF)
        extra = np.zeros((n, Hkv, d))
        with np.errstate(invalid="ignore"):
            for t in range(n):
                for u in range(n):
                    if (words[b][t] >> u) & 1:
                        extra[t] += odd[b, u]
        extra = np.repeat(extra, G, 1)
        want = extra != 0                                    # (NaN too)
        got = out[b, :n]
        np.testing.assert_array_equal(got[want], extra[want], err_msg=f"sequence {b}")
        assert np.isfinite(got[~want]).all(), b
        assert (np.abs(got - o)[~want] <= to[~want]).all(), b
        assert (np.abs(lse[b, :n] - e) <= te).all(), b
        assert (out[b, n:] == 0).all() and np.isneginf(lse[b, n:]).all(), b
    first = r.out.clone(), r.lse.clone()
    r.call()                                                 # the words of the call before are clear
    assert torch.equal(first[0].view(torch.uint8), r.out.view(torch.uint8)) and torch.equal(first[1], r.lse)


@pytest.mark.parametrize("d", [64, 128])
def test_verify_nan_keys_in_pairs(d):
    """A drafted token's NaN key reaches the rows that see it, in every row tile, and no other; the same bits
    for those as without it."""
    B, T, Hq, Hkv = 6, 48, 16, 2
    lens, drafts = _batch(B, T, 0, 300)
    g = torch.Generator().manual_seed(530)
    par = R.random_parents(B, T, g, width=6)
    words = [R.ancestors(par[b], T)[0] for b in range(B)]
    r = VerifyRun(lens, drafts, T, Hq, Hkv, d, 32, BF, words=words, seed=531)
    r.call()
    r.check()
    clean = R.f64(r.out)
    at = [max(0, n - 20) for n in drafts]
    for b, n in enumerate(drafts):
        if n:
            p, row = r.case.cell(b, lens[b] + at[b])
            r.cache.k[0, p, :, row] = float("nan")
    r.call()
    out, lse = R.f64(r.out), R.f64(r.lse)
    seen_by = 0
    for b, n in enumerate(drafts):
        sees = np.array([(words[b][t] >> at[b]) & 1 for t in range(n)], bool)
        seen_by += sees.sum()
        assert np.isnan(out[b, :n][sees]).all() and np.isnan(lse[b, :n][sees]).all(), b
        np.testing.assert_array_equal(out[b, :n][~sees], clean[b, :n][~sees])
    assert seen_by > B                                       # more than the tokens themselves
