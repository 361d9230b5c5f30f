"""The verify tests' bounds tell a wrong page of values from rounding at the longest contexts that
they use.  64-bit forms only, no GPU."""
import numpy as np
import pytest
import torch

import attn_bounds
import attn_ref as R

# tokens, draft, query and key heads, head size, page: as in test_gpu_attn_long.py
LONG = [(40007, 16, 16, 2, 128, 64), (20011, 17, 8, 1, 128, 64), (52000, 2, 16, 2, 256, 64), (30000, 5, 8, 4, 64, 64),
        (12345, 5, 8, 1, 128, 16)]


@pytest.mark.parametrize("marks", [True, False])
@pytest.mark.parametrize("i", range(len(LONG)))
def test_a_wrong_page_of_values_is_out_of_bounds(i, marks):
    """Every sampled page's values replaced by its neighbour's (marked columns), or by others of the same
    distribution: some element moves by more than it may.  (With values of mean zero a page
    of little weight may stay inside; most do not.)"""
    ln, n, Hq, Hkv, d, page = LONG[i]
    g = torch.Generator().manual_seed(i)
    n = min(n, 4)                                            # rows enough to show it
    k = R.f64((1.3 * torch.randn(ln + n, Hkv, d, generator=g)).bfloat16())
    v = attn_bounds.page_marks(ln + n, Hkv, d, page, g) if marks else torch.randn(ln + n, Hkv, d, generator=g)
    v, q = R.f64(v.bfloat16()), R.f64((1.3 * torch.randn(n, Hq, d, generator=g)).bfloat16())
    words, scale = [(2 << t) - 1 for t in range(n)], d ** -0.5
    out, lse, A, S = R.attention(q, k, v, words, ln, scale)
    bound = attn_bounds.verify_bounds(out, A, S, ln + n, d, True)
    G, shown, pages = Hq // Hkv, 0, list(range(0, ln // page - 1, max(1, ln // page // 24)))
    for p in pages:
        rows = slice(p * page, (p + 1) * page)
        other = v[(p + 1) * page:(p + 2) * page] if marks else np.asarray(R.f64(torch.randn(page, Hkv, d, generator=g)))
        moved = np.zeros_like(out)
        for t in range(n):
            for h in range(Hq):
                w = np.exp(k[rows, h // G] @ q[t, h] * scale - lse[t, h])
                moved[t, h] = w @ (other[:, h // G] - v[rows, h // G])
        shown += bool((np.abs(moved) > bound).any())
    assert shown == len(pages) if marks else shown >= 0.75 * len(pages), (shown, len(pages))
