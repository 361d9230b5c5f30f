"""Infinite and NaN values and keys among a chunk's own tokens: they reach the rows that see them and none before."""
import numpy as np
import pytest
import torch

import attn_bounds
import attn_ref as R
from test_gpu_attn_chunk import BF, F32, Case, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


class Odd(Case):
    """(``flags``: of the layer's dims.)  ``values``: (sequence, token of the whole context, key head, column, number); ``keys``: (sequence, token, key head)."""

    def __init__(self, *a, flags=0, **kw):
        import speculative_decode_recurrent_gb300 as lib
        super().__init__(*a, **kw)
        self.one_term = self.c.dtype == BF and not flags
        if flags:
            d = self.layer.d
            self.layer = lib.AttnLayer(lib.AttnDims(B=d.B, T=d.T, Hq=d.Hq, scale=d.scale, flags=flags), self.cache, self.c.layers - 1,
                                       state_idx=self.layer.state_idx)

    def spoil(self, values, keys=()):
        c = self.c
        self.odd = [np.zeros((self.past[b] + n, c.Hkv, c.d), bool) for b, n in enumerate(self.lens)]
        self.bad_keys = keys
        for b, t, h, col, y in values:
            pg, row = c.cell(b, t)
            c.v[-1, pg, h, row, col] = y
            self.odd[b][t, h, col] = True
        for b, t, h in keys:
            pg, row = c.cell(b, t)
            c.k[-1, pg, h, row, t % c.d] = float("nan")
        self.cache.k.copy_(c.k)
        self.cache.v.copy_(c.v)

    def check_odd(self):
        c, G = self.c, self.qd.shape[2] // self.c.Hkv
        torch.cuda.synchronize()
        assert int(self.cache.status.item()) == 0
        out, bf = R.f64(self.out), c.dtype == BF
        for b, n in enumerate(self.lens):
            m, past = self.past[b] + n, self.past[b]
            k, v = (c.rows(x, b, m, c.layers - 1) for x in (c.k, c.v))
            v = np.where(self.odd[b], 0.0, v)
            nan_from = np.full(c.Hkv, m)                     # the first row that sees a NaN key, by key head
            for bb, t, h in self.bad_keys:
                if bb == b:
                    nan_from[h] = min(nan_from[h], t)
                    k[t, h] = 0.0
            ref, _, A, S = reference(R.f64(self.q[b, :n]), k, v, past, self.scale)
            tol = attn_bounds.verify_bounds(ref, A, S, m, c.d, bf) + (1.01 * 2.0 ** -8 * A if self.one_term else 0)
            seen = np.cumsum(self.odd[b], 0)[past:] > 0       # [n, Hkv, d]
            seen = seen | (np.arange(past, m)[:, None] >= nan_from)[:, :, None]
            seen = np.repeat(seen, G, 1)
            got = out[b, :n]
            assert not np.isfinite(got[seen]).any(), b
            assert (np.abs(got - ref)[~seen] <= tol[~seen]).all(), (b, np.argwhere(~(np.abs(got - ref) <= tol) & ~seen)[:5])
            assert (out[b, n:] == 0).all()


SHAPES = [
    # past, lens, T, Hq, Hkv, d, page
    ([0, 60, 130], [300, 299, 1], 300, 16, 2, 128, 64),      # several pairs of row tiles, both groups on a tile
    ([0, 500], [65, 130], 130, 2, 2, 64, 16),                # one query head per key head: a pair sees 256 tokens
    ([77], [260], 260, 10, 2, 128, 32),                      # five: every tile has rows that are not in use
    ([100, 0], [200, 90], 200, 8, 2, 256, 16),               # halves of the values, tiles of 64 keys
    ([6000], [100], 100, 16, 2, 128, 128),                   # keys in parts
    ([20001], [66], 66, 2, 2, 128, 64),
    ([3000], [96], 96, 64, 1, 64, 64),
]


@pytest.mark.parametrize("dtype,flags", [(BF, 0), (F32, 0), (BF, 4)])          # (4: FLAG_TWO_TERMS)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_values_reach_the_rows_that_see_them(i, dtype, flags):
    c = Odd(*SHAPES[i], dtype, seed=71, flags=flags)
    d, Hkv, inf, values = c.c.d, c.c.Hkv, float("inf"), []
    for b, n in enumerate(c.lens):
        at = sorted({n - 1, n // 2, n // 3, min(n - 1, 1), min(n - 1, 15), min(n - 1, 16), min(n - 1, 47), min(n - 1, 64), 3 * n // 4})
        for j, t in enumerate(at):
            values.append((b, c.past[b] + t, j % Hkv, (17 * j + 5 * b) % d, (inf, -inf, float("nan"))[j % 3]))
        if c.past[b] > 50:                                   # a committed one: every row sees it
            values.append((b, c.past[b] - 40, 0, d - 1, inf))
    c.spoil(values)
    c.run()
    c.check_odd()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", [0, 1, 3, 4])
def test_keys_reach_the_rows_that_see_them(i, dtype):
    c = Odd(*SHAPES[i], dtype, seed=72)
    c.spoil([(0, c.past[0] + c.lens[0] // 2, 0, 3, float("inf"))], [(0, c.past[0] + 2 * c.lens[0] // 3, 0)])
    c.run()
    c.check_odd()


@pytest.mark.parametrize("d,Hq", [(64, 2), (128, 16), (256, 8)])
def test_a_whole_token_of_nan_and_many_units(d, Hq):
    """Tokens of NaN alone in some of many sequences, so that a CTA's later units are others'; the second call gives the same bits."""
    B = 40
    c = Odd([10 * (b % 7) for b in range(B)], [130 - (b * 13) % 66 for b in range(B)], 130, Hq, 2, d, 16, BF, seed=73)
    c.spoil([(b, c.past[b] + (b * 29) % c.lens[b], h, x, float("nan")) for b in range(0, B, 3) for h in range(2) for x in range(d)])
    c.run()
    c.check_odd()
    first = c.out.clone()
    c.out.fill_(1)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out.view(torch.int16), first.view(torch.int16))
