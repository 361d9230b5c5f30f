"""gdn_attn_chunk with FLAG_TWO_TERMS: within the verify's bounds, which have no 2^-8 of a weight, at any number of tokens; and what the flag costs
nothing of: fp32, short chunks, the other calls of a layer."""
import math

import numpy as np
import pytest
import torch

import attn_bounds
import attn_ref as R
from test_gpu_attn_chunk import BF, F32, SHAPES, Case, i32, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


class Two(Case):
    def __init__(self, *a, **kw):
        import speculative_decode_recurrent_gb300 as lib
        super().__init__(*a, **kw)
        d = self.layer.d
        self.one = self.layer
        self.layer = lib.AttnLayer(lib.AttnDims(B=d.B, T=d.T, Hq=d.Hq, scale=d.scale, flags=lib.FLAG_TWO_TERMS), self.cache, self.c.layers - 1,
                                   state_idx=self.layer.state_idx)

    def check_tight(self):
        c = self.c
        torch.cuda.synchronize()
        assert int(self.cache.status.item()) == 0
        out, lse = R.f64(self.out), R.f64(self.lse)
        for b, n in enumerate(self.lens):
            m = self.past[b] + n
            if n:
                k, v = (c.rows(x, b, m, c.layers - 1) for x in (c.k, c.v))
                ref, rl, A, S = reference(R.f64(self.q[b, :n]), k, v, self.past[b], self.scale)
                tol = attn_bounds.verify_bounds(ref, A, S, m, c.d, c.dtype == BF)
                assert (np.abs(out[b, :n] - ref) <= tol).all(), (b, n, (np.abs(out[b, :n] - ref) / tol).max())
            assert (out[b, n:] == 0).all() and (lse[b, n:] == -math.inf).all()


@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_within_the_bounds_of_a_verify(shape):
    c = Two(*shape, BF, seed=31)
    c.run()
    c.check_tight()


@pytest.mark.parametrize("T", [64, 65])
def test_short_and_long_chunks_are_equally_near(T):
    """The outputs' own rounding is what is left of the error, on either side of 64 tokens."""
    c = Two([700], [T], T, 16, 2, 128, 16, BF, seed=46)
    c.run()
    c.check_tight()
    k, v = (c.c.rows(x, 0, 700 + T, c.c.layers - 1) for x in (c.c.k, c.c.v))
    ref = reference(R.f64(c.q[0]), k, v, 700, c.scale)[0]
    rounded = R.f64(torch.from_numpy(ref).to(BF))
    err, own = (np.sqrt(np.square(x - ref).mean()) for x in (R.f64(c.out[0]), rounded))
    assert err <= 1.01 * own + 2.0 ** -15 * np.sqrt(np.square(ref).mean())


def test_the_flag_changes_nothing_else():
    import speculative_decode_recurrent_gb300 as lib
    for dtype, T in ((F32, 100), (BF, 40)):
        c = Two([300, 20], [T, T - 7], T, 4, 2, 64, 16, dtype, seed=47)
        c.run()
        c.check_tight()
        out, lse = c.out.clone(), c.lse.clone()
        c.one.chunk(c.qd, c.out, lse=c.lse, chunk_len=i32(c.lens))
        torch.cuda.synchronize()
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)
    c.out.fill_(1)
    c.layer.verify(c.qd, c.out, lse=c.lse, draft_len=i32(c.lens))
    torch.cuda.synchronize()
    assert torch.equal(out, c.out)
    with pytest.raises(lib.GdnError):
        lib.AttnLayer(lib.AttnDims(B=2, T=40, Hq=4, scale=0.1, flags=2), c.cache, 0)


def test_graph_and_many_units():
    c = Two([0, 3, 300, 64] * 4, [130, 80, 1, 0, 65, 127, 128, 129, 66, 130, 9, 100, 130, 2, 78, 130], 130, 16, 2, 128, 16, BF, seed=48)
    lens = i32(c.lens)
    c.layer.chunk(c.qd, c.out, lse=c.lse, chunk_len=lens)
    c.check_tight()
    out = c.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.layer.chunk(c.qd, c.out, lse=c.lse, chunk_len=lens)
    for _ in range(20):
        c.out.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, out)


def test_expired_wait_writes_nothing():
    import speculative_decode_recurrent_gb300 as lib
    c = Two([100], [80], 80, 4, 2, 128, 16, BF, seed=49)
    bad = lib.AttnLayer(lib.AttnDims(B=1, T=80, Hq=4, scale=c.scale, flags=lib.FLAG_TEST_EXPIRE | lib.FLAG_TWO_TERMS), c.cache, 1,
                        state_idx=c.layer.state_idx)
    bad.chunk(c.qd, c.out, lse=c.lse)
    torch.cuda.synchronize()
    assert int(c.cache.status.item()) == lib.STATUS_TIMEOUT
    c.cache.status.zero_()
    c.run()
    c.check_tight()
