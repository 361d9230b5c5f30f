"""gdn_attn_chunk against a plain 64-bit form: lengths around the tiles, odd groups, every head dim and page size,
unused rows, garbage behind the last token."""
import math

import numpy as np
import pytest
import torch

import attn_bounds
import attn_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def reference(q, k, v, ln, scale):
    """q [n, Hq, d], k, v [ln + n, Hkv, d]: out, lse and the bounds' A and S (tests/attn_ref.py), head by head."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    out, A = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, S = np.zeros((n, Hq)), np.zeros((n, Hq))
    seen = np.arange(len(k))[None] <= ln + np.arange(n)[:, None]
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        s = np.where(seen, q[:, h] @ kk.T * scale, -np.inf)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(1, keepdims=True)
        out[:, h], A[:, h] = p @ vv / l, p @ np.abs(vv) / l
        lse[:, h] = (m + np.log(l))[:, 0]
        S[:, h] = np.where(seen, np.abs(q[:, h]) @ np.abs(kk).T * scale, 0).max(1)
    return out, lse, A, S


class Case:
    def __init__(self, past, lens, T, Hq, Hkv, d, page, dtype, seed=0, layers=2):
        import speculative_decode_recurrent_gb300 as lib
        g = torch.Generator().manual_seed(seed)
        self.past, self.lens, self.T, self.scale = past, lens, T, d ** -0.5
        c = self.c = R.CacheCase(past, T, Hkv, d, page, dtype, layers=layers, seed=seed + 1)
        for b, n in enumerate(lens):                         # what lies behind the chunk's end
            for t in range(past[b] + n, past[b] + T):
                pg, row = c.cell(b, t)
                c.k[:, pg, :, row], c.v[:, pg, :, row] = float("nan"), float("inf")
        self.cache = lib.PagedCache(c.dims(lib), c.init())
        self.layer = lib.AttnLayer(lib.AttnDims(B=len(past), T=T, Hq=Hq, scale=self.scale), self.cache, layers - 1,
                                   state_idx=c.state_idx.cuda())
        self.q = (1.3 * torch.randn(len(past), T, Hq, d, generator=g)).to(dtype)
        for b, n in enumerate(lens):
            self.q[b, n:] = float("nan")
        self.qd = self.q.cuda()
        self.out = torch.full_like(self.qd, 7.0)
        self.lse = torch.full((len(past), T, Hq), 7.0, device="cuda")

    def run(self, **kw):
        self.layer.chunk(self.qd, self.out, lse=self.lse, chunk_len=i32(self.lens), **kw)

    def check(self, only=None):
        c = self.c
        torch.cuda.synchronize()
        out, lse, bf = R.f64(self.out), R.f64(self.lse), c.dtype == BF
        for b, n in enumerate(self.lens):
            if only is not None and b not in only:
                continue
            m = self.past[b] + n
            if n:
                k, v = (c.rows(x, b, m, c.layers - 1) for x in (c.k, c.v))
                ref, rl, A, S = reference(R.f64(self.q[b, :n]), k, v, self.past[b], self.scale)
                tol = attn_bounds.verify_bounds(ref, A, S, m, c.d, bf)
                if bf:                                       # a weight as one bf16 term: 2^-8 of it
                    tol = tol + 1.01 * 2.0 ** -8 * A
                assert (np.abs(out[b, :n] - ref) <= tol).all(), (b, n, np.abs(out[b, :n] - ref).max())
                # scores: (d + 8) 2^-24 S; the sum of m weights of relative error 2^-21, and the logarithm
                ltol = 1.01 * ((c.d + 8) * 2.0 ** -24 * S + (m * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -21 * np.abs(rl))
                assert (np.abs(lse[b, :n] - rl) <= ltol).all(), (b, np.abs(lse[b, :n] - rl).max())
            assert (out[b, n:] == 0).all() and (lse[b, n:] == -math.inf).all()


SHAPES = [
    # past, lens, T, Hq, Hkv, d, page
    ([0], [65], 65, 1, 1, 64, 16),
    ([0, 63, 130], [200, 1, 0], 200, 4, 2, 128, 16),
    ([1], [127], 127, 2, 2, 128, 32),
    ([128], [128], 128, 8, 1, 128, 128),
    ([300, 0], [129, 77], 129, 10, 2, 64, 64),
    ([5, 1000], [140, 139], 150, 7, 1, 256, 32),
    ([77], [260], 260, 12, 3, 128, 64),
    ([0, 0, 0], [66, 100, 33], 100, 3, 3, 256, 128),
    ([2000], [70], 70, 64, 1, 64, 16),
    ([3000], [96], 96, 16, 1, 128, 64),
    ([0], [700], 700, 5, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_chunk_matches_the_formula(shape, dtype):
    c = Case(*shape, dtype, seed=31)
    c.run()
    c.check()
    assert int(c.cache.status.item()) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 17, 64])
def test_short_chunks_are_a_verify(T, dtype):
    c = Case([40, 0], [T, T - 1], T, 4, 2, 64, 16, dtype, seed=32)
    c.run()
    c.check()


def test_many_units_and_split_keys():
    """More CTAs than SMs (no parts), and one row tile over a long context (many parts)."""
    c = Case([10] * 6, [600, 511, 512, 513, 90, 600], 600, 8, 2, 128, 64, BF, seed=33, layers=1)
    c.run()
    c.check()
    c = Case([20001], [66], 66, 2, 2, 128, 64, BF, seed=34, layers=1)
    assert c.layer.workspace.numel() > 0
    c.run()
    c.check()


def test_scores_that_rise_and_fall():
    """Keys whose scores grow along the context (every tile rescales) and a first tile far above the rest."""
    for sign in (1, -1):
        c = Case([900], [130], 130, 2, 1, 128, 16, BF, seed=35)
        ramp = torch.linspace(0, 40, 1030)
        ramp = ramp if sign > 0 else ramp.flip(0)
        u = torch.zeros(128)
        u[0] = 1.0
        for t in range(1030):
            pg, row = c.c.cell(0, t)
            c.c.k[:, pg, :, row, 0] = ramp[t].bfloat16()
        c.cache.k.copy_(c.c.k)
        c.q[0, :, :, 0] = 3.0
        c.qd.copy_(c.q)
        c.run()
        c.check()


def test_bad_sequences_are_skipped():
    import speculative_decode_recurrent_gb300 as lib
    c = Case([40, 50, 60, 70], [80, 80, 80, 80], 80, 4, 2, 128, 16, BF, seed=36)
    idx = c.layer.state_idx
    c.cache.n_owned[int(idx[1])] -= 1
    c.cache.seq_len[int(idx[2])] = -1
    idx[0] = 1000
    c.run()
    torch.cuda.synchronize()
    assert int(c.cache.status.item()) == lib.STATUS_BAD_SLOT | lib.STATUS_BAD_PAGE | lib.STATUS_BAD_LEN
    assert (c.out[:3] == 7).all() and (c.lse[:3] == 7).all()
    c.check(only=[3])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_graph_and_stream_give_the_same_bits(dtype):
    c = Case([500, 20], [150, 149], 150, 8, 2, 128, 16, dtype, seed=37)
    lens = i32(c.lens)
    c.layer.chunk(c.qd, c.out, lse=c.lse, chunk_len=lens)
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.out.fill_(1)
    side.wait_stream(torch.cuda.current_stream())
    c.layer.chunk(c.qd, c.out, lse=c.lse, chunk_len=lens, stream=side)
    side.synchronize()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.layer.chunk(c.qd, c.out, lse=c.lse, chunk_len=lens)
    for _ in range(2):
        c.out.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_expired_wait_writes_nothing(d):
    import speculative_decode_recurrent_gb300 as lib
    c = Case([100], [80], 80, 4, 2, d, 16, BF, seed=38)
    bad = lib.AttnLayer(lib.AttnDims(B=1, T=80, Hq=4, scale=c.scale, flags=lib.FLAG_TEST_EXPIRE), c.cache, 1,
                        state_idx=c.c.state_idx.cuda())
    bad.chunk(c.qd, c.out, lse=c.lse)
    torch.cuda.synchronize()
    assert int(c.cache.status.item()) == lib.STATUS_TIMEOUT
    c.cache.status.zero_()
    c.run()                                                  # and the next call is sound
    c.check()


def test_a_layer_for_staging_takes_a_smaller_workspace():
    """A layer of more tokens than a verify takes may share a verify's workspace; chunk refuses one that it needs more of."""
    import speculative_decode_recurrent_gb300 as lib
    c = Case([5000], [100], 100, 4, 2, 128, 16, BF, seed=39)     # (long enough for parts of the keys)
    idx = c.layer.state_idx
    dims = lib.AttnDims(B=1, T=100, Hq=4, scale=c.scale)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    layer = lib.AttnLayer(dims, c.cache, 1, state_idx=idx, workspace=small)
    assert c.layer.workspace.numel() > 16
    with pytest.raises(ValueError, match="chunk: needs a workspace"):
        layer.chunk(c.qd, c.out)
    with pytest.raises(ValueError, match="workspace"):
        lib.AttnLayer(lib.AttnDims(B=1, T=64, Hq=4, scale=c.scale), c.cache, 1, state_idx=idx, workspace=small)
    other = lib.AttnLayer(dims, c.cache, 1, state_idx=idx, workspace=c.layer.workspace)
    other.chunk(c.qd, c.out, lse=c.lse, chunk_len=i32(c.lens))
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_sequences_and_wrong_tensors(dtype):
    import speculative_decode_recurrent_gb300 as lib
    c = Case([30], [70], 70, 4, 2, 128, 16, dtype, seed=40)
    none = lib.AttnLayer(lib.AttnDims(B=0, T=70, Hq=4, scale=c.scale), c.cache, 0)
    none.chunk(c.qd[:0], c.out[:0])
    for bad in (c.qd[:, :69].contiguous(), c.qd.float() if dtype == BF else c.qd.bfloat16(), c.qd.cpu(), c.qd.transpose(1, 2)):
        with pytest.raises((ValueError, TypeError)):
            c.layer.chunk(bad, c.out)
    assert (c.out == 7).all()


@pytest.mark.parametrize("past,T", [(0, 130), (1500, 80)])
def test_outputs_on_any_16_byte_boundary(past, T):
    c = Case([past], [T - 3], T, 6, 2, 128, 16, BF, seed=41)
    room = torch.full((c.out.numel() + 16,), 7.0, dtype=BF, device="cuda")
    c.out = room[8:-8].view(c.out.shape)
    assert c.out.data_ptr() % 32 == 16
    c.run()
    c.check()
    assert (room[:8] == 7).all() and (room[-8:] == 7).all()


@pytest.mark.parametrize("d,Hq,Hkv", [(256, 8, 2), (128, 16, 2), (64, 16, 2)])
def test_many_short_units_and_calls(d, Hq, Hkv):
    """Prompts of a few tiles, so that a CTA takes many units one after the other, and many calls in a row: every one gives
    the first one's bits."""
    c = Case([0, 3, 300, 64] * 4, [130, 80, 1, 0, 65, 127, 128, 129, 66, 130, 9, 100, 130, 2, 78, 130], 130, Hq, Hkv, d, 16, BF, seed=42)
    lens = i32(c.lens)
    c.layer.chunk(c.qd, c.out, lse=c.lse, chunk_len=lens)
    first = c.out.clone(), c.lse.clone()
    c.check()
    for _ in range(200):
        c.layer.chunk(c.qd, c.out, lse=c.lse, chunk_len=lens)
    torch.cuda.synchronize()
    assert int(c.cache.status.item()) == 0
    assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


def test_calls_on_two_streams_at_once():
    """Two layers' chunks, one whose keys are cut and one of many units, on two streams: the bits of one after the other."""
    cases = [Case([6000], [120], 120, 16, 2, 128, 16, BF, seed=43), Case([0] * 12, [200, 130, 5, 0] * 3, 200, 16, 2, 128, 16, BF, seed=44),
             Case([900, 0], [140, 77], 140, 8, 2, 256, 16, BF, seed=45)]
    lens, want = [i32(c.lens) for c in cases], []
    for c in cases:
        c.run()
        torch.cuda.synchronize()
        want.append((c.out.clone(), c.lse.clone()))
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        for c in cases:
            c.out.fill_(3)
        torch.cuda.synchronize()
        for _ in range(3):
            for c, n, stream in zip(cases, lens, streams):
                c.layer.chunk(c.qd, c.out, lse=c.lse, chunk_len=n, stream=stream)
        torch.cuda.synchronize()
        for c, (out, lse) in zip(cases, want):
            assert torch.equal(c.out, out) and torch.equal(c.lse, lse) and int(c.cache.status.item()) == 0
