"""GPU tests of the attention-layer operators (include/gdnattn.h) against their plain
64-bit forms in attn_ref.py.

Bounds, derived from the arithmetic before the first run: verify as in
attn_ref.verify_bounds; stage in fp32: the sum of squares, the root, the weight and the
rotation each contribute a few 2^-24, (d/2 + 16) 2^-24 of the terms' size in all; a bf16
result is the rounding of a value within that band; moved and copied rows, lengths,
tables, counts and free lists: exact.
"""
import numpy as np
import pytest
import torch

import attn_ref as R
from harness import assert_bf16_rounding

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def _lib():
    import speculative_decode_recurrent_gb300 as lib
    return lib


def _guarded(shape, dtype, fill):
    """A tensor inside a larger one whose other elements must stay as they are."""
    n, pad = int(np.prod(shape)), 512
    flat = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")

    def intact():
        a, b = flat[:pad].cpu(), flat[pad + n:].cpu()
        return bool((a == fill).all()) and bool((b == fill).all())
    return flat[pad:pad + n].view(shape), intact


class VerifyRun:
    """One verify over a CacheCase: device tensors, the call, the comparison."""

    def __init__(self, lens, drafts, T, Hq, Hkv, d, page, dtype, words=None, seed=1, layers=1, layer=0):
        lib = _lib()
        self.case = c = R.CacheCase(lens, T, Hkv, d, page, dtype, layers=layers, seed=seed)
        self.B, self.T, self.Hq, self.drafts, self.words, self.layer = len(lens), T, Hq, drafts, words, layer
        for b, n in enumerate(drafts):                        # rows past the draft: nothing staged
            for t in range(n, T):
                p, r = c.cell(b, lens[b] + t)
                c.k[:, p, :, r], c.v[:, p, :, r] = float("nan"), float("inf")
        self.q = (1.3 * torch.randn(self.B, T, Hq, d, generator=c.g)).to(dtype)
        self.scale = d ** -0.5
        self.cache = lib.PagedCache(c.dims(lib), c.init())
        self.attn = lib.AttnLayer(lib.AttnDims(B=self.B, T=T, Hq=Hq, scale=self.scale), self.cache, layer,
                                  state_idx=c.state_idx.cuda())
        self.attn.workspace.fill_(0xFF)                       # no initial content (NaN patterns)
        self.out, self.out_ok = _guarded((self.B, T, Hq, d), dtype, 7.0)
        self.lse, self.lse_ok = _guarded((self.B, T, Hq), F32, 7.0)

    def call(self, stream=None, lse=True):
        tree = None
        if self.words is not None:
            tree = torch.tensor([R.as_int64(w) for w in self.words], dtype=torch.int64).cuda()
        dl = None if self.drafts == [self.T] * self.B else torch.tensor(self.drafts, dtype=torch.int32).cuda()
        q = self.q.cuda()
        torch.cuda.synchronize()
        self.attn.verify(q, self.out, lse=self.lse if lse else None, tree=tree, draft_len=dl, stream=stream)
        torch.cuda.synchronize()

    def check(self, skip=(), status=0):
        c = self.case
        assert int(self.cache.status.item()) == status
        assert self.out_ok() and self.lse_ok()
        out, lse = R.f64(self.out), R.f64(self.lse)
        for b in range(self.B):
            if b in skip:
                continue
            n, ln = self.drafts[b], c.lens[b]
            words = self.words[b] if self.words is not None else [(2 << t) - 1 for t in range(n)]
            k, v = (c.rows(x, b, ln + n, self.layer) for x in (c.k, c.v))
            o, e, A, S = R.attention(R.f64(self.q[b, :n]), k, v, words, ln, self.scale)
            to, te = R.verify_bounds(A, S, e, ln + n, c.d, c.dtype == BF)
            err = np.abs(out[b, :n] - o)
            assert (err <= to).all(), (b, float((err / to).max()))
            fin = np.isfinite(e)
            assert np.array_equal(np.isneginf(lse[b, :n]), ~fin), b
            assert (np.abs(lse[b, :n][fin] - e[fin]) <= te[fin]).all(), b
            assert (out[b, n:] == 0).all() and np.isneginf(lse[b, n:]).all(), b


# key head groups, head sizes, pages that end inside a tile, lengths around page and tile ends,
# drafts of no, one, some and all rows
VERIFY = [
    # lens, drafts, T, Hq, Hkv, d, page
    ([5], [1], 1, 4, 4, 64, 16),
    ([0, 1, 15, 16], [4, 4, 1, 0], 4, 6, 2, 64, 16),
    ([63, 64, 65, 31], [1, 1, 1, 1], 1, 8, 1, 128, 32),
    ([47, 112, 127, 129], [16, 16, 16, 16], 16, 16, 2, 128, 16),
    ([200, 0, 77], [13, 7, 1], 13, 10, 2, 128, 64),
    ([130, 255, 256], [9, 3, 9], 9, 12, 4, 256, 128),
    ([300, 1], [64, 33], 64, 8, 2, 128, 16),
    ([90], [37], 37, 14, 2, 256, 32),
    ([700, 3, 450], [8, 8, 5], 8, 3, 3, 64, 128),
    ([1000], [3], 3, 64, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(VERIFY)))
def test_verify_chain(i, dtype):
    lens, drafts, T, Hq, Hkv, d, page = VERIFY[i]
    r = VerifyRun(lens, drafts, T, Hq, Hkv, d, page, dtype, seed=10 + i)
    r.call()
    r.check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(VERIFY)))
def test_verify_tree(i, dtype):
    lens, drafts, T, Hq, Hkv, d, page = VERIFY[i]
    g = torch.Generator().manual_seed(90 + i)
    par = R.random_parents(len(lens), T, g)
    words = [R.ancestors(par[b], T)[0] for b in range(len(lens))]
    r = VerifyRun(lens, drafts, T, Hq, Hkv, d, page, dtype, words=words, seed=40 + i)
    r.call()
    r.check()


# several row tiles per key head (in pairs, with one left over, with tiles whose rows are all past
# the draft), head groups that do not divide a row tile
ROW_TILES = [
    ([150, 40, 0], [48, 20, 3], 48, 16, 2, 128, 64),        # 3 tiles: a pair and one
    ([70, 300], [64, 17], 64, 16, 1, 64, 16),               # 8 tiles
    ([33, 129], [64, 64], 64, 64, 1, 128, 32),              # 32 tiles, two tokens each
    ([100, 65], [40, 26], 40, 15, 3, 128, 16),              # 25 tokens of 5 heads: 125 rows a tile
    ([513], [64], 64, 24, 2, 64, 128),                      # 10 tokens of 12 heads
    ([77, 5], [50, 50], 50, 9, 3, 256, 16),                 # wide heads: one group, two tiles
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(ROW_TILES)))
def test_verify_row_tiles(i, dtype):
    lens, drafts, T, Hq, Hkv, d, page = ROW_TILES[i]
    par = R.random_parents(len(lens), T, torch.Generator().manual_seed(200 + i))
    words = [R.ancestors(par[b], T)[0] for b in range(len(lens))] if i % 2 else None
    r = VerifyRun(lens, drafts, T, Hq, Hkv, d, page, dtype, words=words, seed=210 + i)
    r.call()
    r.check()


@pytest.mark.parametrize("T,Hq,d", [(16, 8, 128), (40, 8, 64), (24, 16, 128), (9, 4, 256)])
def test_verify_ragged_batch(T, Hq, d):
    """Shares that begin and end anywhere in units of very different lengths: units of one CTA, of
    two and of many, several units of one CTA; the same bits from one call to the next."""
    lens = [3000, 7, 64, 0, 1900, 333, 128, 5000, 12, 700]
    r = VerifyRun(lens, [max(0, T - (3 * b) % (T + 1)) for b in range(len(lens))], T, Hq, 1, d, 32, BF, seed=230)
    r.call()
    r.check()
    first = r.out.clone(), r.lse.clone()
    for _ in range(3):
        r.call()
        assert torch.equal(first[0], r.out) and torch.equal(first[1], r.lse)


def test_verify_more_sequences_than_one_launch_takes():
    B = 1100
    lens = [(29 * b) % 150 for b in range(B)]
    r = VerifyRun(lens, [b % 3 for b in range(B)], 2, 2, 1, 64, 16, BF, seed=240)
    r.call()
    r.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_verify_rows_that_see_nothing(dtype):
    """Words without bits over an empty context, and words whose bits lie past the draft."""
    T = 6
    words = [[0] * T, [0, 1, 0, 5, 0, 1 << 40], [0] * T, [63 << 6] * T]
    r = VerifyRun([0, 0, 20, 0], [6, 6, 6, 5], T, 8, 2, 128, 16, dtype, words=words, seed=3)
    r.call()
    r.check()
    assert (R.f64(r.out)[0] == 0).all() and np.isneginf(R.f64(r.lse)[0]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_verify_unseen_rows_hold_anything(dtype, d):
    """A draft token's NaN or infinite key and value reach only the rows that see it."""
    T, lens = 8, [70, 9]
    words = [[1, 3, 5, 9, 1 | 16, 33, 65, 129] for _ in lens]     # token 0's children, but none of each other
    r = VerifyRun(lens, [T, T], T, 4, 2, d, 16, dtype, words=words, seed=5)
    c = r.case
    for b in range(2):
        p, row = c.cell(b, lens[b] + 3)
        r.cache.k[:, p, :, row] = float("nan")
        p, row = c.cell(b, lens[b] + 5)
        r.cache.v[:, p, 0, row, 1] = float("inf")
        r.cache.v[:, p, 0, row, d - 1] = float("nan")
    r.call()
    out = R.f64(r.out)
    G = r.Hq // c.Hkv
    for b in range(2):
        assert np.isnan(out[b, 3]).all()
        assert np.isposinf(out[b, 5, :G, 1]).all() and np.isnan(out[b, 5, :G, d - 1]).all()
        assert np.isfinite(out[b, 5, :G, 2:d - 1]).all() and np.isfinite(out[b, 5, G:]).all()
        rest = [0, 1, 2, 4, 6, 7]
        k, v = (c.rows(x, b, lens[b] + T) for x in (c.k, c.v))
        o, e, A, S = R.attention(R.f64(r.q[b]), k, v, words[b], lens[b], r.scale)
        to, _ = R.verify_bounds(A, S, e, lens[b] + T, d, dtype == BF)
        assert (np.abs(out[b, rest] - o[rest]) <= to[rest]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_verify_large_scores(dtype):
    """Scores of several hundred (one key far above the rest, late in the row): the running
    maximum is replaced after most keys have been summed."""
    r = VerifyRun([900, 333], [5, 5], 5, 4, 2, 128, 16, dtype, seed=8)
    c = r.case
    for b, at in ((0, 850), (0, 300), (1, 20), (1, 331)):
        p, row = c.cell(b, at)
        c.k[0, p, :, row] = (torch.randn(c.Hkv, c.d, generator=c.g) * 20 * (1 + at / 900)).to(dtype)
    r.cache.k.copy_(c.k)
    r.call()
    r.check()


@pytest.mark.parametrize("dtype,lens,T,Hq,Hkv", [(BF, [40007], 16, 16, 2), (BF, [12345, 1, 64, 3000], 5, 8, 1),
                                                 (F32, [20011], 3, 4, 2)])
def test_verify_long_contexts_are_split(dtype, lens, T, Hq, Hkv):
    r = VerifyRun(lens, [T] * len(lens), T, Hq, Hkv, 128, 64, dtype, seed=21)
    r.call()
    r.check()
    first = r.out.clone(), r.lse.clone()
    r.call()
    assert torch.equal(first[0], r.out) and torch.equal(first[1], r.lse)     # the same bits again


@pytest.mark.parametrize("lens,drafts,T,Hq,Hkv,d", [
    ([30000, 17, 9000, 20011], [5, 5, 0, 3], 5, 8, 4, 64),                # one row tile
    ([14000, 17, 0, 20011], [40, 40, 0, 17], 40, 32, 4, 128),             # a pair and one more; a pair; none
    ([30000, 63, 64, 52000], [7, 7, 1, 2], 7, 16, 2, 256)])               # one group
def test_verify_many_tiles_per_cta(lens, drafts, T, Hq, Hkv, d):
    """Enough keys that a unit's beginning and end count as work."""
    r = VerifyRun(lens, drafts, T, Hq, Hkv, d, 64, BF, seed=26)
    r.call()
    r.check()
    first = r.out.clone(), r.lse.clone()
    r.call()
    assert torch.equal(first[0], r.out) and torch.equal(first[1], r.lse)     # the same bits again


def test_verify_many_sequences():
    """More (sequence, head) units than resident CTAs, lengths from none to several tiles."""
    B = 300
    lens = [(37 * b) % 211 for b in range(B)]
    r = VerifyRun(lens, [1 + b % 2 for b in range(B)], 2, 4, 2, 64, 16, BF, seed=22)
    r.call()
    r.check()


def test_verify_layers_and_streams():
    """The layer's own keys and values; a call on another stream; no lse."""
    r = VerifyRun([100, 40], [4, 4], 4, 8, 2, 128, 16, BF, seed=23, layers=3, layer=2)
    r.call(stream=torch.cuda.Stream())
    r.check()
    first = r.out.clone()
    r.lse.fill_(7.0)
    r.call(lse=False)
    assert torch.equal(first, r.out) and bool((r.lse == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_verify_past_32_bit_offsets(dtype):
    """Pages whose rows lie past 2^32 elements of the cache."""
    lib = _lib()
    Hkv, page, d, T = 8, 128, 256, 3
    n_page = (1 << 32) // (Hkv * page * d) + 40 if dtype == BF else (1 << 31) // (Hkv * page * d) + 40
    small = R.CacheCase([300], T, Hkv, d, page, dtype, seed=31)
    k = torch.empty(1, n_page, Hkv, page, d, dtype=dtype, device="cuda")
    v = torch.empty_like(k)
    shift = n_page - small.n_page
    k[0, shift:], v[0, shift:] = small.k[0].cuda(), small.v[0].cuda()
    own = int(small.n_owned[small.state_idx[0].long()])
    table = small.block_table.clone()
    table[small.state_idx[0].long(), :own] += shift
    ref = torch.zeros(n_page, dtype=torch.int32)
    dims = small.dims(lib)
    dims.n_page = n_page
    cache = lib.PagedCache(dims, dict(small.init(), k=k, v=v, block_table=table, ref=ref, free_list=ref.clone()))
    layer = lib.AttnLayer(lib.AttnDims(B=1, T=T, Hq=16, scale=d ** -0.5), cache, 0, state_idx=small.state_idx.cuda())
    q = torch.randn(1, T, 16, d, generator=small.g).to(dtype)
    out, lse = torch.zeros(1, T, 16, d, dtype=dtype, device="cuda"), torch.zeros(1, T, 16, device="cuda")
    layer.verify(q.cuda(), out, lse=lse)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0
    kk, vv = (small.rows(x, 0, 303) for x in (small.k, small.v))
    o, e, A, S = R.attention(R.f64(q[0]), kk, vv, [1, 3, 7], 300, d ** -0.5)
    to, te = R.verify_bounds(A, S, e, 303, d, dtype == BF)
    assert (np.abs(R.f64(out)[0] - o) <= to).all() and (np.abs(R.f64(lse)[0] - e) <= te).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_verify_faults_skip_the_sequence(dtype):
    """A slot, a length or a draft length out of range, no room, a page out of range: the
    status word tells, the other sequences are right, skipped outputs stay unwritten."""
    lib = _lib()
    r = VerifyRun([100, 50, 60, 70, 80, 90], [4, 4, 4, 4, 4, 4], 4, 4, 2, 64, 16, dtype, seed=24)
    c, sl = r.case, r.case.state_idx.long()
    bad = c.state_idx.clone()
    bad[0] = c.n_slot
    r.attn.state_idx.copy_(bad)
    r.cache.seq_len[sl[1]] = -3
    r.cache.seq_len[sl[2]] = c.max_pages * c.page - 1
    r.drafts = [4, 4, 4, 4, 4, 4]
    r.cache.block_table[sl[3], 1] = -1
    out0 = r.out.clone()
    dl = torch.tensor([4, 4, 4, 4, 9, 4], dtype=torch.int32).cuda()
    r.attn.verify(r.q.cuda(), r.out, lse=r.lse, draft_len=dl)
    torch.cuda.synchronize()
    for b in (0, 1, 2, 4):
        assert torch.equal(r.out[b], out0[b]) and bool((r.lse[b] == 7.0).all()), b
    r.check(skip=(0, 1, 2, 3, 4), status=lib.STATUS_BAD_SLOT | lib.STATUS_BAD_LEN | lib.STATUS_NO_ROOM | lib.STATUS_BAD_PAGE)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_verify_wait_expiry(d):
    """The tensor-core kernel's wait-expiry exit (taken at the first wait, with nothing in
    flight): the status word tells, the device stays usable, the next call is right."""
    lib = _lib()
    r = VerifyRun([100, 700], [4, 4], 4, 8, 2, d, 16, BF, seed=25)
    good, dims = r.attn, r.attn.d
    dims.flags = lib.FLAG_TEST_EXPIRE
    r.attn = lib.AttnLayer(dims, r.cache, 0, state_idx=r.case.state_idx.cuda())
    r.call()
    assert int(r.cache.status.item()) == lib.STATUS_TIMEOUT
    r.attn = good
    r.cache.status.zero_()
    r.call()
    r.check()


# ------------------------------------------------------------------------ stage
STAGE = [
    # lens, drafts, T, Hq, Hkv, d, page, rot, pairs, packed
    ([0], [1], 1, 4, 2, 64, 16, 64, False, False),
    ([0, 5, 15, 16], [3, 0, 2, 3], 3, 6, 3, 64, 16, 32, True, True),
    ([31, 100], [16, 16], 16, 16, 2, 128, 32, 128, False, True),
    ([7, 90, 64], [5, 9, 1], 9, 5, 1, 128, 64, 96, False, False),
    ([11, 300], [33, 40], 40, 12, 4, 256, 128, 64, False, True),
    ([3], [200], 200, 7, 7, 256, 16, 256, True, False),
    ([40], [2], 2, 33, 3, 64, 16, 0, False, False),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("with_pos", [False, True])
@pytest.mark.parametrize("i", range(len(STAGE)))
def test_stage(i, with_pos, dtype):
    lib = _lib()
    lens, drafts, T, Hq, Hkv, d, page, rot, pairs, packed = STAGE[i]
    c = R.CacheCase(lens, T, Hkv, d, page, dtype, layers=2, seed=50 + i)
    B, g, eps, max_pos = len(lens), c.g, 1e-6, max(lens) + T + 5
    width = [Hq * d, Hkv * d, Hkv * d]
    # rows of very different size: the norm removes it
    rows = torch.randn(B, T, sum(width), generator=g) * torch.exp2(6 * torch.rand(B, T, 1, generator=g) - 3)
    rows[0, 0, :d] = 0                                        # a row of zeros stays zero
    dev = rows.to(dtype).cuda()
    q, k, v = (x.unflatten(-1, (-1, d)) for x in dev.split(width, -1))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw, kw = 1 + 0.3 * torch.randn(d, generator=g), 1 + 0.3 * torch.randn(d, generator=g)
    a = torch.rand(max_pos, rot // 2, generator=g, dtype=torch.float64) * 6.28
    tab = torch.cat([a.cos(), a.sin()], 1).float()
    pos = torch.randint(0, max_pos, (B, T), generator=g, dtype=torch.int32)
    cache = lib.PagedCache(c.dims(lib), c.init())
    rope = lib.RopeDims(rot=rot, style=lib.ROPE_PAIRS if pairs else lib.ROPE_HALF, max_pos=max_pos, eps=eps)
    layer = lib.AttnLayer(lib.AttnDims(B=B, T=T, Hq=Hq, scale=1.0), cache, 1, rope, qw.cuda(), kw.cuda(),
                          tab.cuda() if rot else None, state_idx=c.state_idx.cuda())
    q_out, intact = _guarded((B, T, Hq, d), dtype, 7.0)
    layer.stage(q, k, v, q_out, pos=pos.cuda() if with_pos else None,
                draft_len=torch.tensor(drafts, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0 and intact()
    ks, vs = c.k.clone(), c.v.clone()                        # what the cache must hold
    want, band = np.zeros((B, T, Hq, d)), np.zeros((B, T, Hq, d))
    x = R.f64(rows.to(dtype))
    tol = (d / 2 + 16) * 2.0 ** -24
    got_k = cache.k.cpu()
    for b in range(B):
        for t in range(drafts[b]):
            p = int(pos[b, t]) if with_pos else lens[b] + t
            cos, sin = R.f64(tab[p, :rot // 2]), R.f64(tab[p, rot // 2:])
            xq, xk = x[b, t, :width[0]].reshape(Hq, d), x[b, t, width[0]:width[0] + width[1]].reshape(Hkv, d)
            y, size = R.norm_rotate(xq, R.f64(qw), eps, cos, sin, rot, pairs)
            want[b, t], band[b, t] = y, tol * size + 1e-30
            y, size = R.norm_rotate(xk, R.f64(kw), eps, cos, sin, rot, pairs)
            pg, r = c.cell(b, lens[b] + t)
            if dtype == BF:
                assert_bf16_rounding(f"k {b} {t}", got_k[1, pg, :, r], y, tol * size + 1e-30)
            else:
                assert (np.abs(R.f64(got_k[1, pg, :, r]) - y) <= tol * size + 1e-30).all(), (b, t)
            ks[1, pg, :, r] = got_k[1, pg, :, r]             # compared just now
            vs[1, pg, :, r] = rows.to(dtype)[b, t, width[0] + width[1]:].reshape(Hkv, d)
    if dtype == BF:
        assert_bf16_rounding("q_out", q_out, want, band)
    else:
        assert (np.abs(R.f64(q_out) - want) <= band).all()
    for got, ref in ((got_k, ks), (cache.v.cpu(), vs)):       # every other row untouched
        np.testing.assert_array_equal(R.f64(got), R.f64(ref))


def test_stage_faults():
    lib = _lib()
    c = R.CacheCase([20, 30, 40, 50], 4, 2, 64, 16, BF, seed=70)
    sl = c.state_idx.long()
    cache = lib.PagedCache(c.dims(lib), c.init())
    rope = lib.RopeDims(rot=16, style=lib.ROPE_HALF, max_pos=64, eps=1e-6)
    w = torch.ones(64, device="cuda")
    layer = lib.AttnLayer(lib.AttnDims(B=4, T=4, Hq=4, scale=1.0), cache, 0, rope, w, w,
                          torch.ones(64, 16, device="cuda"), state_idx=c.state_idx.cuda())
    x = torch.randn(4, 4, 8, 64, generator=c.g).to(BF).cuda()
    q_out = torch.full((4, 4, 4, 64), 7.0, dtype=BF, device="cuda")
    pos = torch.zeros(4, 4, dtype=torch.int32)
    pos[1, 2] = 64                                           # no such rotation
    cache.seq_len[sl[0]] = c.max_pages * c.page + 1          # a length out of range
    cache.block_table[sl[2], 40 // 16] = c.n_page            # a page out of range
    layer.stage(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], q_out, pos=pos.cuda())
    torch.cuda.synchronize()
    assert int(cache.status.item()) == lib.STATUS_BAD_LEN | lib.STATUS_BAD_POS | lib.STATUS_BAD_PAGE
    assert bool((q_out[0] == 7.0).all()) and bool((q_out[1, 2] == 0).all()) and not bool((q_out[1, 1] == 0).any())
    assert not bool((q_out[2] == 7.0).any())                 # queries do not need the page
    k = cache.k.cpu()
    p, r = c.cell(1, 32)
    assert torch.equal(k[0, p, :, r], c.k[0, p, :, r])        # the skipped token's row
    p, r = c.cell(1, 33)
    assert not torch.equal(k[0, p, :, r], c.k[0, p, :, r])


@pytest.mark.parametrize("d,dtype,pairs", [(64, BF, True), (128, F32, False), (256, BF, False)])
def test_stage_many_tokens(d, dtype, pairs):
    """Ragged prompts of some thousand tokens: a sample against the formula, and every row the same
    bits as when the tokens come some hundred at a time (a row's arithmetic does not depend on how
    many tokens a call has)."""
    lib = _lib()
    lens, drafts, T, Hq, Hkv, rot, eps = [3, 100, 0], [1700, 0, 1033], 1700, 6, 2, 48, 1e-6
    c = R.CacheCase(lens, T, Hkv, d, 32, dtype, seed=71)
    B, g, width, max_pos = len(lens), c.g, (Hq + 2 * Hkv) * d, max(lens) + T
    rows = torch.randn(B, T, width, generator=g).to(dtype)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in rows.cuda().split([Hq * d, Hkv * d, Hkv * d], -1))
    qw, kw = 1 + 0.3 * torch.randn(d, generator=g), 1 + 0.3 * torch.randn(d, generator=g)
    a = torch.rand(max_pos, rot // 2, generator=g, dtype=torch.float64) * 6.28
    tab = torch.cat([a.cos(), a.sin()], 1).float()
    rope = lib.RopeDims(rot=rot, style=lib.ROPE_PAIRS if pairs else lib.ROPE_HALF, max_pos=max_pos, eps=eps)

    def layer(cache, B, T, idx):
        return lib.AttnLayer(lib.AttnDims(B=B, T=T, Hq=Hq, scale=1.0), cache, 0, rope, qw.cuda(), kw.cuda(), tab.cuda(),
                             state_idx=idx.cuda())
    whole, parts = lib.PagedCache(c.dims(lib), c.init()), lib.PagedCache(c.dims(lib), c.init())
    q_out, intact = _guarded((B, T, Hq, d), dtype, 7.0)
    layer(whole, B, T, c.state_idx).stage(q, k, v, q_out, draft_len=torch.tensor(drafts, dtype=torch.int32).cuda())
    other = torch.zeros(B, T, Hq, d, dtype=dtype, device="cuda")
    for b in range(B):
        idx = c.state_idx[b:b + 1]
        for t in range(0, drafts[b], 300):
            n = min(300, drafts[b] - t)
            parts.seq_len[int(idx)] = lens[b] + t
            layer(parts, 1, n, idx).stage(q[b:b + 1, t:t + n], k[b:b + 1, t:t + n], v[b:b + 1, t:t + n], other[b:b + 1, t:t + n])
    torch.cuda.synchronize()
    assert int(whole.status.item()) == int(parts.status.item()) == 0 and intact()
    assert torch.equal(q_out, other)
    np.testing.assert_array_equal(R.f64(whole.k.cpu()), R.f64(parts.k.cpu()))
    np.testing.assert_array_equal(R.f64(whole.v.cpu()), R.f64(parts.v.cpu()))
    x, tol, got = R.f64(rows), (d / 2 + 16) * 2.0 ** -24, q_out.cpu()
    for b, t in [(0, 0), (0, 28), (0, 29), (0, 1699), (2, 0), (2, 517), (2, 1032)]:
        p = lens[b] + t
        cos, sin = R.f64(tab[p, :rot // 2]), R.f64(tab[p, rot // 2:])
        y, size = R.norm_rotate(x[b, t, :Hq * d].reshape(Hq, d), R.f64(qw), eps, cos, sin, rot, pairs)
        if dtype == BF:
            assert_bf16_rounding(f"q {b} {t}", got[b, t], y, tol * size + 1e-30)
        else:
            assert (np.abs(R.f64(got[b, t]) - y) <= tol * size + 1e-30).all(), (b, t)


def test_stage_single_token_of_any_stride():
    """One token's stride says nothing: a row of a width that is no multiple of 16 bytes is taken."""
    lib = _lib()
    c = R.CacheCase([20], 1, 2, 64, 16, BF, seed=72)
    rope = lib.RopeDims(rot=16, style=lib.ROPE_HALF, max_pos=64, eps=1e-6)
    w, tab = torch.ones(64, device="cuda"), torch.rand(64, 16, generator=c.g).cuda()
    row = torch.randn(1, 1, 8 * 64 + 4, generator=c.g).to(BF).cuda()
    q, k, v = (x.unflatten(-1, (-1, 64)) for x in row[..., :8 * 64].split([4 * 64, 2 * 64, 2 * 64], -1))
    got = []
    for dense in (False, True):
        cache = lib.PagedCache(c.dims(lib), c.init())
        layer = lib.AttnLayer(lib.AttnDims(B=1, T=1, Hq=4, scale=1.0), cache, 0, rope, w, w, tab, state_idx=c.state_idx.cuda())
        q_out = torch.zeros(1, 1, 4, 64, dtype=BF, device="cuda")
        layer.stage(*((x.contiguous() for x in (q, k, v)) if dense else (q, k, v)), q_out)
        torch.cuda.synchronize()
        assert int(cache.status.item()) == 0
        got.append((q_out, cache.k, cache.v))
    for x, y in zip(*got):
        np.testing.assert_array_equal(R.f64(x.cpu()), R.f64(y.cpu()))


# ------------------------------------------------------------------------ trees
@pytest.mark.parametrize("B,T,drafts", [(1, 1, None), (5, 7, [7, 0, 1, 4, 7]), (9, 64, None), (3, 33, [33, 32, 2])])
def test_tree_build(B, T, drafts):
    lib = _lib()
    c = R.CacheCase([3 * b for b in range(B)], T, 1, 64, 16, BF, seed=60)
    cache = lib.PagedCache(c.dims(lib), c.init())
    layer = lib.AttnLayer(lib.AttnDims(B=B, T=T, Hq=1, scale=1.0), cache, 0, state_idx=c.state_idx.cuda())
    par = R.random_parents(B, T, c.g, width=6)
    if T == 64:
        par[0] = torch.arange(T) - 1                          # a chain of 64
        par[1] = -1                                           # 64 roots
    tree = torch.zeros(B, T, dtype=torch.int64, device="cuda")
    pos = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    n = drafts or [T] * B
    layer.build_tree(par.cuda(), tree, pos, None if drafts is None else torch.tensor(drafts, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0
    for b in range(B):
        words, depth = R.ancestors(par[b], n[b])
        words, depth = words + [0] * (T - n[b]), depth + [0] * (T - n[b])
        assert tree[b].tolist() == R.as_int64(words)
        assert pos[b].tolist() == [3 * b + x for x in depth]
    par[0, 0] = 0                                             # its own parent
    tree.fill_(-5)
    layer.build_tree(par.cuda(), tree, pos)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == lib.STATUS_BAD_TREE and bool((tree[0] == -5).all())


# ----------------------------------------------------------------------- accept
@pytest.mark.parametrize("dtype,Hkv,d,page,layers,T,B,in_place", [
    (BF, 2, 128, 16, 3, 16, 6, False), (F32, 1, 64, 32, 1, 64, 5, True), (BF, 3, 256, 128, 2, 33, 3, True),
    (BF, 8, 64, 16, 5, 5, 1, False)])
def test_accept_moves_the_path(dtype, Hkv, d, page, layers, T, B, in_place):
    lib = _lib()
    lens = [(13 * b * b) % 97 for b in range(B)]
    c = R.CacheCase(lens, T, Hkv, d, page, dtype, layers=layers, seed=80)
    cache = lib.PagedCache(c.dims(lib), c.init())
    counts = [min(T, x) for x in ([0, T, 1, 9, T // 2, 12] * 3)[:B]]
    path = torch.full((B, T), -1, dtype=torch.int32)
    for b, p in enumerate(counts):
        path[b, :p] = torch.randperm(T, generator=c.g)[:p].sort()[0].to(torch.int32)
    new = None if in_place else torch.full((c.n_slot,), -9, dtype=torch.int32, device="cuda")
    cache.accept(torch.tensor(counts, dtype=torch.int32).cuda(), path=path.cuda(), state_idx=c.state_idx.cuda(), new_len=new)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0
    k, v, ln = c.k.clone(), c.v.clone(), c.seq_len.clone()
    for b, p in enumerate(counts):
        at = [c.cell(b, lens[b] + int(j)) for j in path[b, :p]]
        for x, y in ((k, c.k), (v, c.v)):
            for j, (pg, r) in enumerate(at):
                z = c.cell(b, lens[b] + j)
                x[:, z[0], :, z[1]] = y[:, pg, :, r]
        ln[c.state_idx[b].long()] += p
    np.testing.assert_array_equal(R.f64(cache.k), R.f64(k))
    np.testing.assert_array_equal(R.f64(cache.v), R.f64(v))
    if in_place:
        assert torch.equal(cache.seq_len.cpu(), ln)
    else:
        got = new.cpu()
        batch = c.state_idx.long()
        assert torch.equal(got[batch], ln[batch]) and int((got == -9).sum()) == c.n_slot - B
        assert torch.equal(cache.seq_len.cpu(), c.seq_len)


def test_accept_chain_and_faults():
    lib = _lib()
    c = R.CacheCase([20, 30, 40, 50, 60, 70], 8, 2, 64, 16, BF, seed=81)
    cache = lib.PagedCache(c.dims(lib), c.init())
    idx, sl = c.state_idx.cuda(), c.state_idx.long()
    acc = torch.tensor([0, 8, 3, 1, 5, 2], dtype=torch.int32)
    cache.accept(acc.cuda(), state_idx=idx)                   # a chain: lengths only
    torch.cuda.synchronize()
    want = c.seq_len.clone()
    want[sl] += acc
    assert int(cache.status.item()) == 0 and torch.equal(cache.seq_len.cpu(), want)
    np.testing.assert_array_equal(R.f64(cache.k), R.f64(c.k))
    cache.seq_len.copy_(c.seq_len)
    path = torch.arange(8, dtype=torch.int32).repeat(6, 1)
    path[0, 1] = 0                                            # not increasing
    path[1, 2] = 8                                            # not a token
    acc = torch.tensor([2, 3, 9, 3, 2, 2], dtype=torch.int32)  # the third: more than T
    bad = c.state_idx.clone()
    bad[3] = -1
    cache.block_table[sl[4], (60 + 1) // 16] = -7
    cache.accept(acc.cuda(), path=path.cuda(), state_idx=bad.cuda())
    torch.cuda.synchronize()
    assert int(cache.status.item()) == (lib.STATUS_BAD_TREE | lib.STATUS_BAD_ACCEPT | lib.STATUS_BAD_SLOT | lib.STATUS_BAD_PAGE)
    want = c.seq_len.clone()
    want[sl[5]] += 2
    assert torch.equal(cache.seq_len.cpu(), want)
    np.testing.assert_array_equal(R.f64(cache.k), R.f64(c.k))


# ------------------------------------------------------------------------ pages
def _same_pool(cache, p):
    for name, ref in (("block_table", p.table), ("seq_len", p.len), ("n_owned", p.owned), ("ref", p.ref),
                      ("free_list", p.list)):
        np.testing.assert_array_equal(getattr(cache, name).cpu().numpy(), ref, err_msg=name)
    assert int(cache.free_count.item()) == p.count
    np.testing.assert_array_equal(R.f64(cache.k), R.f64(p.k))
    np.testing.assert_array_equal(R.f64(cache.v), R.f64(p.v))
    assert int(cache.status.item()) == p.status


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("seed", range(6))
def test_pool_random_steps(seed):
    """Random reserves, forks and releases (some with slots out of range or in use, some past
    the end of the free list) against the row-by-row model: every array after every call."""
    lib = _lib()
    rng = np.random.RandomState(seed)
    page = [16, 32, 64, 128, 16, 16][seed]
    c = R.CacheCase([rng.randint(0, 5 * page) for _ in range(5)], 0, 1, 64, page, BF, layers=2, seed=seed,
                    spare=[40, 12, 25, 9, 4, 60][seed], extra_slots=25)
    cache, p = lib.PagedCache(c.dims(lib), c.init()), R.Pool(c)
    for step in range(25):
        cache.status.zero_()
        p.status = 0
        kind = rng.randint(0, 4)
        live = [s for s in range(c.n_slot) if p.owned[s]]
        empty = [s for s in range(c.n_slot) if not p.owned[s]]
        if kind == 0 and live:
            rows = list(rng.permutation(live)[:rng.randint(1, len(live) + 1)])
            if rng.rand() < 0.3:
                rows.insert(rng.randint(len(rows) + 1), -1)
            extra = int(rng.randint(0, 2 * page))
            cache.reserve(_i32(rows), extra)
            p.reserve(rows, extra)
        elif kind in (1, 2) and live and empty:
            n = min(len(empty), rng.randint(1, 8))
            dst = list(rng.permutation(empty)[:n])
            if rng.rand() < 0.3 and len(live) > 1:
                dst[0] = live[0]                              # in use: refused
            src = [int(rng.choice([s for s in live if s not in dst] or [-1])) for _ in dst]
            copies = _i32([[5, 5]] * n)
            cache.fork(_i32(src), _i32(dst), copies)
            want = p.fork(src, dst)
            assert copies.cpu().tolist() == [list(x) for x in want]
        elif live:
            rows = list(rng.permutation(live)[:rng.randint(1, len(live) + 1)])
            if rng.rand() < 0.3:
                rows.append(c.n_slot + 4)
            cache.release(_i32(rows))
            p.release(rows)
        torch.cuda.synchronize()
        _same_pool(cache, p)


def test_pool_many_rows():
    """Thousands of rows and of shared pages: more than one round of the CTA's threads, and
    pages shared by hundreds of sequences released in one call."""
    lib = _lib()
    c = R.CacheCase([1000, 37], 0, 1, 64, 16, BF, seed=90, spare=1500, extra_slots=1400)
    cache, p = lib.PagedCache(c.dims(lib), c.init()), R.Pool(c)
    a, b = (int(x) for x in c.state_idx)
    empty = [s for s in range(c.n_slot) if s not in (a, b)]
    src = [a if i % 3 else b for i in range(1300)]
    dst = empty[:1300]
    copies = torch.zeros(1300, 2, dtype=torch.int32, device="cuda")
    cache.fork(_i32(src), _i32(dst), copies)
    p.fork(src, dst)
    cache.reserve(_i32(dst), 40)                              # the free list runs out on the way
    p.reserve(dst, 40)
    torch.cuda.synchronize()
    _same_pool(cache, p)
    assert p.status == p.NO_PAGES | p.NO_ROOM                 # some rows need more entries than a table row has
    cache.release(_i32([a] + dst[::-1] + [b]))
    p.release([a] + dst[::-1] + [b])
    torch.cuda.synchronize()
    _same_pool(cache, p)
    assert p.count == c.n_page


def test_pool_faults():
    """A page released more often than it was shared and corrupt entries are reported and
    never pushed; nothing leaves the arrays' bounds."""
    lib = _lib()
    c = R.CacheCase([40, 40], 0, 1, 64, 16, BF, seed=91)
    cache = lib.PagedCache(c.dims(lib), c.init())
    a, b = (int(x) for x in c.state_idx)
    cache.block_table[b, 0] = cache.block_table[a, 0]         # held twice, counted once
    cache.block_table[b, 1] = c.n_page + 5
    before = int(cache.free_count.item())
    cache.release(_i32([a, b]))
    torch.cuda.synchronize()
    assert int(cache.status.item()) == lib.STATUS_BAD_PAGE
    assert int(cache.free_count.item()) == before + 3         # a's other two and b's last
    cache.status.zero_()
    cache.fork(_i32([a]), _i32([c.n_slot]), _i32([[0, 0]]))
    torch.cuda.synchronize()
    assert int(cache.status.item()) == lib.STATUS_BAD_SLOT
    lib._check("gdn_pages_copy", cache._lib.gdn_pages_copy(cache._c, 1, _i32([[0, c.n_page]]).data_ptr(), cache._status, None))
    torch.cuda.synchronize()
    assert int(cache.status.item()) == lib.STATUS_BAD_SLOT | lib.STATUS_BAD_PAGE
