"""A slot that got no pages: what its block-table row still holds from an earlier sequence belongs to
others by now, and no attention call may read or write it.

Expected values: rows of the cache and lengths exactly; outputs of the sequence beside it as in
attn_ref.verify_bounds."""
import numpy as np
import pytest
import torch

import attn_ref as R
from test_gpu_attn import BF, F32, _i32

pytestmark = pytest.mark.gpu
T, HQ, HKV, D, PAGE = 8, 4, 2, 64, 16


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def _lib():
    import speculative_decode_recurrent_gb300 as lib
    return lib


class Loop:
    """Two slots over a pool of six pages; slot 0's first sequence is gone and slot 1 has all pages."""

    def __init__(self, dtype, layers=2, seed=3):
        lib = self.lib = _lib()
        self.g, self.dtype = torch.Generator().manual_seed(seed), dtype
        self.cache = c = lib.PagedCache(lib.PageDims(n_slot=3, max_pages=6, n_page=6, page=PAGE, n_layer=layers, Hkv=HKV,
                                                     d=D, dtype=lib.DTYPE_BF16 if dtype == BF else lib.DTYPE_F32))
        w, tab = torch.ones(D, device="cuda"), torch.zeros(128, 16, device="cuda")
        tab[:, :8] = 1.0                                     # (angles of zero)
        rope = lib.RopeDims(rot=16, style=lib.ROPE_HALF, max_pos=128, eps=1e-6)
        self.layer = lib.AttnLayer(lib.AttnDims(B=2, T=T, Hq=HQ, scale=D ** -0.5), c, 1, rope, w, w, tab,
                                   state_idx=_i32([0, 1]))
        c.k.copy_(torch.randn(c.k.shape, generator=self.g))
        c.v.copy_(torch.randn(c.v.shape, generator=self.g))
        c.reserve(_i32([0]), 40)                             # three pages
        c.seq_len[0] = 40
        c.release(_i32([0]))
        c.reserve(_i32([1]), 88)                             # all six, slot 0's old ones among them
        c.seq_len[1] = 80
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0 and int(c.free_count.item()) == 0 and c.n_owned.tolist() == [0, 6, 0]

    def block(self):
        return [torch.randn(2, T, h, D, generator=self.g).to(self.dtype).cuda() for h in (HQ, HKV, HKV)]

    def others(self, length):
        """Rows of slot 1's first `length` tokens."""
        at = torch.arange(length)
        ids = self.cache.block_table[1].cpu()[at // PAGE].long()
        return [x.cpu()[:, ids, :, at % PAGE].clone() for x in (self.cache.k, self.cache.v)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("how", ["reserve", "fork"])
def test_a_slot_without_pages_touches_nobodys_rows(how, dtype):
    x = Loop(dtype)
    c, lib = x.cache, x.lib
    if how == "reserve":
        c.reserve(_i32([0]), T)                              # no page left: skipped, on the device
    else:
        c.seq_len[1] = 75                                    # a part of a page to copy, and no page for it
        c.fork(_i32([1]), _i32([0]), torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
        c.seq_len[1] = 80
    torch.cuda.synchronize()
    assert int(c.status.item()) == lib.STATUS_NO_PAGES and c.n_owned.tolist() == [0, 6, 0]
    c.status.zero_()
    before, q = x.others(80), torch.empty(2, T, HQ, D, dtype=dtype, device="cuda")
    x.layer.stage(*x.block(), q)
    torch.cuda.synchronize()
    assert int(c.status.item()) == lib.STATUS_BAD_PAGE
    for was, now in zip(before, x.others(80)):
        assert torch.equal(was, now)
    # the other sequence's draft is staged, its outputs are right
    c.status.zero_()
    out, lse = torch.empty_like(q), torch.empty(2, T, HQ, device="cuda")
    x.layer.verify(q, out, lse=lse)
    torch.cuda.synchronize()
    assert int(c.status.item()) == lib.STATUS_BAD_PAGE
    k, v = (R.f64(y[:, 1]) for y in x.others(88))
    o, e, A, S = R.attention(R.f64(q[1]), k, v, [(2 << t) - 1 for t in range(T)], 80, D ** -0.5)
    to, te = R.verify_bounds(A, S, e, 88, D, dtype == BF)
    assert (np.abs(R.f64(out)[1] - o) <= to).all() and (np.abs(R.f64(lse)[1] - e) <= te).all()
    # along a path and as a chain: nothing of the slot without pages moves, neither rows nor length
    for path in (_i32([[1, 3, 0, 0, 0, 0, 0, 0], [0, 1, 0, 0, 0, 0, 0, 0]]), None):
        c.status.zero_()
        before, ln = x.others(88), int(c.seq_len[1])
        c.accept(_i32([2, 2]), path=path, state_idx=_i32([0, 1]))
        torch.cuda.synchronize()
        assert int(c.status.item()) == lib.STATUS_BAD_PAGE and c.seq_len.tolist() == [0, ln + 2, 0]
        for was, now in zip(before, x.others(88)):
            assert torch.equal(was, now)
    # no token accepted needs no page
    c.status.zero_()
    c.accept(_i32([0, 0]), state_idx=_i32([0, 1]))
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0 and c.seq_len.tolist() == [0, 84, 0]


def test_entries_past_the_owned_ones_are_not_used():
    """A sequence that keeps its pages but gets no more: the tokens that lie in its own pages are staged
    and accepted, those past them are not, whatever its block-table row holds there."""
    x = Loop(BF)
    c, lib = x.cache, x.lib
    c.release(_i32([1]))
    c.reserve(_i32([0]), 20)                                 # two pages
    c.reserve(_i32([1]), 50)                                 # the other four
    c.seq_len[0], c.seq_len[1] = 28, 48
    own0, own1 = c.block_table[0, :2].tolist(), c.block_table[1, :4].tolist()
    assert sorted(own0 + own1) == list(range(6)) and int(c.block_table[0, 2]) in own1      # a stale entry
    keys = c.k.clone()
    x.layer.stage(*x.block(), torch.empty(2, T, HQ, D, dtype=BF, device="cuda"))
    torch.cuda.synchronize()
    assert int(c.status.item()) == lib.STATUS_BAD_PAGE
    changed = (keys != c.k).any(-1).any(2)[1]                # [page, row] of layer 1
    want = torch.zeros_like(changed)
    want[own0[1], 12:] = True                                # tokens 28 to 31 of slot 0
    want[own1[3], :8] = True                                 # tokens 48 to 55 of slot 1
    assert torch.equal(changed, want)
    for p, status, ln in ((5, lib.STATUS_BAD_PAGE, 28), (4, 0, 32)):
        c.status.zero_()
        c.accept(_i32([p]), state_idx=_i32([0]))
        torch.cuda.synchronize()
        assert int(c.status.item()) == status and int(c.seq_len[0]) == ln


def test_without_the_pool_the_block_table_is_taken_as_it_is():
    """n_owned NULL: the caller keeps the pages; any entry in range is used."""
    x = Loop(BF)
    c = x.cache
    c.d.n_owned = None
    c.block_table[0, 0], c.block_table[1, 5] = 3, 3          # a page for slot 0 (and none shared)
    c.block_table[1].copy_(_i32([0, 1, 2, 4, 5, -1]))
    c.seq_len[1] = 60
    q = torch.empty(2, T, HQ, D, dtype=BF, device="cuda")
    x.layer.stage(*x.block(), q)
    x.layer.verify(q, torch.empty_like(q))
    c.accept(_i32([T, T]), state_idx=_i32([0, 1]))
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0 and c.seq_len.tolist() == [8, 68, 0]
