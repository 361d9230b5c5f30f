"""What the Python binding of the attention layers checks beyond the library's own refusals."""
import pytest
import torch

import attn_ref as R
from test_gpu_attn import BF, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def _lib():
    import speculative_decode_recurrent_gb300 as lib
    return lib


def test_accept_of_more_than_the_draft():
    """A chain's accept knows the draft's length: a count past it commits nothing."""
    lib = _lib()
    c = R.CacheCase([20, 30, 40], 16, 2, 64, 16, BF, seed=300)
    cache, idx = lib.PagedCache(c.dims(lib), c.init()), c.state_idx.cuda()
    want = c.seq_len.clone()
    cache.accept(_i32([3, 6, 5]), state_idx=idx, T=5)
    torch.cuda.synchronize()
    want[c.state_idx[0].long()] += 3
    want[c.state_idx[2].long()] += 5
    assert int(cache.status.item()) == lib.STATUS_BAD_ACCEPT and torch.equal(cache.seq_len.cpu(), want)
    cache.status.zero_()
    cache.accept(_i32([1, 6, 0]), state_idx=idx)              # without it, up to 64
    torch.cuda.synchronize()
    want[c.state_idx[0].long()] += 1
    want[c.state_idx[1].long()] += 6
    assert int(cache.status.item()) == 0 and torch.equal(cache.seq_len.cpu(), want)
    path = torch.arange(5, dtype=torch.int32, device="cuda").repeat(3, 1)
    with pytest.raises(ValueError, match="path: expected 4 tokens"):
        cache.accept(_i32([1, 1, 1]), path=path, state_idx=idx, T=4)
    with pytest.raises(lib.GdnError):
        cache.accept(_i32([1, 1, 1]), state_idx=idx, T=65)
    assert torch.equal(cache.seq_len.cpu(), want)
