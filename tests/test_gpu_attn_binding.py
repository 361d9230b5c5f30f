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


def test_shapes_of_the_calls():
    """A tensor of the right size in another order is refused; one that lies in memory as the call reads
    it is taken, whatever it is called."""
    lib = _lib()
    B, T, Hq, Hkv, d = 3, 5, 6, 2, 64
    c = R.CacheCase([20, 30, 40], T, Hkv, d, 16, BF, seed=301)
    cache = lib.PagedCache(c.dims(lib), c.init())
    rope = lib.RopeDims(rot=16, style=lib.ROPE_HALF, max_pos=64, eps=1e-6)
    w, tab = torch.ones(d, device="cuda"), torch.ones(64, 16, device="cuda")
    layer = lib.AttnLayer(lib.AttnDims(B=B, T=T, Hq=Hq, scale=0.1), cache, 0, rope, w, w, tab, state_idx=c.state_idx.cuda())
    kv = [torch.randn(B, T, Hkv, d, generator=c.g).to(BF).cuda() for _ in range(2)]
    q = torch.randn(B, T, Hq, d, generator=c.g).to(BF).cuda()
    parent = (torch.arange(T, dtype=torch.int32, device="cuda") - 1).repeat(B, 1)
    i64, i32, f32 = (dict(dtype=x, device="cuda") for x in (torch.int64, torch.int32, torch.float32))

    def same(shape):
        return torch.empty(shape, dtype=BF, device="cuda")
    tree, pos, lse, out = torch.empty(B, T, **i64), torch.empty(B, T, **i32), torch.empty(B, T, Hq, **f32), same((B, T, Hq, d))
    refused = [
        ("q", lambda: layer.verify(q.transpose(1, 2).contiguous(), out)),
        ("q", lambda: layer.verify(q.transpose(1, 2).reshape(B * Hq, T, d), out)),
        ("out", lambda: layer.verify(q, same((B, Hq, T, d)))),
        ("lse", lambda: layer.verify(q, out, lse=torch.empty(B, Hq, T, **f32))),
        ("tree", lambda: layer.verify(q, out, tree=torch.empty(T, B, **i64))),
        ("q_out", lambda: layer.stage(q, *kv, same((B, Hq, T, d)))),
        ("pos", lambda: layer.stage(q, *kv, out, pos=torch.zeros(T, B, **i32))),
        ("parent", lambda: layer.build_tree(parent.t().contiguous(), tree)),
        ("tree", lambda: layer.build_tree(parent, torch.empty(T, B, **i64))),
        ("pos", lambda: layer.build_tree(parent, tree, torch.empty(T, B, **i32)))]
    for name, call in refused:
        with pytest.raises(ValueError, match=f"^{name}: expected shape"):
            call()
    layer.build_tree(parent.flatten(), tree.view(1, B, T), pos)
    layer.stage(q, *kv, out, pos=pos.flatten())
    got = []
    for shape in ((B, T, Hq, d), (B, T, Hq * d), (B * T, Hq, d), (B * T * Hq, d), (-1,), (1, B, T, Hq, d), (B, T * Hq, 1, d)):
        o, z = torch.zeros(B + 1, T, Hq, d, dtype=BF, device="cuda"), torch.zeros(B, T, Hq, **f32)
        layer.verify(q.view(shape), o, lse=z.view(B, -1), tree=tree.view(-1))
        got.append(o[:B])
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0 and all(torch.equal(got[0], x) for x in got[1:])


def test_one_token_in_any_order_of_its_extents():
    """[B, Hq, 1, d] lies in memory as [B, 1, Hq, d]."""
    lib = _lib()
    c = R.CacheCase([20, 30], 1, 2, 64, 16, BF, seed=302)
    cache = lib.PagedCache(c.dims(lib), c.init())
    layer = lib.AttnLayer(lib.AttnDims(B=2, T=1, Hq=4, scale=0.1), cache, 0, state_idx=c.state_idx.cuda())
    q = torch.randn(2, 1, 4, 64, generator=c.g).to(BF).cuda()
    a, b = torch.zeros_like(q), torch.zeros(2, 4, 1, 64, dtype=BF, device="cuda")
    layer.verify(q, a)
    layer.verify(q.transpose(1, 2), b)
    torch.cuda.synchronize()
    assert torch.equal(a.flatten(), b.flatten()) and bool(a.any())


def test_tensors_of_another_device():
    """Tensors are compared with the cache's device before anything is launched (one GPU: the cache is
    told that its device is another one)."""
    lib = _lib()
    B, T, Hq, Hkv, d = 2, 3, 4, 2, 64
    c = R.CacheCase([20, 30], T, Hkv, d, 16, BF, seed=303)
    cache, idx = lib.PagedCache(c.dims(lib), c.init()), c.state_idx.cuda()
    rope = lib.RopeDims(rot=16, style=lib.ROPE_HALF, max_pos=64, eps=1e-6)
    w, tab = torch.ones(d, device="cuda"), torch.ones(64, 16, device="cuda")
    dims = lib.AttnDims(B=B, T=T, Hq=Hq, scale=0.1)
    layer = lib.AttnLayer(dims, cache, 0, rope, w, w, tab, state_idx=idx)
    x, kv = torch.zeros(B, T, Hq, d, dtype=BF, device="cuda"), torch.zeros(B, T, Hkv, d, dtype=BF, device="cuda")
    n, tree = _i32([1, 1]), torch.zeros(B, T, dtype=torch.int64, device="cuda")
    cache._index = layer._index = 5
    stream = torch.cuda.current_stream()
    for call in (lambda: cache.reserve(n, 1, stream), lambda: cache.release(n, stream),
                 lambda: cache.fork(n, n, torch.zeros(2, 2, dtype=torch.int32, device="cuda"), stream),
                 lambda: cache.accept(n, stream=stream), lambda: cache.accept(n, path=_i32([[0], [0]]), stream=stream),
                 lambda: layer.stage(x, kv, kv, x, stream=stream), lambda: layer.verify(x, x, stream=stream),
                 lambda: layer.build_tree(tree.to(torch.int32), tree, stream=stream),
                 lambda: lib.AttnLayer(dims, cache, 0, state_idx=idx)):
        with pytest.raises(ValueError, match="cache's device"):
            call()


def test_the_layer_keeps_what_its_calls_read():
    """The calls use the tensors that the layer was made with; it holds on to them, whatever its attributes
    are set to."""
    import gc
    import weakref
    lib = _lib()
    c = R.CacheCase([20, 30], 3, 2, 64, 16, BF, seed=304)
    cache = lib.PagedCache(c.dims(lib), c.init())
    layer = lib.AttnLayer(lib.AttnDims(B=2, T=3, Hq=4, scale=0.1), cache, 0, state_idx=c.state_idx.cuda())
    held = [weakref.ref(layer.state_idx), weakref.ref(layer.workspace)]
    layer.state_idx = layer.workspace = None
    gc.collect()
    assert all(x() is not None for x in held)
