"""The workspace of a chunk: none for a layer that only stages, allocated with the first chunk, shared or passed as before."""
import pytest
import torch

from test_gpu_attn_chunk import BF, Case, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def need(lib, cache, dims):
    import ctypes
    return lib.load().gdn_attn_chunk_workspace(cache._c, ctypes.byref(dims))


def test_layers_that_stage_hold_none():
    import speculative_decode_recurrent_gb300 as lib
    cache = lib.PagedCache(lib.PageDims(n_slot=2, max_pages=512, n_page=16, page=128, n_layer=1, Hkv=2, d=128, dtype=lib.DTYPE_BF16))
    dims = lib.AttnDims(B=1, T=2048, Hq=16, scale=0.1)
    assert need(lib, cache, dims) > 1 << 20
    w = torch.ones(128, device="cuda")
    rope = lib.RopeDims(rot=0, style=lib.ROPE_HALF, max_pos=100, eps=1e-6)
    q, kv = torch.randn(1, 2048, 16, 128, device="cuda").bfloat16(), torch.randn(1, 2048, 2, 128, device="cuda").bfloat16()
    out = torch.empty_like(q)
    cache.reserve(i32([0]), 100)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    layers = [lib.AttnLayer(dims, cache, 0, rope, w, w) for _ in range(8)]
    for layer in layers:
        layer.stage(q, kv, kv, out, draft_len=i32([100]))
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before < 1 << 16 and int(cache.status.item()) == 0
    layers[0].chunk(q, out, chunk_len=i32([100]))
    assert torch.cuda.memory_allocated() - before >= need(lib, cache, dims)
    assert layers[0].workspace.numel() == need(lib, cache, dims)
    held = torch.cuda.memory_allocated()
    layers[0].chunk(q, out, chunk_len=i32([100]))
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() <= held and int(cache.status.item()) == 0


@pytest.mark.parametrize("first", ["chunk", "workspace", "graph", "stream"])
def test_first_use_of_the_workspace(first):
    c = Case([5000, 40], [100, 66], 100, 4, 2, 128, 16, BF, seed=61)
    lens = i32(c.lens)
    torch.cuda.synchronize()
    call = lambda **kw: c.layer.chunk(c.qd, c.out, lse=c.lse, chunk_len=lens, **kw)
    if first == "workspace":
        c.layer.workspace.fill_(0xFF)                        # no initial content
    if first == "graph":                                     # (with nothing allocated before the capture)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graph.replay()
    elif first == "stream":
        side = torch.cuda.Stream()
        call(stream=side)
        side.synchronize()
    else:
        call()
    c.check()
    c.out.fill_(7)
    call()
    c.check()


def test_a_layer_of_dims_that_chunk_refuses_still_stages():
    """Rows of a stage that a chunk may not have: the constructor does not mind, chunk says so."""
    import speculative_decode_recurrent_gb300 as lib
    c = Case([30], [70], 70, 4, 2, 128, 16, BF, seed=62)
    many = lib.AttnLayer(lib.AttnDims(B=300, T=1 << 20, Hq=4, scale=c.scale), c.cache, 0)
    with pytest.raises(lib.GdnError):
        many.chunk(c.qd, c.out)
    assert many.workspace.numel() == 0
