"""Committed tokens and sampling where offsets pass 32 bits: the last sequence begins 2^31 elements into its tensors."""
import numpy as np
import pytest
import torch

import advance_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
T = 1 << 20


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    yield
    torch.cuda.empty_cache()


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_advance():
    import speculative_decode_recurrent_gb300 as lib
    H, d, n = 16, 128, 100
    g = torch.Generator().manual_seed(1)
    unit = torch.nn.functional.normalize
    dims = lib.Dims(B=2, H=H, dk=d, dv=d, T=1, cap=2, threshold=1, n_slot=2, in_dtype=lib.DTYPE_BF16, scale=d ** -0.5)
    init = dict(state=torch.zeros(2, H, d, d), state_idx=None, buf_k=torch.zeros(2, H, 2, d, dtype=BF), buf_v=torch.zeros(2, H, 2, d, dtype=BF),
                buf_g=torch.zeros(2, H, 2), buf_beta=torch.zeros(2, H, 2), buf_len=torch.zeros(2, dtype=torch.int32))
    layer = lib.ReplayLayer(dims, init)
    q, k, v = (torch.empty(2, T, H, d, dtype=BF, device="cuda") for _ in range(3))
    gate, beta = (torch.empty(2, T, H, device="cuda") for _ in range(2))
    out = torch.full((2, T, H, d), 7.0, device="cuda")
    small = [unit(torch.randn(n, H, d, generator=g), dim=-1).to(BF), unit(torch.randn(n, H, d, generator=g), dim=-1).to(BF),
             torch.randn(n, H, d, generator=g).to(BF), -torch.rand(n, H, generator=g), torch.rand(n, H, generator=g)]
    for x, y in zip((q, k, v, gate, beta), small):
        x[1, :n] = y.cuda()
    layer.advance(q, k, v, gate, beta, out, chunk_len=i32([0, n]))
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    o, S, norm, eff = R.advance(np.zeros((H, d, d)), *(f64(x) for x in small), d ** -0.5)
    tol = R.advance_bound(norm, eff, d, True)
    assert np.abs(f64(layer.t["state"][1]) - S).max() <= tol and (layer.t["state"][0] == 0).all()
    assert np.abs(f64(out[1, :n]) - o).max() <= 1.01 * tol * d ** -0.5
    assert (out[0, ::4099] == 0).all() and (out[1, n:][::4099] == 0).all() and (out[1, -1] == 0).all() and (out[0, -1] == 0).all()


def test_conv():
    import speculative_decode_recurrent_gb300 as lib
    D, W = 2048, 4
    g = torch.Generator().manual_seed(2)
    dims = lib.ConvDims(B=2, D=D, W=W, T=1, cap=W, n_slot=2, act=lib.CONV_ACT_NONE, in_dtype=lib.DTYPE_BF16, out_dtype=lib.DTYPE_BF16)
    weight = torch.randn(D, W, generator=g)
    layer = lib.ConvLayer(dims, dict(ring=torch.zeros(2, W, D, dtype=BF), pos=torch.zeros(2, dtype=torch.int32), state_idx=None, weight=weight))
    x = torch.randn(2, T, D, dtype=BF, device="cuda")
    y = torch.empty_like(x)
    layer.advance(x, y)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    part = f64(x[1, -70:])
    ref, _, mag = R.conv(part[:W - 1], part[W - 1:], f64(weight), np.zeros(D), False)
    assert (np.abs(f64(y[1, -67:]) - ref) <= 1.01 * (2.0 ** -20 * mag + 2.0 ** -8 * np.abs(ref))).all()
    pos = int(layer.t["pos"][1])
    assert pos == T % W
    for j in range(1, W):
        assert torch.equal(layer.t["ring"][1, (pos - j) % W], x[1, -j])


def test_chunk():
    import speculative_decode_recurrent_gb300 as lib
    Hq, Hkv, d, n = 16, 2, 128, 70
    g = torch.Generator().manual_seed(3)
    cache = lib.PagedCache(lib.PageDims(n_slot=2, max_pages=T // 128, n_page=8, page=128, n_layer=1, Hkv=Hkv, d=d, dtype=lib.DTYPE_BF16))
    cache.reserve(i32([0, 1]), n)
    cache.k.copy_(torch.randn(cache.k.shape, generator=g).to(BF))
    cache.v.copy_(torch.randn(cache.v.shape, generator=g).to(BF))
    layer = lib.AttnLayer(lib.AttnDims(B=2, T=T, Hq=Hq, scale=d ** -0.5), cache, 0)
    q = torch.empty(2, T, Hq, d, dtype=BF, device="cuda")
    small = torch.randn(n, Hq, d, generator=g).to(BF)
    q[1, :n] = small.cuda()
    out = torch.full_like(q, 7.0)
    layer.chunk(q, out, chunk_len=i32([0, n]))
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0
    page = int(cache.block_table[1, 0])
    k, v = (f64(x[0, page, :, :n]).repeat(Hq // Hkv, 0) for x in (cache.k, cache.v))       # [Hq, n, d]
    s = np.einsum("thd,hjd->htj", f64(small), k) * d ** -0.5
    s = np.where(np.arange(n)[None, None] <= np.arange(n)[None, :, None], s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    ref, A = np.einsum("htj,hjd->thd", p, v), np.einsum("htj,hjd->thd", p, np.abs(v))
    # a weight's rounding to bf16 and the output's; the scores' and sums' errors in fp32 are below 2^-12 of A
    assert (np.abs(f64(out[1, :n]) - ref) <= 1.01 * (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -8 * np.abs(ref)).all()
    assert (out[0, ::4099] == 0).all() and (out[1, n:][::4099] == 0).all() and (out[1, -1] == 0).all()


def test_sampling():
    import speculative_decode_recurrent_gb300 as lib
    B, n, V = 3, 64, 1 << 24
    s = lib.DraftSampler(lib.DraftDims(B=B, T=n, V=V))
    probs = torch.zeros(B, n, V, device="cuda")
    tokens = torch.randint(0, V, (B, n), dtype=torch.int32, generator=torch.Generator().manual_seed(4)).cuda()
    for t in range(1, n):
        probs[2, t - 1, tokens[2, t].long()] = 1.0          # every draft of the last sequence is certain
    probs[2, n - 1, V - 3] = 1.0
    probs[:2, 0, 5] = 1.0                                   # the others accept none
    tokens[:2, 1] = 6
    acc, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    s.accept(tokens, probs, torch.full((B, n), 0.5, device="cuda"), acc, nxt)
    torch.cuda.synchronize()
    assert acc.tolist() == [1, 1, n] and nxt.tolist() == [5, 5, V - 3] and int(s.status.item()) == 0
