"""Calls on committed tokens and drafts captured in CUDA graphs and replayed: the bits of eager calls.  Prompts of several launches, groups
of sequences, the convolution in one launch and in two, chains and trees."""
import pytest
import torch

from advance_plan import plan
from test_gpu_advance import BF, Case, i32
from test_gpu_draft import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def replayed(calls, tensors, start):
    """Eager results of ``calls`` on ``tensors``, which ``start`` sets back, against those of three replays of one graph."""
    start()
    calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in tensors]
    graph = torch.cuda.CUDAGraph()
    start()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        start()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(tensors, want):
            assert torch.equal(t, w)


@pytest.mark.parametrize("lens,T,H,dk,dv,launches", [
    ([4096], 4096, 16, 128, 128, 2), ([1500], 1500, 30, 64, 64, 2), ([700, 33, 0], 700, 96, 128, 64, 1), ([65, 40] * 45, 70, 64, 128, 128, 4)])
def test_advance_of_several_launches(lens, T, H, dk, dv, launches):
    c = Case(lens, T, H, H, dk, dv, BF, seed=81, fresh=[b % 2 for b in range(len(lens))])
    p = plan(len(lens), T, H, dk, dv, torch.cuda.get_device_properties(0).multi_processor_count)
    assert len(p["sizes"]) * -(-len(lens) // p["seqs"]) >= launches
    first, n, f = c.state.cuda(), i32(c.lens), i32(c.fresh)
    ws = c.layer.advance_workspace(T, H)

    def start():
        c.layer.t["state"].copy_(first)
        c.out.fill_(3)

    def calls():                                             # (twice: the second goes on from the first one's state)
        for fresh in (f, None):
            c.layer.advance(c.q, c.k, c.v, c.g, c.beta, c.out, chunk_len=n, fresh=fresh, workspace=ws)

    if any(c.fresh):
        first[c.slots.long().cuda()[f.bool()]] = 0.0         # (NaN there would not compare)
    replayed(calls, [c.out, c.layer.t["state"]], start)
    assert int(c.layer.status.item()) == 0


@pytest.mark.parametrize("B,T,D", [(2, 9, 264), (3, 200, 2056), (8, 1500, 2048)])
def test_conv(B, T, D):
    import speculative_decode_recurrent_gb300 as lib
    g = torch.Generator().manual_seed(82)
    dims = lib.ConvDims(B=B, D=D, W=4, T=1, cap=7, n_slot=B, in_dtype=lib.DTYPE_BF16, out_dtype=lib.DTYPE_BF16, act=lib.CONV_ACT_SILU)
    ring, pos = torch.randn(B, 7, D, generator=g).to(BF).cuda(), i32([b % 7 for b in range(B)])
    layer = lib.ConvLayer(dims, dict(ring=ring, pos=pos, state_idx=None, weight=torch.randn(D, 4, generator=g)))
    x = torch.randn(B, T, D, generator=g).to(BF).cuda()
    y, n = torch.empty_like(x), i32([T - b for b in range(B)])

    def start():
        layer.t["ring"].copy_(ring)
        layer.t["pos"].copy_(pos)
        y.fill_(1)

    def calls():
        for _ in range(2):
            layer.advance(x, y, chunk_len=n)

    ring, pos = ring.clone(), pos.clone()
    replayed(calls, [y, layer.t["ring"], layer.t["pos"]], start)
    assert int(layer.status.item()) == 0


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,T,V", [(1, 8, 3000), (5, 12, 40001)])
def test_sampling(B, T, V, tree):
    import speculative_decode_recurrent_gb300 as lib
    tokens, parent, p, q, u = (x.cuda() for x in inputs(B, T, V, torch.Generator().manual_seed(83), tree))
    s = lib.DraftSampler(lib.DraftDims(B=B, T=T, V=V))
    acc, nxt = i32([0] * B), i32([0] * B)
    path = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    parent = parent.contiguous() if tree else None

    def start():
        for t in (acc, nxt, path):
            t.fill_(-5)

    replayed(lambda: s.accept(tokens, p, u, acc, nxt, draft=q, parent=parent, path=path), [acc, nxt, path], start)
    assert int(s.status.item()) == 0 and (acc >= 1).all() and (nxt >= 0).all()
