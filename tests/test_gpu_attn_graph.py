"""A decode loop's attention calls captured in a CUDA graph: the same bits as called one by one."""
import pytest
import torch

import attn_ref as R
from test_gpu_attn import BF, F32, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


class Loop:
    """Two layers over one cache: room, a tree, staging and verify in each layer, an accepted path; a fork
    given up again."""

    def __init__(self, dtype, B, T, Hq, Hkv, d, page):
        import speculative_decode_recurrent_gb300 as lib
        g = torch.Generator().manual_seed(700)
        c = R.CacheCase([37 * b % 200 for b in range(B)], 0, Hkv, d, page, dtype, layers=2, seed=701, spare=8 * B + 40,
                        extra_slots=2)
        dims = c.dims(lib)
        dims.max_pages = c.max_pages + -(-4 * T // page)
        init = dict(c.init(), block_table=torch.nn.functional.pad(c.block_table, (0, dims.max_pages - c.max_pages), value=-1))
        self.cache, self.idx, self.T, self.rows = lib.PagedCache(dims, init), c.state_idx.cuda(), T, c.state_idx
        self.first, self.spare = self.idx[:1].clone(), _i32([s for s in range(c.n_slot) if s not in c.state_idx.tolist()][:1])
        rope = lib.RopeDims(rot=d // 2, style=lib.ROPE_HALF, max_pos=512, eps=1e-6)
        w, a = (1 + 0.2 * torch.randn(2, d, generator=g)).cuda(), 6.28 * torch.rand(512, d // 4, generator=g)
        tab = torch.cat([a.cos(), a.sin()], 1).cuda()
        self.layers = [lib.AttnLayer(lib.AttnDims(B=B, T=T, Hq=Hq, scale=d ** -0.5), self.cache, x, rope, w[0], w[1], tab,
                                     state_idx=self.idx) for x in range(2)]
        self.x = [torch.empty(B, T, h, d, dtype=dtype, device="cuda") for h in (Hq, Hkv, Hkv)]
        self.parent = torch.empty(B, T, dtype=torch.int32, device="cuda")
        self.path, self.accepted = torch.zeros_like(self.parent), torch.empty(B, dtype=torch.int32, device="cuda")
        self.tree, self.pos = torch.empty(B, T, dtype=torch.int64, device="cuda"), torch.empty_like(self.parent)
        self.q, self.out = torch.empty_like(self.x[0]), [torch.empty_like(self.x[0]) for _ in range(2)]
        self.lse = [torch.empty(B, T, Hq, device="cuda") for _ in range(2)]
        self.copies = torch.empty(1, 2, dtype=torch.int32, device="cuda")

    def inputs(self, seed):
        g = torch.Generator().manual_seed(seed)
        B, T = self.parent.shape
        for x in self.x:
            x.copy_(torch.randn(x.shape, generator=g))
        self.parent.copy_(R.random_parents(B, T, g))
        n = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
        self.accepted.copy_(n)
        self.path.copy_(torch.stack([torch.nn.functional.pad(torch.randperm(T, generator=g)[:k].sort()[0], (0, T - k))
                                     for k in n.tolist()]))

    def step(self):
        self.cache.reserve(self.idx, self.T)
        self.layers[0].build_tree(self.parent, self.tree, self.pos)
        for layer, out, lse in zip(self.layers, self.out, self.lse):
            layer.stage(*self.x, self.q, pos=self.pos)
            layer.verify(self.q, out, lse=lse, tree=self.tree)
        self.cache.accept(self.accepted, path=self.path, state_idx=self.idx)
        self.cache.fork(self.first, self.spare, self.copies)
        self.cache.release(self.spare)

    def state(self):
        c = self.cache
        return [x.clone().view(torch.uint8) for x in (*self.out, *self.lse, self.q, c.k, c.v, c.block_table, c.seq_len, c.n_owned,
                                                      c.ref, c.free_list, c.free_count, c.status)]


@pytest.mark.parametrize("dtype,B,T,Hq,Hkv,d,page", [(BF, 5, 8, 8, 2, 128, 16), (BF, 4, 24, 24, 2, 64, 64),
                                                     (BF, 2, 5, 4, 1, 256, 32), (F32, 3, 6, 6, 2, 64, 16)])
def test_a_captured_step(dtype, B, T, Hq, Hkv, d, page):
    eager, graphed = (Loop(dtype, B, T, Hq, Hkv, d, page) for _ in range(2))
    want = []
    for seed in range(3):
        eager.inputs(seed)
        eager.step()
        want.append(eager.state())
    assert int(eager.cache.status.item()) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    assert int(graphed.cache.status.item()) == 0 and torch.equal(graphed.cache.seq_len[graphed.rows.long()].cpu(),
                                                                 torch.tensor([37 * b % 200 for b in range(B)], dtype=torch.int32))
    for seed in range(3):
        graphed.inputs(seed)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(want[seed], graphed.state())):
            assert torch.equal(a, b), (seed, i)
