"""gdn_draft_accept against a plain 64-bit form (tests/advance_ref.py)."""
import numpy as np
import pytest
import torch

import advance_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def inputs(B, T, V, g, tree, spread=1.5, noise=0.7):
    z = spread * torch.randn(B, T, V, generator=g)
    p = torch.softmax(z, -1)
    q = torch.softmax(z + noise * torch.randn(B, T, V, generator=g), -1)
    t = torch.arange(T)
    parent = (t - 1).expand(B, T)
    if tree:
        parent = torch.where(t == 0, -1, (t - 1 - (torch.rand(B, T, generator=g) * 4).long()).clamp(min=0))
    tokens = torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        for i in range(1, T):
            tokens[b, i] = torch.multinomial(q[b, max(int(parent[b, i]), 0)], 1, generator=g)
    return tokens.int(), parent.int(), p, q, torch.rand(B, T, generator=g)


def run(tokens, parent, p, q, u, lens, tree, pad=0):
    import speculative_decode_recurrent_gb300 as lib
    B, T, V = p.shape
    s = lib.DraftSampler(lib.DraftDims(B=B, T=T, V=V))
    acc, nxt = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    path = torch.full((B, T), -7, dtype=torch.int32, device="cuda")

    def dev(x):
        if x is None:
            return None
        y = torch.full((B, T, V + pad), float("nan"), device="cuda")
        y[..., :V] = x
        return y[..., :V]

    s.accept(tokens.cuda(), dev(p), u.cuda(), acc, nxt, draft=dev(q), parent=parent.cuda() if tree else None, path=path,
             draft_len=i32(lens))
    torch.cuda.synchronize()
    return acc.tolist(), nxt.tolist(), path.tolist(), int(s.status.item())


@pytest.mark.parametrize("drafter", ["dist", "point"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,T,V,pad", [(3, 1, 5, 0), (9, 6, 2, 1), (7, 16, 1000, 0), (5, 64, 1025, 3), (3, 9, 4097, 0),
                                       (2, 12, 40001, 0), (2, 7, 65536, 4)])
def test_accept_matches_the_definition(B, T, V, pad, tree, drafter):
    g = torch.Generator().manual_seed(100 + V)
    tokens, parent, p, q, u = inputs(B, T, V, g, tree)
    lens = [T] + [int(torch.randint(0, T + 1, (1,), generator=g)) for _ in range(B - 1)]
    qq = q if drafter == "dist" else None
    acc, nxt, path, status = run(tokens, parent, p, qq, u, lens, tree, pad)
    assert status == 0
    for b, n in enumerate(lens):
        ref, v, near = R.sample(tokens[b].tolist(), parent[b].tolist(), p[b].double().numpy(), None if qq is None else q[b].double().numpy(),
                                u[b].double().numpy(), n)
        assert near > 2.0 ** -40                   # the seed is not one of the undecided ones
        assert acc[b] == len(ref) and path[b] == ref + [-1] * (T - len(ref)) and nxt[b] == v, (b, n)


def test_borders_are_exact():
    """Probabilities of a power of two: the running sums are exact, and a draw on a border takes the next token."""
    V, T, B = 1 << 16, 2, 64
    p = torch.full((B, T, V), 2.0 ** -16)
    u = torch.zeros(B, T)
    at = torch.randint(0, V, (B,), generator=torch.Generator().manual_seed(3))
    u[:, 0] = at / V
    tokens = torch.zeros(B, T, dtype=torch.int32)
    acc, nxt, _, status = run(tokens, None, p, None, u, [1] * B, False)
    assert status == 0 and acc == [1] * B and nxt == at.tolist()
    # accepted where u q < p, so not at u q = p
    q = torch.full((B, T, V), 2.0 ** -15)
    u[:, 1] = 0.5
    u[::2, 1] = 0.5 - 2.0 ** -24
    acc, _, _, _ = run(tokens, None, p, q, u, [2] * B, False)
    assert acc == [2, 1] * (B // 2)


def test_no_mass_left_and_no_mass_at_all():
    import speculative_decode_recurrent_gb300 as lib
    V, T = 5000, 2
    p = torch.zeros(5, T, V)
    p[:, :, 4321] = 1.0
    q = p.clone()
    p[1] = 0
    p[2, 0, 7] = float("inf")
    p[3, 0, 7] = float("nan")                      # counts as 0
    p[4, 0, 9] = -3.0                              # as well
    q[2:] = 0
    tokens = torch.full((5, T), 17, dtype=torch.int32)
    acc, nxt, _, status = run(tokens, None, p, q, torch.full((5, T), 0.75), [2] * 5, False)
    # q has no mass at 17 and p neither: rejected; the rest p - q has none, so p is drawn from
    assert acc == [1] * 5 and nxt == [4321, -1, -1, 4321, 4321] and status == lib.STATUS_BAD_PROB


def test_bad_inputs_accept_nothing():
    import speculative_decode_recurrent_gb300 as lib
    g = torch.Generator().manual_seed(5)
    tokens, parent, p, q, u = inputs(6, 5, 300, g, True)
    tokens[0, 2], tokens[1, 1] = 300, -1
    parent[2, 3], parent[3, 1] = 3, -2
    tokens[5, 0] = 99999                           # token 0 is not looked at
    acc, nxt, path, status = run(tokens, parent, p, q, u, [5, 5, 5, 5, 6, 5], True)
    assert status == lib.STATUS_BAD_TOKEN | lib.STATUS_BAD_TREE | lib.STATUS_BAD_LEN
    assert acc[:5] == [0] * 5 and nxt[:5] == [-1] * 5 and path[:5] == [[-1] * 5] * 5
    assert acc[5] >= 1 and nxt[5] >= 0


def test_accepted_and_next_are_distributed_as_the_target():
    """4096 drafts of two children over 3 tokens: token after the root is distributed as p_0 (5 standard deviations)."""
    n, V = 4096, 3
    g = torch.Generator().manual_seed(9)
    p0, q0 = torch.tensor([0.5, 0.2, 0.3]), torch.tensor([0.1, 0.6, 0.3])
    p = p0.expand(n, 3, V).contiguous()
    q = q0.expand(n, 3, V).contiguous()
    tokens = torch.multinomial(q0, n * 3, replacement=True, generator=g).reshape(n, 3).int()
    parent = torch.tensor([-1, 0, 0], dtype=torch.int32).expand(n, 3).contiguous()
    acc, nxt, path, status = run(tokens, parent, p, q, torch.rand(n, 3, generator=g), [3] * n, True)
    first = [int(tokens[i, path[i][1]]) if acc[i] > 1 else nxt[i] for i in range(n)]
    count = np.bincount(first, minlength=V) / n
    assert status == 0 and (np.abs(count - p0.numpy()) <= 5 * np.sqrt(p0.numpy() * (1 - p0.numpy()) / n)).all()


def test_graph_replay_follows_its_inputs():
    import speculative_decode_recurrent_gb300 as lib
    B, T, V = 4, 8, 9000
    s = lib.DraftSampler(lib.DraftDims(B=B, T=T, V=V))
    bufs = [torch.zeros(B, T, dtype=torch.int32, device="cuda"), torch.zeros(B, T, dtype=torch.int32, device="cuda"),
            torch.zeros(B, T, V, device="cuda"), torch.zeros(B, T, V, device="cuda"), torch.zeros(B, T, device="cuda")]
    acc, nxt = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    path = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.accept(bufs[0], bufs[2], bufs[4], acc, nxt, draft=bufs[3], parent=bufs[1], path=path)
    for seed in (1, 2):
        x = inputs(B, T, V, torch.Generator().manual_seed(seed), True)
        for a, b in zip(bufs, x):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            ref, v, _ = R.sample(x[0][b].tolist(), x[1][b].tolist(), x[2][b].double().numpy(), x[3][b].double().numpy(), x[4][b].double().numpy(), T)
            assert acc.tolist()[b] == len(ref) and nxt.tolist()[b] == v and path.tolist()[b][:len(ref)] == ref


@pytest.mark.parametrize("drafter", ["dist", "point"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,T,V,pad", [(3, 5, 150001, 0), (1, 2, 1 << 24, 0), (4, 3, 4096, 2), (1, 64, 70000, 0)])
def test_large_vocabularies(B, T, V, pad, tree, drafter):
    g = torch.Generator().manual_seed(7 + T)
    z = torch.randn(B, T, V, generator=g)
    p = torch.softmax(z, -1)
    q = torch.softmax(z + 0.7 * torch.randn(B, T, V, generator=g), -1)
    parent = torch.arange(-1, T - 1, dtype=torch.int32).expand(B, T).contiguous()
    if tree:
        parent[:, 1:] = (torch.arange(T - 1, dtype=torch.int32) // 3)[None]
    tokens = torch.empty(B, T, dtype=torch.int32)
    for b in range(B):
        for t in range(T):
            tokens[b, t] = (q if t % 2 else p)[b, max(int(parent[b, t]), 0)].argmax()
    u = torch.rand(B, T, generator=g)
    u[:, 1:] *= 0.9                                # (the likeliest token of a row: often accepted, siblings alike)
    acc, nxt, path, status = run(tokens, parent, p, q if drafter == "dist" else None, u, [T] * B, tree, pad)
    assert status == 0
    for b in range(B):
        ref, v, near = R.sample(tokens[b].tolist(), parent[b].tolist(), p[b].double().numpy(),
                                q[b].double().numpy() if drafter == "dist" else None, u[b].double().numpy(), T)
        assert near > 2.0 ** -40
        assert acc[b] == len(ref) and path[b] == ref + [-1] * (T - len(ref)) and nxt[b] == v, b


@pytest.mark.parametrize("V", [3, 4099, 140000])
def test_random_numbers_at_and_past_the_ends(V):
    """u of 0 takes the first token with mass, one just below 1 (or, outside what the header asks for, 1 and more) the last;
    NaN and negative numbers still give a token with mass."""
    p = torch.zeros(6, 1, V)
    p[..., 1], p[..., V - 2] = 0.5, 0.5
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 3.0, float("nan"), -1.0])[:, None]
    acc, nxt, _, status = run(torch.zeros(6, 1, dtype=torch.int32), None, p, None, u, [1] * 6, False)
    assert status == 0 and acc == [1] * 6
    assert nxt[0] == 1 and nxt[1:4] == [V - 2] * 3 and all(x in (1, V - 2) for x in nxt[4:])


def test_another_stream_and_no_sequences():
    import speculative_decode_recurrent_gb300 as lib
    tokens, _, p, q, u = inputs(3, 4, 9000, torch.Generator().manual_seed(8), False)
    want = run(tokens, None, p, q, u, [4] * 3, False)[:2]
    s, side = lib.DraftSampler(lib.DraftDims(B=3, T=4, V=9000)), torch.cuda.Stream()
    x = [t.cuda() for t in (tokens, p, u, q)]
    acc, nxt = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    side.wait_stream(torch.cuda.current_stream())
    s.accept(*x[:3], acc, nxt, draft=x[3], stream=side)
    side.synchronize()
    assert (acc.tolist(), nxt.tolist()) == want
    none = lib.DraftSampler(lib.DraftDims(B=0, T=4, V=9000))
    none.accept(*(t[:0] for t in x[:3]), acc[:0], nxt[:0])
    with pytest.raises(ValueError, match="u: needs"):
        s.accept(*x[:2], x[2][:, :3].contiguous(), acc, nxt)
    with pytest.raises((ValueError, TypeError)):
        s.accept(x[0].long(), *x[1:3], acc, nxt)
    with pytest.raises(lib.GdnError):              # a tree needs a path
        s.accept(*x[:3], acc, nxt, parent=x[0])
