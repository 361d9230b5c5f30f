"""gdn_replay_advance and gdn_conv_advance against plain 64-bit forms (tests/advance_ref.py)."""
import numpy as np
import pytest
import torch

import advance_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A layer of B + 2 slots under a random map, and tokens whose rows past a sequence's length hold NaN; q, k and v
    lie in one tensor, so that a token's stride is not its width."""

    def __init__(self, lens, T, H, Hk, dk, dv, dtype, seed=0, fresh=None, gates="normal", packed=True):
        import speculative_decode_recurrent_gb300 as lib
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.lens, self.T, self.H, self.Hk, self.dk, self.dv, self.B = lens, T, H, Hk, dk, dv, B
        unit = torch.nn.functional.normalize
        w = [Hk * dk, Hk * dk, H * dv]
        all_ = torch.empty(B, T, sum(w) + 16)
        q, k, v = (x.unflatten(-1, (-1, n)) for x, n in zip(all_[..., :-16].split(w, -1), (dk, dk, dv)))
        q.copy_(unit(torch.randn(B, T, Hk, dk, generator=g), dim=-1))
        k.copy_(unit(torch.randn(B, T, Hk, dk, generator=g), dim=-1))
        v.copy_(torch.randn(B, T, H, dv, generator=g))
        gate = -torch.nn.functional.softplus(torch.randn(B, T, H, generator=g))
        beta = torch.sigmoid(torch.randn(B, T, H, generator=g))
        if gates == "extreme":
            r = torch.rand(B, T, H, generator=g)
            gate = torch.where(r < 0.3, torch.zeros_like(gate), torch.where(r < 0.4, torch.full_like(gate, -20.0), 0.05 * gate))
            beta = torch.where(r > 0.9, torch.full_like(beta, 1 - 1e-4), torch.where(r > 0.8, torch.full_like(beta, 1e-4), beta))
        elif gates == "slow":
            gate = 1e-3 * gate
        for b, n in enumerate(lens):
            all_[b, n:] = gate[b, n:] = beta[b, n:] = float("nan")
        all_ = all_.to(dtype).cuda()
        parts = all_[..., :-16].split(w, -1) if packed else [x.contiguous() for x in all_[..., :-16].split(w, -1)]
        self.q, self.k, self.v = (x.unflatten(-1, (-1, n)) for x, n in zip(parts, (dk, dk, dv)))
        self.g, self.beta = gate.cuda(), beta.cuda()
        self.slots = torch.randperm(B + 2, generator=g)[:B].to(torch.int32)
        self.state = 0.3 * torch.randn(B + 2, H, dv, dk, generator=g)
        self.fresh = fresh if fresh is not None else [0] * B
        for b in range(B):
            if self.fresh[b]:
                self.state[self.slots[b].item()] = float("nan")
        cap = 20
        self.dims = lib.Dims(B=B, H=H, dk=dk, dv=dv, T=4, cap=cap, threshold=8, n_slot=B + 2,
                             in_dtype=lib.DTYPE_BF16 if dtype == BF else lib.DTYPE_F32, scale=dk ** -0.5)
        init = dict(state=self.state, state_idx=self.slots, buf_k=torch.zeros(B + 2, H, cap, dk, dtype=dtype),
                    buf_v=torch.zeros(B + 2, H, cap, dv, dtype=dtype), buf_g=torch.zeros(B + 2, H, cap),
                    buf_beta=torch.zeros(B + 2, H, cap), buf_len=torch.zeros(B + 2, dtype=torch.int32))
        self.layer = lib.ReplayLayer(self.dims, init)
        self.out = torch.full((B, T, H, dv), 7.0, device="cuda")

    def run(self, **kw):
        self.layer.advance(self.q, self.k, self.v, self.g, self.beta, self.out, chunk_len=i32(self.lens),
                           fresh=i32(self.fresh), **kw)

    def check(self, chunked, out=None, state=None):
        torch.cuda.synchronize()
        out, state = f64(self.out if out is None else out), f64(self.layer.t["state"] if state is None else state)
        assert int(self.layer.status.item()) == 0
        used = set()
        for b, n in enumerate(self.lens):
            s = int(self.slots[b])
            used.add(s)
            S0 = np.zeros_like(state[s]) if self.fresh[b] else f64(self.state[s])
            o, S, norm, eff = R.advance(S0, f64(self.q[b, :n]), f64(self.k[b, :n]), f64(self.v[b, :n]), f64(self.g[b, :n]),
                                        f64(self.beta[b, :n]), self.dk ** -0.5)
            tol = R.advance_bound(norm, eff, self.dk, chunked)
            assert np.abs(state[s] - S).max() <= tol, (b, n)
            if n:
                assert np.abs(out[b, :n] - o).max() <= tol * 1.01 * self.dk ** -0.5, (b, n)
            assert (out[b, n:] == 0).all()
        for s in set(range(self.B + 2)) - used:
            assert (state[s] == f64(self.state[s])).all()


def is_chunked(dtype, T):
    return dtype == BF                       # (the wider bound; short chunks stay far below it)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,T,H,Hk,dk,dv,fresh", [
    ([1], 1, 1, 1, 128, 128, [0]),
    ([1, 1, 0], 1, 4, 2, 64, 64, [0, 1, 1]),
    ([5, 0, 17, 16], 17, 3, 3, 64, 128, [1, 0, 0, 1]),
    ([63, 64, 65, 1], 65, 2, 1, 128, 64, [0, 1, 0, 0]),
    ([127, 128, 129, 200, 0], 200, 6, 2, 128, 128, [0, 0, 1, 1, 0]),
    ([333, 61], 333, 2, 2, 64, 64, [0, 1]),
    ([700], 700, 5, 1, 128, 128, [0]),
])
def test_advance_matches_the_formula(lens, T, H, Hk, dk, dv, fresh, dtype):
    c = Case(lens, T, H, Hk, dk, dv, dtype, seed=11, fresh=fresh)
    c.run()
    c.check(is_chunked(dtype, T))


@pytest.mark.parametrize("gates", ["extreme", "slow"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_advance_gates(gates, dk, dv):
    c = Case([450, 321], 450, 3, 3, dk, dv, BF, seed=12, gates=gates, packed=False)
    c.run()
    c.check(True)


def ragged(B, T, seed):
    """Lengths of B sequences in chunks of T, among them T, 0 and what lies around a tile's end."""
    g = np.random.default_rng(seed)
    lens = g.integers(0, T + 1, B)
    edge = [x for x in (T, 0, 1, 32, 33, 63, 64, 65, T - 1) if x <= T][:B]
    lens[g.permutation(B)[:len(edge)]] = edge
    return [int(x) for x in lens]


@pytest.mark.parametrize("B,T,H,Hk,dk,dv", [
    (20, 140, 2, 1, 128, 128),               # heads walked whole
    (20, 150, 2, 2, 64, 128),
    (6, 140, 4, 2, 128, 128),                # slices of 32 columns
    (10, 150, 5, 5, 64, 64),
    (11, 90, 4, 1, 128, 64),
    (2, 1100, 12, 12, 64, 128),
    (3, 1100, 2, 1, 128, 128),               # a long prompt's further launches, by slices of 16
    (2, 1300, 3, 3, 64, 64),
    (3, 1100, 14, 7, 128, 128),              # and by heads
    (4, 1090, 10, 10, 64, 128),
    (110, 40, 16, 4, 128, 128),              # more sequences than a launch's workspace holds
])
def test_advance_many_heads_and_long_prompts(B, T, H, Hk, dk, dv):
    lens = ragged(B, T, T)
    c = Case(lens, T, H, Hk, dk, dv, BF, seed=19, fresh=[b % 3 == 1 for b in range(B)])
    c.run()
    first = c.out.clone(), c.layer.t["state"].clone()
    c.check(True)
    c.layer.t["state"].copy_(c.state)
    c.out.fill_(5)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, first[0]) and torch.equal(c.layer.t["state"], first[1])


@pytest.mark.parametrize("B,H,dk,dv", [(1, 4, 128, 128), (2, 9, 128, 128), (5, 6, 64, 64), (3, 13, 64, 128), (12, 16, 128, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_advance_token_by_token_at_every_share_of_the_sms(B, H, dk, dv, dtype):
    c = Case(ragged(B, 19, 3 * B), 19, H, H, dk, dv, dtype, seed=24, fresh=[b % 2 for b in range(B)])
    c.run()
    c.check(False)


@pytest.mark.parametrize("T,dtype", [(300, BF), (20, BF), (70, F32)])
def test_advance_decays_that_forget_the_state(T, dtype):
    """A log-decay of -infinity or far below what fp32 holds is a decay of 0: nothing of the state before it is left."""
    c = Case([T, T - 3], T, 2, 1, 128, 64, dtype, seed=20)
    g = torch.Generator().manual_seed(21)
    pick = torch.rand(c.g.shape, generator=g).cuda()
    for b, n in enumerate(c.lens):
        for lo, x in ((0.0, -float("inf")), (0.03, -1e30), (0.06, -150.0), (0.09, -1e-30), (0.12, 0.0)):
            hit = (pick[b, :n] >= lo) & (pick[b, :n] < lo + 0.03)
            c.g[b, :n][hit] = x
    c.g[0, 0] = -float("inf")
    c.run()
    c.check(is_chunked(dtype, T))


def test_advance_keeps_a_bad_head_to_itself():
    """NaN in a token of one head: the other heads and sequences are as if it were not there."""
    c = Case([130, 130], 130, 4, 4, 128, 128, BF, seed=22)
    c.run()
    out, state = c.out.clone(), c.layer.t["state"].clone()
    c.layer.t["state"].copy_(c.state)
    c.v[0, 70, 1, 5] = float("nan")
    c.q[1, 100, 3, 7] = float("inf")
    c.run()
    torch.cuda.synchronize()
    s0, s1 = (int(x) for x in c.slots)
    same = c.out == out
    assert same[0, :, [0, 2, 3]].all() and same[1, :, :3].all() and same[0, :64, 1].all() and same[1, :64, 3].all()
    assert not torch.isfinite(c.out[1, 100, 3]).all() and torch.isnan(c.out[0, 70:, 1, 5]).all()
    now = c.layer.t["state"]
    assert torch.equal(now[s1], state[s1]) and torch.equal(now[s0, [0, 2, 3]], state[s0, [0, 2, 3]])


def test_advance_in_pieces_is_the_whole():
    """A prompt in chunks of odd lengths, then single tokens: the state is that of one call, within the bound."""
    c = Case([256], 256, 4, 4, 128, 128, BF, seed=13)
    at = 0
    for n in (100, 1, 64, 65, 25, 1):
        part = slice(at, at + n)
        o = torch.empty(1, n, 4, 128, device="cuda")
        c.layer.advance(*(x[:, part] for x in (c.q, c.k, c.v)), c.g[:, part].contiguous(), c.beta[:, part].contiguous(), o)
        c.out[:, part] = o
        at += n
    assert at == 256
    c.check(True)


def test_advance_then_decode_is_one_sequence():
    """Prompt, then a draft verified, accepted and folded: the state is that of all tokens in a row."""
    c = Case([90, 75], 90, 2, 2, 128, 128, BF, seed=14, fresh=[1, 1])
    c.run()
    first = c.out.clone()
    d = Case([4, 4], 4, 2, 2, 128, 128, BF, seed=15, packed=False)
    o = torch.empty(2, 4, 2, 128, device="cuda")
    dense = [x.contiguous() for x in (d.q, d.k, d.v)]
    c.layer.verify(*dense, d.g, d.beta, o)
    c.layer.accept(i32([3, 4]))
    c.layer.flush(force=True)
    torch.cuda.synchronize()
    state = f64(c.layer.t["state"])
    for b, (n, m) in enumerate(zip(c.lens, (3, 4))):
        cat = [np.concatenate([f64(x[b, :n]), f64(y[b, :m])]) for x, y in ((c.q, d.q), (c.k, d.k), (c.v, d.v), (c.g, d.g), (c.beta, d.beta))]
        ref, S, norm, eff = R.advance(np.zeros((2, 128, 128)), *cat, 128 ** -0.5)
        tol = R.advance_bound(norm, eff, 128, True)
        assert np.abs(state[int(c.slots[b])] - S).max() <= tol
        assert np.abs(f64(first[b, :n]) - ref[:n]).max() <= tol
        assert np.abs(f64(o[b, :m]) - ref[n:]).max() <= 2e-3 * np.abs(ref[n:]).max() + tol


def test_advance_bad_sequences_are_skipped():
    import speculative_decode_recurrent_gb300 as lib
    c = Case([70, 70, 70, 70], 70, 2, 2, 128, 128, BF, seed=16)
    idx = c.layer.t["state_idx"]
    idx[0] = 99
    c.layer.t["buf_len"][int(c.slots[1])] = 3
    c.lens = [70, 70, 71, 70]
    c.run()
    torch.cuda.synchronize()
    assert int(c.layer.status.item()) == lib.STATUS_BAD_SLOT | lib.STATUS_BAD_LEN
    assert (c.out[:3] == 7).all() and not (c.out[3] == 7).any()
    for b in (1, 2):
        s = int(c.slots[b])
        assert torch.equal(c.layer.t["state"][s].cpu(), c.state[s])
    s = int(c.slots[3])
    o, S, norm, eff = R.advance(f64(c.state[s]), *(f64(x[3]) for x in (c.q, c.k, c.v, c.g, c.beta)), 128 ** -0.5)
    assert np.abs(f64(c.layer.t["state"][s]) - S).max() <= R.advance_bound(norm, eff, 128, True)


def test_advance_graph_and_stream_give_the_same_bits():
    c = Case([200, 150], 200, 4, 2, 128, 128, BF, seed=17)
    ws = c.layer.advance_workspace(200, 2)
    start = c.layer.t["state"].clone()
    c.run(workspace=ws)
    torch.cuda.synchronize()
    state, out = c.layer.t["state"].clone(), c.out.clone()
    lens, fresh = i32(c.lens), i32(c.fresh)
    args = (c.q, c.k, c.v, c.g, c.beta, c.out, lens, fresh, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.layer.t["state"].copy_(start)
    side.wait_stream(torch.cuda.current_stream())
    c.layer.advance(*args, stream=side)
    side.synchronize()
    assert torch.equal(c.layer.t["state"], state) and torch.equal(c.out, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.layer.advance(*args)
    for _ in range(2):
        c.layer.t["state"].copy_(start)
        c.out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.layer.t["state"], state) and torch.equal(c.out, out)


# ------------------------------------------------------------------ convolution
@pytest.mark.parametrize("din,dout", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("W,cap,D,T,lens,fresh,silu,bias", [
    (4, 20, 264, 70, [70, 1, 0, 2, 33], [0, 1, 1, 0, 0], True, True),
    (4, 3, 8, 9, [9, 2, 0], [0, 0, 0], False, True),
    (3, 7, 520, 65, [65, 1], [1, 1], True, False),
    (2, 1, 16, 1, [1, 0], [0, 1], False, True),
    (1, 1, 24, 130, [129, 8], [0, 1], True, True),
    (4, 8, 6144, 1, [1, 0, 1], [0, 0, 1], True, True),       # a cluster's CTAs beside one another
    (4, 3, 2056, 16, [16, 2, 15], [0, 1, 0], True, False),
    (3, 4, 1032, 129, [129, 1, 64], [1, 0, 0], True, True),  # two CTAs of channels, more runs than a cluster has
])
def test_conv_advance_matches_the_formula(W, cap, D, T, lens, fresh, silu, bias, din, dout):
    import speculative_decode_recurrent_gb300 as lib
    g = torch.Generator().manual_seed(21)
    B = len(lens)
    code = {BF: lib.DTYPE_BF16, F32: lib.DTYPE_F32}
    # (ConvLayer's own T only serves verify)
    dims = lib.ConvDims(B=B, D=D, W=W, T=1, cap=cap, n_slot=B + 1, in_dtype=code[din], out_dtype=code[dout],
                        act=lib.CONV_ACT_SILU if silu else lib.CONV_ACT_NONE)
    slots = torch.randperm(B + 1, generator=g)[:B].to(torch.int32)
    ring = torch.randn(B + 1, cap, D, generator=g).to(din)
    pos = torch.randint(0, cap, (B + 1,), generator=g, dtype=torch.int32)
    x = torch.randn(B, T, D, generator=g)
    for b, n in enumerate(lens):
        x[b, n:] = float("nan")
        if fresh[b]:
            ring[int(slots[b])] = float("nan")
    x = x.to(din).cuda()
    init = dict(ring=ring, pos=pos, state_idx=slots, weight=torch.randn(D, W, generator=g),
                bias=0.3 * torch.randn(D, generator=g) if bias else None)
    layer = lib.ConvLayer(dims, init)
    y = torch.full((B, T, D), 7.0, dtype=dout, device="cuda")
    layer.advance(x, y, chunk_len=i32(lens), fresh=i32(fresh))
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    got_ring, got_pos, want = f64(layer.t["ring"]), layer.t["pos"].cpu(), f64(ring)
    for b, n in enumerate(lens):
        s, p = int(slots[b]), int(pos[int(slots[b])])
        win = np.array([np.zeros(D) if fresh[b] else f64(ring[s, (p - j) % cap]) for j in range(W - 1, 0, -1)]).reshape(W - 1, D)
        ref, last, mag = R.conv(win, f64(x[b, :n]), f64(init["weight"]), f64(init["bias"]) if bias else np.zeros(D), silu)
        # W + 1 roundings of the sum, two fast functions of 2^-21 each, then the output's own
        tol = 2.0 ** -20 * mag + 1e-7 + (2.0 ** -8 * np.abs(ref) if dout == BF else 0)
        assert (np.abs(f64(y[b, :n]) - ref) <= 1.01 * tol).all()
        assert (f64(y[b, n:]) == 0).all()
        assert int(got_pos[s]) == (p + n) % cap
        for j in range(1, W):
            want[s, (p + n - j) % cap] = last[W - 1 - j]
    assert np.array_equal(got_ring, want, equal_nan=True)


def test_conv_advance_then_verify_is_one_sequence():
    import speculative_decode_recurrent_gb300 as lib
    g = torch.Generator().manual_seed(22)
    D, W, n, T = 64, 4, 50, 5
    dims = lib.ConvDims(B=1, D=D, W=W, T=T, cap=11, n_slot=1, in_dtype=lib.DTYPE_F32, out_dtype=lib.DTYPE_F32,
                        act=lib.CONV_ACT_NONE)
    init = dict(ring=torch.full((1, 11, D), float("nan")), pos=i32([4]), state_idx=None, weight=torch.randn(D, W, generator=g))
    layer = lib.ConvLayer(dims, init)
    x = torch.randn(1, n + T, D, generator=g).cuda()
    y = torch.empty_like(x)
    a, b = torch.empty(1, n, D, device="cuda"), torch.empty(1, T, D, device="cuda")
    layer.advance(x[:, :n].contiguous(), a, fresh=i32([1]))
    layer.verify(x[:, n:].contiguous(), b)
    y = np.concatenate([f64(a[0]), f64(b[0])])
    ref, _, mag = R.conv(np.zeros((W - 1, D)), f64(x[0]), f64(init["weight"]), np.zeros(D), False)
    assert (np.abs(y - ref) <= 2.0 ** -20 * mag).all() and int(layer.status.item()) == 0


def test_conv_advance_bad_sequences_are_skipped():
    import speculative_decode_recurrent_gb300 as lib
    dims = lib.ConvDims(B=3, D=16, W=2, T=1, cap=4, n_slot=3, in_dtype=lib.DTYPE_F32, out_dtype=lib.DTYPE_F32, act=0)
    init = dict(ring=torch.ones(3, 4, 16), pos=i32([1, 9, 2]), state_idx=i32([0, 1, -1]), weight=torch.ones(16, 2))
    layer = lib.ConvLayer(dims, init)
    y = torch.full((3, 6, 16), 7.0, device="cuda")
    layer.advance(torch.ones(3, 6, 16, device="cuda"), y, chunk_len=i32([7, 6, 6]))
    torch.cuda.synchronize()
    assert int(layer.status.item()) == lib.STATUS_BAD_SLOT | lib.STATUS_BAD_LEN
    assert (y == 7).all() and (layer.t["ring"] == 1).all() and layer.t["pos"].tolist() == [1, 9, 2]


def test_advance_expired_wait_writes_nothing():
    """The tensor-core kernels' exit at their first bounded wait, with nothing issued; the layer is sound afterwards."""
    import speculative_decode_recurrent_gb300 as lib
    c = Case([150, 90], 150, 2, 2, 128, 128, BF, seed=18)
    c.layer.d.flags = lib.FLAG_TEST_EXPIRE
    c.run()
    torch.cuda.synchronize()
    assert int(c.layer.status.item()) == lib.STATUS_TIMEOUT
    assert torch.equal(c.layer.t["state"].cpu(), c.state)
    c.layer.status.zero_()
    c.layer.d.flags = 0
    c.run()
    c.check(True)


@pytest.mark.parametrize("B,H,dk,dv", [(1, 16, 128, 128), (2, 4, 64, 64), (8, 16, 128, 128), (1, 64, 128, 64), (40, 40, 64, 128)])
def test_a_workspace_is_enough_for_fewer_tokens(B, H, dk, dv):
    import speculative_decode_recurrent_gb300 as lib
    need = [lib.gdn_replay_advance_workspace(lib.AdvanceDims(B=B, T=T, H=H, Hk=H, dk=dk, dv=dv, n_slot=B, in_dtype=lib.DTYPE_BF16, scale=1.0,
                                                             q_stride=H * dk, k_stride=H * dk, v_stride=H * dv))
            for T in list(range(1, 3000, 37)) + [4096, 8192, 10000, 30000, 100000]]
    assert all(a <= b for a, b in zip(need, need[1:])) and need[-1] <= 768 << 20


@pytest.mark.parametrize("lens,T,H,dv", [([2500], 2500, 2, 128), ([1500, 700, 1400], 1500, 14, 128), ([40, 1, 64], 70, 3, 64)])
def test_advance_stays_in_its_workspace(lens, T, H, dv):
    c = Case(lens, T, H, H, 128, dv, BF, seed=23)
    n = c.layer.advance_workspace(T, H).numel()
    room = torch.full((n + 8192,), 171, dtype=torch.uint8, device="cuda")
    c.run(workspace=room[4096:4096 + n])
    c.check(True)
    assert (room[:4096] == 171).all() and (room[4096 + n:] == 171).all()
    with pytest.raises(Exception, match="-2|dims|DIMS|workspace"):
        c.run(workspace=room[4096:4096 + n - 16])


def test_calls_on_two_streams_at_once():
    """Prompts of several launches on two streams, each with its own workspace: the bits of one after the other."""
    cases = [Case([2100, 1900], 2100, 3, 3, 128, 128, BF, seed=25), Case(ragged(9, 1100, 26), 1100, 8, 8, 128, 128, BF, seed=26)]
    ws = [c.layer.advance_workspace(c.T, c.Hk) for c in cases]
    want = []
    for c, w in zip(cases, ws):
        c.run(workspace=w)
        torch.cuda.synchronize()
        want.append((c.out.clone(), c.layer.t["state"].clone()))
    lens, fresh = [i32(c.lens) for c in cases], [i32(c.fresh) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    start = [c.state.cuda() for c in cases]
    for _ in range(5):
        for c, s in zip(cases, start):
            c.layer.t["state"].copy_(s)
            c.out.fill_(3)
        torch.cuda.synchronize()
        for c, w, n, f, stream in zip(cases, ws, lens, fresh, streams):
            c.layer.advance(c.q, c.k, c.v, c.g, c.beta, c.out, chunk_len=n, fresh=f, workspace=w, stream=stream)
        torch.cuda.synchronize()
        for c, (out, state) in zip(cases, want):
            assert torch.equal(c.out, out) and torch.equal(c.layer.t["state"], state) and int(c.layer.status.item()) == 0
