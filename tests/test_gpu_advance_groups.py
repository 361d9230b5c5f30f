"""gdn_replay_advance in more than one launch: where its workspace holds only some of the sequences or of their chunks at a time (groups of
sequences, launches cut short, both), and where the chunks' operators are made beside the walk; tokens in every launch."""
import numpy as np
import pytest
import torch

import advance_ref as R
from advance_plan import plan

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def reference(S, q, k, v, g, beta, lens, scale):
    """advance_ref.advance for all sequences at once, on the GPU in 64 bits: out, states, and the bound's norm and eff."""
    q, k, v, g, beta, S = (x.double() for x in (q, k, v, g, beta, S))
    rep = v.shape[2] // k.shape[2]
    q, k = (x.repeat_interleave(rep, 2) for x in (q, k))
    out, norm, e, eff = torch.zeros_like(v), S.square().sum(-1).amax(), torch.zeros_like(g[:, 0]), 1.0
    for t in range(max(lens)):
        on = [b for b, n in enumerate(lens) if n > t]
        kt, a = k[on, t], g[on, t].exp()
        X = a[..., None, None] * S[on]
        w = beta[on, t][..., None] * (v[on, t] - (X @ kt[..., None])[..., 0])
        X = X + w[..., None] * kt[:, :, None]
        out[on, t] = (X @ q[on, t][..., None])[..., 0] * scale
        S[on] = X
        norm = torch.maximum(norm, X.square().sum(-1).amax())
        e[on] = a * e[on] + 1
        eff = max(eff, e.max().item())
    live = torch.arange(v.shape[1], device="cuda") < i32(lens)[:, None]
    return out, S, max(norm.sqrt().item(), v[live].abs().max().item()), eff


# (what the shape is there for: groups of sequences, launches cut short; neither: several launches beside one another)
@pytest.mark.parametrize("B,T,H,Hk,dk,dv,groups,cut", [
    (1, 8192, 16, 16, 128, 128, False, False),       # three launches, the last by slices of 16
    (1, 1500, 30, 15, 64, 64, False, False),
    (2, 1500, 16, 16, 128, 64, False, False),
    (90, 70, 64, 16, 128, 128, True, True),          # heads walked whole, a last group of six sequences, a chunk a launch
    (360, 64, 16, 16, 128, 128, True, False),        # a group of 338 and one of 22
    (350, 60, 32, 32, 64, 64, True, False),          # slices
    (8, 1400, 64, 64, 128, 128, False, True),        # three launches of up to ten chunks
    (3, 3000, 96, 96, 128, 64, False, True),         # by slices, three launches over two workspaces
    (4, 900, 160, 160, 64, 128, False, True),
])
def test_advance_in_more_than_one_launch(B, T, H, Hk, dk, dv, groups, cut):
    import speculative_decode_recurrent_gb300 as lib
    p = plan(B, T, H, dk, dv, torch.cuda.get_device_properties(0).multi_processor_count)
    assert (p["seqs"] < B) == groups and (p["most"] < p["all"]) == cut and (groups or len(p["sizes"]) > 1), p
    gen = torch.Generator(device="cuda").manual_seed(B + T)
    unit = torch.nn.functional.normalize

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    lens = [0] * B
    for b in range(B):                               # few long sequences where T is long, ragged ones elsewhere
        lens[b] = T - (b * 37) % T if T < 100 or b < 3 else (b * 61) % 70
    lens[0], lens[B - 1] = T, min(T, 65)             # tokens in every launch, the last group's among them
    q, k = (unit(randn(B, T, Hk, dk), dim=-1).to(BF) for _ in range(2))
    v = randn(B, T, H, dv).to(BF)
    g, beta = -0.2 * torch.rand(B, T, H, generator=gen, device="cuda"), torch.rand(B, T, H, generator=gen, device="cuda")
    for b, n in enumerate(lens):
        for x in (q, k, v, g, beta):
            x[b, n:] = float("nan")
    state = 0.3 * randn(B + 1, H, dv, dk)
    slots = torch.randperm(B + 1, generator=gen, device="cuda")[:B]
    fresh = [int(b % 5 == 2) for b in range(B)]
    dims = lib.Dims(B=B, H=H, dk=dk, dv=dv, T=1, cap=2, threshold=1, n_slot=B + 1, in_dtype=lib.DTYPE_BF16, scale=dk ** -0.5)
    init = dict(state=state.clone(), state_idx=slots.to(torch.int32), buf_k=torch.zeros(B + 1, H, 2, dk, dtype=BF),
                buf_v=torch.zeros(B + 1, H, 2, dv, dtype=BF), buf_g=torch.zeros(B + 1, H, 2), buf_beta=torch.zeros(B + 1, H, 2),
                buf_len=torch.zeros(B + 1, dtype=torch.int32))
    layer = lib.ReplayLayer(dims, init)
    n = layer.advance_workspace(T, Hk).numel()
    assert n == p["bytes"]
    room = torch.full((n + 8192,), 171, dtype=torch.uint8, device="cuda")
    out, first = torch.full((B, T, H, dv), 7.0, device="cuda"), None
    for _ in range(2):
        layer.t["state"].copy_(state)
        out.fill_(7)
        layer.advance(q, k, v, g, beta, out, chunk_len=i32(lens), fresh=i32(fresh), workspace=room[4096:4096 + n])
        torch.cuda.synchronize()
        assert int(layer.status.item()) == 0
        if first is None:
            first = out.clone(), layer.t["state"].clone()
    assert torch.equal(out, first[0]) and torch.equal(layer.t["state"], first[1])
    assert (room[:4096] == 171).all() and (room[4096 + n:] == 171).all()
    S0 = state[slots] * (1 - i32(fresh))[:, None, None, None]
    o, S, norm, eff = reference(S0, q, k, v, g, beta, lens, dk ** -0.5)
    tol = R.advance_bound(norm, eff, dk, True)
    assert (layer.t["state"][slots].double() - S).abs().max().item() <= tol
    for b, m in enumerate(lens):
        if m:
            assert (out[b, :m].double() - o[b, :m]).abs().max().item() <= 1.01 * tol * dk ** -0.5, (b, m)
        assert (out[b, m:] == 0).all(), (b, m)
    left = [s for s in range(B + 1) if s not in set(slots.tolist())]
    assert torch.equal(layer.t["state"][left], state[left])


def test_calls_of_several_launches_on_two_streams_at_once():
    """Each with its own workspace: the bits of one after the other."""
    from test_gpu_advance import Case
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cases = [Case([4096], 4096, 16, 16, 128, 128, BF, seed=91), Case([1500], 1500, 30, 30, 64, 64, BF, seed=92)]
    assert all(len(plan(1, c.T, c.H, c.dk, c.dv, sms)["sizes"]) > 1 for c in cases)
    ws = [c.layer.advance_workspace(c.T, c.Hk) for c in cases]
    lens, start, streams, want = [i32(c.lens) for c in cases], [c.state.cuda() for c in cases], [torch.cuda.Stream() for _ in cases], []
    for c, w in zip(cases, ws):
        c.run(workspace=w)
        torch.cuda.synchronize()
        want.append((c.out.clone(), c.layer.t["state"].clone()))
    for _ in range(5):
        for c, s in zip(cases, start):
            c.layer.t["state"].copy_(s)
            c.out.fill_(3)
        torch.cuda.synchronize()
        for c, w, n, stream in zip(cases, ws, lens, streams):
            c.layer.advance(c.q, c.k, c.v, c.g, c.beta, c.out, chunk_len=n, workspace=w, stream=stream)
        torch.cuda.synchronize()
        for c, (out, state) in zip(cases, want):
            assert torch.equal(c.out, out) and torch.equal(c.layer.t["state"], state) and int(c.layer.status.item()) == 0
