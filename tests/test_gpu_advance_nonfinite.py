"""Infinite and NaN inputs of gdn_replay_advance: every output before the token that has them, every other head and (for values) every
other column keeps its bits; what the recurrence takes them into is not finite."""
import pytest
import torch

from advance_plan import plan
from test_gpu_advance import BF, F32, Case

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


# lengths, T, H, Hk, dk, dv
SHAPES = {
    "slices of 16": ([200, 70], 200, 2, 1, 128, 128, BF),
    "slices of 32": ([330, 140, 64], 330, 13, 13, 128, 128, BF),
    "slices of 64 rows": ([150] * 9, 150, 5, 5, 64, 64, BF),
    "heads": ([200, 150] * 5, 200, 8, 4, 128, 128, BF),
    "heads of 64 key dims": ([140] * 20, 140, 4, 4, 64, 128, BF),
    "two launches": ([1500], 1500, 30, 30, 64, 64, BF),
    "token by token": ([19, 17], 19, 4, 2, 128, 64, BF),
    "fp32": ([90, 75], 90, 3, 3, 64, 64, F32),
}


@pytest.mark.parametrize("at", ["first", "middle", "border", "last"])
@pytest.mark.parametrize("name", SHAPES)
def test_bad_inputs_go_forward_alone(name, at):
    lens, T, H, Hk, dk, dv, dtype = SHAPES[name]
    if name == "two launches":
        assert len(plan(1, T, H, dk, dv, torch.cuda.get_device_properties(0).multi_processor_count)["sizes"]) == 2
    c = Case(lens, T, H, Hk, dk, dv, dtype, seed=31)
    c.run()
    torch.cuda.synchronize()
    out, state, rep = c.out.clone(), c.layer.t["state"].clone(), H // Hk
    B, clean = len(lens), {n: getattr(c, n).clone() for n in ("q", "k", "v", "g", "beta")}
    for i, (what, bad) in enumerate((("v", INF), ("v", NAN), ("k", NAN), ("k", INF), ("q", -INF), ("g", NAN), ("beta", NAN), ("beta", INF), ("state", NAN))):
        b, h = i % B, (2 * i + 1) % H
        n = lens[b]
        t = {"first": 0, "middle": n // 2 + 5, "border": min(64, n - 1), "last": n - 1}[at]
        col = (37 * i) % dv
        for name_, x in clean.items():
            getattr(c, name_).copy_(x)
        c.layer.t["state"].copy_(c.state)
        want_out, want_state = torch.zeros_like(out, dtype=torch.bool), torch.zeros_like(state, dtype=torch.bool)     # not finite
        s = int(c.slots[b])
        heads = [h]
        if what in "qk":
            heads = list(range(h // rep * rep, h // rep * rep + rep))
            getattr(c, what)[b, t, h // rep, (13 * i) % dk] = bad
        elif what == "v":
            c.v[b, t, h, col] = bad
        elif what == "state":
            c.layer.t["state"][s, h, col, 3] = bad
        else:
            getattr(c, what)[b, t, h] = bad
        if what == "q":
            want_out[b, t, heads] = True
        elif what == "v":
            want_out[b, t:n, h, col] = True
            want_state[s, h, col] = True
        elif what == "state":
            want_out[b, :n, h, col] = True
            want_state[s, h, col] = True
        else:
            want_out[b, t:n, heads] = True
            want_state[s, heads] = True
        c.out.fill_(7)
        c.run()
        torch.cuda.synchronize()
        now = c.layer.t["state"]
        assert int(c.layer.status.item()) == 0
        assert torch.equal(c.out[~want_out], out[~want_out]), (what, bad, b, t, h)
        assert torch.equal(now[~want_state], state[~want_state]), (what, bad, b, t, h)
        assert not torch.isfinite(c.out[want_out]).any(), (what, bad, b, t, h)
        assert not torch.isfinite(now[want_state]).any(), (what, bad, b, t, h)


def test_many_bad_tokens_of_one_head():
    """Several columns from several tokens on, beside a head whose first key is bad."""
    c = Case([190], 190, 20, 20, 128, 128, BF, seed=32)
    c.run()
    torch.cuda.synchronize()
    out = c.out.clone()
    c.layer.t["state"].copy_(c.state)
    first = [190] * 128
    for j, (t, col) in enumerate(((150, 3), (20, 3), (70, 4), (70, 5), (63, 6), (64, 7), (189, 127), (0, 126))):
        c.v[0, t, 2, col] = (INF, NAN, -INF)[j % 3]
        first[col] = min(first[col], t)
    c.k[0, 0, 5, 100] = NAN
    c.run()
    torch.cuda.synchronize()
    for col, t in enumerate(first):
        assert torch.equal(c.out[0, :t, 2, col], out[0, :t, 2, col]) and not torch.isfinite(c.out[0, t:, 2, col]).any(), (col, t)
    assert not torch.isfinite(c.out[0, :, 5]).any()
    rest = [h for h in range(20) if h not in (2, 5)]
    assert torch.equal(c.out[:, :, rest], out[:, :, rest])
