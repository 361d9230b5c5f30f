"""Drafters within a few last places of the target: after two rejections what is left of a token's probability is what
p and c q differ in past 24 bits."""
from fractions import Fraction as F

import pytest
import torch

from test_gpu_draft import run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def draw(p, q, u):
    """The token drawn from max(r - m q, 0), r = max(p - q, 0), and how near the draw came to a border (relative), exactly."""
    p, q = ([F(x) for x in y.tolist()] for y in (p, q))
    r = [max(a - b, F(0)) for a, b in zip(p, q)]
    m = sum(r)
    r = [max(a - m * b, F(0)) for a, b in zip(r, q)]
    goal, acc, hit, near = F(u) * sum(r), F(0), None, F(1)
    for i, x in enumerate(r):
        acc += x
        if x:
            near = min(near, abs(acc - goal) / sum(r))
        if hit is None and acc > goal:
            hit = i
    return hit, float(near)


@pytest.mark.parametrize("bits", [14, 17, 20])
def test_second_rejections_of_a_drafter_near_the_target(bits):
    B, V = 1000, 8
    g = torch.Generator().manual_seed(5)
    p = torch.softmax(1.5 * torch.randn(B, V, generator=g, dtype=torch.float64), -1).float()
    q = p.double() * (1 + 2.0 ** -bits * torch.randn(B, V, generator=g, dtype=torch.float64))
    q = (q / q.sum(-1, keepdim=True) * p.double().sum(-1, keepdim=True)).float()
    u = torch.full((B, 3), 1 - 2.0 ** -24)
    u[:, 0] = torch.rand(B, generator=g)
    over = q > p                                              # such a child is rejected for u nearly 1, a second one too
    use = [b for b in range(B) if over[b].sum() >= 2]
    tokens = torch.zeros(B, 3, dtype=torch.int32)
    for b in use:
        tokens[b, 1:] = over[b].nonzero()[:2, 0]
    p3, q3 = (x[:, None].expand(B, 3, V).contiguous() for x in (p, q))
    parent = torch.tensor([[-1, 0, 0]], dtype=torch.int32).expand(B, 3).contiguous()
    acc, nxt, path, status = run(tokens, parent, p3, q3, u, [3] * B, True)
    assert status == 0
    decided = 0
    for b in use:
        want, near = draw(p[b], q[b], u[b, 0].item())
        if want is not None and near > 0.05:                  # (masses down to 2^-40 of p in terms of 2^-48 of it)
            decided += 1
            assert acc[b] == 1 and path[b] == [0, -1, -1] and nxt[b] == want, (b, want, nxt[b])
    assert decided > 700


def test_an_infinite_probability_after_two_rejections():
    import speculative_decode_recurrent_gb300 as lib
    p = torch.tensor([0.1, 0.2, 0.7, float("inf"), float("nan"), 0.0]).expand(1, 3, 6).contiguous()
    q = torch.tensor([0.5, 0.4, 0.1, 0.0, 0.0, 0.0]).expand(1, 3, 6).contiguous()
    tokens, parent = torch.tensor([[5, 0, 1]], dtype=torch.int32), torch.tensor([[-1, 0, 0]], dtype=torch.int32)
    acc, nxt, _, status = run(tokens, parent, p, q, torch.full((1, 3), 0.9), [3], True)
    assert acc == [1] and nxt == [-1] and status == lib.STATUS_BAD_PROB
    p[0, :, 3] = 0.0                                          # NaN counts as 0
    acc, nxt, _, status = run(tokens, parent, p, q, torch.full((1, 3), 0.9), [3], True)
    assert acc == [1] and nxt == [2] and status == 0
