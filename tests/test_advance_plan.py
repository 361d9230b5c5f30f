"""The launches that a prompt's chunks come in: they cover it, fit their workspaces and are not many more than those need."""
import itertools

import pytest

from advance_plan import UNIT, plan

BATCHES, TOKENS = (1, 2, 3, 8, 16, 40, 64, 90, 360, 4096), (24, 64, 65, 130, 700, 2048, 4096, 8192, 32768, 1 << 20)


@pytest.mark.parametrize("sms", [132, 148, 152])
@pytest.mark.parametrize("H,dk,dv", [(1, 128, 128), (4, 64, 64), (16, 128, 128), (16, 64, 128), (32, 128, 64), (64, 128, 128), (1024, 128, 128)])
def test_launches_are_few_and_fit(H, dk, dv, sms):
    for B, T in itertools.product(BATCHES, TOKENS):
        if B * T > 1 << 28:
            continue
        p = plan(B, T, H, dk, dv, sms)
        s, where = p["sizes"], (B, T, p)
        assert sum(s) == p["all"] == -(-T // 64) and min(s) >= 1 and max(s) <= p["most"], where
        assert len(s) <= -(-p["all"] // p["most"]) + 6, where
        assert p["bytes"] == UNIT[dk] * H * p["seqs"] * p["room"] <= 768 << 20, where
        # the launches of all groups take the two workspaces in turn
        groups, turn = -(-B // p["seqs"]), 0
        for _ in range(min(groups, 3)):
            for size in s:
                assert size <= (p["room"] - p["first_room"] if turn else p["first_room"]), where
                turn ^= 1


def test_launches_limited_by_the_workspace_stay_large():
    """Every launch but the last takes what the workspace holds, where the walk leaves no SMs for the next chunks' operators."""
    for B, T, H in ((16, 4096, 16), (8, 8192, 16), (2, 1 << 20, 16), (64, 1024, 32)):
        p = plan(B, T, H, 128, 128)
        assert p["most"] < p["all"] and all(x == p["most"] for x in p["sizes"][:-1]), p


def test_launches_of_prompts_that_fit():
    """One launch where the walk fills the SMs, growing ones where it leaves some."""
    assert plan(8, 2048, 16, 128, 128)["sizes"] == [32]
    s = plan(1, 8192, 16, 128, 128)["sizes"]
    assert len(s) == 3 and s[0] < s[1] < s[2]
