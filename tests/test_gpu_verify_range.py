"""The draw where p - q leaves FP32's range: such a weight counts as 0."""
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk

pytestmark = pytest.mark.gpu

DEV = "cuda"


def draw(p, q, u, drafted):
    d = lambda a, t: torch.as_tensor(a, dtype=t, device=DEV)
    target = torch.stack((p, p))[None].to(DEV)
    tokens, accepted = sk.verify_draft(target, q[None, None].to(DEV), d([[drafted]], torch.int32), d([[1.0, u]], torch.float32))
    torch.cuda.synchronize()
    assert accepted.tolist() == [0]
    return tokens[0, 0].item()


@pytest.mark.parametrize("V", [8, 4099])
def test_a_difference_past_the_range_weighs_nothing(V):
    p, q = torch.zeros(V), torch.zeros(V)
    p[1], q[1] = 3e38, -3e38            # the difference is an infinity in FP32
    p[5] = 0.25
    q[0] = 1.0                          # the draft's own token, never accepted
    for u in (0.0, 0.5, 1 - 2**-24):
        assert draw(p, q, u, 0) == 5


def test_no_weight_but_one_past_the_range_draws_from_the_target():
    V = 600
    p, q = torch.zeros(V), torch.zeros(V)
    p[300], q[300] = 3e38, -3e38
    q[0] = 1.0
    assert draw(p, q, 0.5, 0) == 300    # nothing is left of p - q: the target's own row
