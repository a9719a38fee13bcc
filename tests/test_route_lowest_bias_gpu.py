"""Routing in groups where biases are the lowest fp32 number, a usual mask."""
import math

import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("tokens", [3, 20000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_with_a_bias_of_the_lowest_value(score, tokens):
    """A finite bias is a number: a group with one usual expert beside one of the lowest
    bias scores lowest + s, below a group of two usual ones; -inf leaves the one alone."""
    low = torch.finfo(torch.float32).min
    x = torch.zeros(tokens, 12, device=DEV)
    x[:, 0] = 5.0                                        # group 0: one large score, the rest masked
    x[:, 4:6] = -0.5                                     # group 1: two small scores
    bias = torch.zeros(12, device=DEV)
    for mask, first in ((low, 4), (-math.inf, 0)):
        bias[[1, 2, 3, 6, 7, 9, 10, 11]] = mask          # group 2: one middling score
        _, idx, _ = mg.muon_route(x, 2, bias=bias, score=score, groups=3, top_groups=1)
        want = [first, 5 if first == 4 else -1]
        assert bool((idx == torch.tensor(want, dtype=torch.int32, device=DEV)).all())
    # a NaN still orders below every number, the lowest included
    bias[:] = 0.0
    bias[4:8] = low
    bias[8:] = low
    x[:, 4] = math.nan
    if score == "sigmoid":
        _, idx, _ = mg.muon_route(x[:, 4:8].contiguous(), 4, bias=bias[4:8].contiguous(), score=score)
        assert bool((idx == torch.tensor([1, 2, 3, 0], dtype=torch.int32, device=DEV)).all())
