"""The routing's gradient where sigmoid scores are near 1, against 64 bits."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 64 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sigmoid_gradient_of_saturated_scores(dtype):
    """s (1 - s) keeps its relative accuracy where s is near 1: 1 - s is the score of -x.
    An exponential, a sum, a division and four products of relative error 2^-23 or less
    each: within TOL of itself."""
    x = np.repeat(np.array([[-30.0, -5.0, 0.0, 5.0, 10.0, 12.0, 15.0, 17.0, 20.0, 30.0, 40.0, 80.0]]), 3, 0)
    k = x.shape[1]
    d = np.array([[1.0], [-2.0], [0.125]]) * np.ones((1, k))
    idx = np.repeat(np.arange(k, dtype=np.int32)[None], 3, 0)
    ref = d * 2.5 / (1 + np.exp(-x)) / (1 + np.exp(x))
    got = mg.muon_route_backward(torch.tensor(d, device=DEV, dtype=torch.float32), torch.tensor(x, device=DEV, dtype=dtype),
                                 torch.tensor(idx, device=DEV), score="sigmoid", renormalize=False, scale=2.5)
    out_tol = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= (TOL + out_tol) * np.abs(ref))
    # renormalised: w / scale in the place of s, and u = d - sum d w / scale is exact for equal w
    x = np.array([[20.0, 20.0], [40.0, 40.0]])
    d = np.array([[3.0, 1.0], [1.0, 3.0]])
    got = mg.muon_route_backward(torch.tensor(d, device=DEV, dtype=torch.float32), torch.tensor(x, device=DEV, dtype=dtype),
                                 torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device=DEV), score="sigmoid")
    ref = 0.5 * (d - 2.0) / (1 + np.exp(x))
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= (TOL + out_tol) * np.abs(ref))
