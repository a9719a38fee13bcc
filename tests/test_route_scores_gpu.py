"""Accuracy of single scores over the whole range in which they are normal fp32 numbers.

An exponential is one ex2 (2^-22) and two roundings: 6 * 2^-24.  A sigmoid adds a sum
and a division (2 ulp): 11 * 2^-24.  A softmax score of two experts adds a sum, a
reciprocal and a product: 9 * 2^-24."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 12 * 2.0 ** -24


def spread(lo, hi, n, seed):
    rng = np.random.RandomState(seed)
    even = np.linspace(lo, hi, n)
    small = np.sign(rng.uniform(lo, hi, n)) * 10.0 ** rng.uniform(-8, 0, n)      # of every size near zero
    return np.concatenate([even, rng.uniform(lo, hi, n), small[(small >= lo) & (small <= hi)]]).astype(np.float32)


def test_sigmoid_scores():
    x = spread(-87.0, 87.0, 100000, 1)
    w, _, _ = mg.muon_route(torch.tensor(x[:, None], device=DEV), 1, score="sigmoid", renormalize=False)
    ref = 1.0 / (1.0 + np.exp(-x.astype(np.float64)))
    assert np.all(np.abs(w.cpu().numpy()[:, 0] - ref) <= TOL * ref)


@pytest.mark.parametrize("tokens", [1000, 200000])
def test_softmax_scores_of_two_experts(tokens):
    d = -np.abs(spread(-86.0, 0.0, tokens // 2, 2))
    x = np.stack([np.zeros_like(d), d], 1)
    w, idx, _ = mg.muon_route(torch.tensor(x, device=DEV), 2, renormalize=False)
    e = np.exp(d.astype(np.float64))
    ref = np.stack([1.0 / (1.0 + e), e / (1.0 + e)], 1)
    ref = np.take_along_axis(ref, idx.cpu().numpy(), 1)
    assert np.all(np.abs(w.cpu().numpy() - ref) <= TOL * ref)
