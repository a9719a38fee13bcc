"""Softmax routing over the whole range of fp32 logits, against 64 bits.

Rows lie around an offset, on a grid of 1/16 or of the offset's own spacing, so
that every logit and every difference is exact in fp32, and scores that differ do
so by 6 % or more; scores that are equal in fp32 go by index.  TOL as in
test_route_gpu.py: a score is an exponential, a sum in a tree and a division."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 64 * 2.0 ** -24


def rows_around(offset, tokens, experts, seed):
    rng = np.random.RandomState(seed)
    unit = max(1 / 16, float(np.spacing(np.float32(abs(offset)))))
    n = np.round(rng.standard_normal((tokens, experts)) * (2 / unit if unit < 1 else 2))
    return (float(np.float32(offset)) + n * unit).astype(np.float32)


def softmax64(x, k, renorm, scale):
    """(weights, experts) of the definition: scores in 64 bits, equal ones (in fp32) by index."""
    x = x.astype(np.float64)
    e = np.exp(x - x.max(1, keepdims=True))
    s = e / e.sum(1, keepdims=True)
    idx = np.argsort(-s.astype(np.float32), axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, idx, 1)
    if renorm:
        c = np.take_along_axis(x, idx, 1)
        w = np.exp(c - c.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
    return w * scale, idx


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("tokens,experts", [(1, 384), (5, 384), (7, 40), (6000, 384), (12000, 60)])
@pytest.mark.parametrize("offset", [0.0, 64.0, 100.0, 1e3, 1e5, 1e8, 2e9, 1e10, 1e20, 1e30, 3e37])
def test_softmax_of_shifted_rows(offset, tokens, experts, renorm):
    for sign in (1.0, -1.0):
        x = rows_around(sign * offset, tokens, experts, tokens + experts)
        w64, i64 = softmax64(x, 8, renorm, 2.5)
        w, idx, counts = mg.muon_route(torch.tensor(x, device=DEV), 8, renormalize=renorm, scale=2.5)
        assert np.array_equal(idx.cpu().numpy(), i64)
        assert np.array_equal(counts.cpu().numpy(), np.bincount(i64.reshape(-1), minlength=experts))
        assert np.all(np.abs(w.cpu().numpy() - w64) <= TOL * w64 + 1e-37)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("experts", [96, 128])
def test_softmax_of_equal_and_lowest_logits(experts, renorm):
    low = float(np.finfo(np.float32).min)
    x = np.zeros((6, experts), np.float32)
    x[0] = 1e12
    x[1] = low
    x[2] = low
    x[2, [5, 50, 90]] = [1.0, 3.0, 2.0]                  # three experts left by a finite mask
    x[3] = -low
    x[4, ::2] = 1e12
    x[5, 7] = 1e29
    w64, i64 = softmax64(x, 6, renorm, 1.0)
    w, idx, _ = mg.muon_route(torch.tensor(x, device=DEV), 6, renormalize=renorm)
    assert np.array_equal(idx.cpu().numpy(), i64)
    assert np.all(np.abs(w.cpu().numpy() - w64) <= TOL * w64 + 1e-37)
    bf = torch.tensor(x[[0, 4]], device=DEV).to(torch.bfloat16)
    w64, i64 = softmax64(bf.float().cpu().numpy(), 6, renorm, 1.0)
    w, idx, _ = mg.muon_route(bf, 6, renormalize=renorm)
    assert np.array_equal(idx.cpu().numpy(), i64)
    assert np.all(np.abs(w.cpu().numpy() - w64) <= TOL * w64 + 1e-37)


def test_softmax_in_groups_of_shifted_rows():
    """The group step on large logits: the row less its offset routes alike."""
    for offset in (1e3, 1e5, 1e6):
        x = rows_around(offset, 40, 96, 9)
        y = torch.tensor(x - np.float32(offset), device=DEV)
        kw = dict(groups=4, top_groups=2, renormalize=False)
        w, idx, _ = mg.muon_route(torch.tensor(x, device=DEV), 6, **kw)
        w0, idx0, _ = mg.muon_route(y, 6, **kw)
        assert torch.equal(idx, idx0)
        assert bool(((w - w0).abs() <= TOL * w0).all())
