"""Routing and its gradient against a plain implementation in 64 bits.

Logits lie on a grid of 1/16 (exact in bf16 and fp32; in the tests of groups
shifted by 1/64, so that no two sigmoids add up to 1), so equal values occur
often and unequal choice values differ by more than fp32 can blur; the
reference counts choice values within 1e-9 as equal.
Tolerances: a score is an exponential (2 ulp), a sum of at most 1024 terms in
a tree of 32 chains (at most 37 roundings on one path) and a division; weights
add a sum over top_k and a division: TOL = 64 * 2^-24.  A gradient is
s (d - dot) or w (1 - s) (d - dot): TOL of itself for s or w, and s or w times
the error of d - dot, at most 4 TOL max|d|; with |d - dot| <= 2 max|d| that is
within 8 TOL max|d| s.  bf16 gradients round to 2^-9 (2^-8 where the error
crosses a boundary)."""
import math

import numpy as np
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 64 * 2.0 ** -24


def scores64(x, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    out = np.zeros_like(x)
    for i, r in enumerate(x):
        if np.isneginf(r).all():
            continue
        e = np.exp(r - r.max())
        out[i] = e / e.sum()
    return out


def route64(x, k, bias, score, groups, top_groups, renorm, scale):
    x = x.astype(np.float64)
    t, e = x.shape
    s = scores64(x, score)
    c = s + (0.0 if bias is None else bias.astype(np.float64))
    c[np.isneginf(x)] = -np.inf
    w = np.zeros((t, k))
    idx = np.full((t, k), -1, np.int32)
    gs = e // groups
    for i in range(t):
        row = np.where(np.isfinite(c[i]), np.round(c[i], 9), -np.inf)
        if groups > 1:
            g = []
            for j in range(groups):
                part = np.sort(row[j * gs:(j + 1) * gs])[::-1][:2]
                part = part[part > -np.inf]
                g.append(round(part.sum(), 9) if len(part) else -np.inf)
            order = sorted(range(groups), key=lambda j: (-g[j], j))[:top_groups]
            keep = np.zeros(e, bool)
            for j in order:
                keep[j * gs:(j + 1) * gs] = True
            row = np.where(keep, row, -np.inf)
        order = [j for j in sorted(range(e), key=lambda j: (-row[j], j)) if row[j] > -np.inf][:k]
        idx[i, :len(order)] = order
        v = s[i, order]
        if renorm and len(order):
            if score == "softmax":
                v = np.exp(x[i, order] - x[i, order].max())
            v = v / v.sum() if v.sum() > 0 else v * 0
        w[i, :len(order)] = v * scale
    counts = np.bincount(idx[idx >= 0], minlength=e).astype(np.int32)
    return w, idx, counts


def grad64(d, x, idx, score, renorm, scale):
    """The formulas, row by row."""
    x = x.astype(np.float64)
    s = scores64(x, score)
    out = np.zeros_like(x)
    for i in range(x.shape[0]):
        at = idx[i][idx[i] >= 0]
        if len(at) == 0:
            continue
        dk = d[i][idx[i] >= 0].astype(np.float64) * scale
        sk = s[i, at]
        if score == "softmax" and renorm:
            p = np.exp(x[i, at] - x[i, at].max())
            p /= p.sum()
            out[i, at] = p * (dk - (dk * p).sum())
            continue
        if renorm:
            total = sk.sum()
            dk = (dk - (dk * sk).sum() / total) / total if total > 0 else dk * 0
        ds = np.zeros(x.shape[1])
        ds[at] = dk
        out[i] = ds * s[i] * (1 - s[i]) if score == "sigmoid" else s[i] * (ds - (ds * s[i]).sum())
    return out


def grid_logits(t, e, seed, dtype, spread=2.0):
    rng = np.random.RandomState(seed)
    x = np.round(rng.standard_normal((t, e)) * spread * 16) / 16
    return x, torch.tensor(x, device=DEV, dtype=dtype)


def check(x, xt, k, bias, score="softmax", groups=1, top_groups=1, renorm=True, scale=1.0, seed=0):
    bt = None if bias is None else torch.tensor(bias, device=DEV, dtype=torch.float32)
    w, idx, counts = mg.muon_route(xt, k, bias=bt, score=score, groups=groups, top_groups=top_groups,
                                   renormalize=renorm, scale=scale)
    w64, i64, c64 = route64(x, k, bias, score, groups, top_groups, renorm, scale)
    assert np.array_equal(idx.cpu().numpy(), i64)
    assert np.array_equal(counts.cpu().numpy(), c64)
    assert np.all(np.abs(w.cpu().numpy() - w64) <= TOL * np.abs(w64) + 1e-37)
    d = np.random.RandomState(seed + 99).standard_normal(i64.shape).astype(np.float32)
    dx = mg.muon_route_backward(torch.tensor(d, device=DEV), xt, idx, score=score, renormalize=renorm, scale=scale)
    assert dx.dtype == xt.dtype and dx.shape == xt.shape
    ref = grad64(d, x, i64, score, renorm, scale)
    top = np.abs(d).max(1, keepdims=True) * scale
    out_tol = 2.0 ** -8 if xt.dtype == torch.bfloat16 else 0.0
    got = dx.float().cpu().numpy().astype(np.float64)
    s = scores64(x, score)
    if renorm:                                           # w / scale in the place of s
        s = np.zeros_like(s)
        rows, cols = np.nonzero(i64 >= 0)
        s[rows, i64[rows, cols]] = w64[rows, cols] / scale
    assert np.all(np.abs(got - ref) <= 8 * TOL * top * s + out_tol * np.abs(ref) + 1e-37)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 384, 8), (3, 7, 2), (70, 33, 5), (129, 100, 6), (257, 384, 8),
                                   (40, 1024, 32), (17, 60, 4), (5, 32, 32), (9, 511, 3)])
def test_sizes(t, e, k, score, dtype):
    x, xt = grid_logits(t, e, t * 1000 + e, dtype)
    for renorm in (True, False):
        check(x, xt, k, None, score, renorm=renorm, scale=1.0 if renorm else 2.5, seed=t)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,top_groups,k", [(384, 8, 4, 8), (384, 4, 1, 8), (208, 8, 3, 8), (96, 3, 2, 5),
                                                   (60, 5, 2, 4), (32, 32, 8, 8), (512, 32, 4, 8), (26, 13, 5, 3),
                                                   (24, 6, 6, 7)])
def test_groups_and_bias(e, groups, top_groups, k, score):
    x, _ = grid_logits(101, e, e + groups, torch.float32)
    x += 1 / 64
    xt = torch.tensor(x, device=DEV, dtype=torch.float32)
    rng = np.random.RandomState(e)
    for bias in (None, np.round(rng.standard_normal(e) * 8) / 64):
        check(x, xt, k, bias, score, groups, top_groups, True, 2.5, seed=groups)


def test_masks_leave_rows_short_or_empty():
    for score in ("softmax", "sigmoid"):
        x, _ = grid_logits(64, 48, 5, torch.float32)
        x[0] = -np.inf                                   # nothing left
        x[1, 1:] = -np.inf                               # one expert left
        x[2, ::2] = -np.inf
        x[3, 12:] = -np.inf                              # one group left
        x[4, :] = -np.inf
        x[4, [5, 13, 40]] = [0.0, 1.0, 1.0]
        xt = torch.tensor(x, device=DEV, dtype=torch.float32)
        for renorm in (True, False):
            check(x, xt, 6, None, score, renorm=renorm)
            check(x, xt, 6, None, score, 4, 2, renorm)
        bias = np.zeros(48)
        bias[7] = -np.inf                                # masked by its bias
        check(x, xt, 6, bias, score, 4, 2)


def test_extreme_logits():
    x = np.zeros((6, 40))
    x[0] = -3e38
    x[1, 3] = 3e38                                       # the others' scores are zero: lowest index first
    x[2] = np.arange(40) * -50.0
    x[3] = 100.0
    x[4] = -200.0
    x[5, ::3] = 90.0
    xt = torch.tensor(x, device=DEV, dtype=torch.float32)
    w, idx, counts = mg.muon_route(xt, 4)
    assert idx[1].tolist() == [3, 0, 1, 2] and idx[3].tolist() == [0, 1, 2, 3] and idx[5].tolist() == [0, 3, 6, 9]
    assert bool(torch.isfinite(w).all()) and float((w.sum(1) - 1).abs().max()) < 1e-6
    assert w[1].tolist() == [1.0, 0.0, 0.0, 0.0]
    dx = mg.muon_route_backward(torch.ones_like(w), xt, idx)
    assert bool(torch.isfinite(dx).all())
    w, idx, _ = mg.muon_route(xt, 4, score="sigmoid")
    assert w[4].tolist() == [0.0] * 4                    # every score underflows: no weight, no NaN
    assert bool(torch.isfinite(mg.muon_route_backward(torch.ones_like(w), xt, idx, score="sigmoid")).all())


def test_nan_reaches_the_weights_and_indices_stay_valid():
    x = torch.randn(5, 64, device=DEV)
    x[2, 7] = math.nan
    x[3] = math.nan
    w, idx, counts = mg.muon_route(x, 8)
    assert bool(torch.isnan(w[2]).all()) and bool(torch.isnan(w[3]).all()) and bool(torch.isfinite(w[[0, 1, 4]]).all())
    assert int(idx.min()) >= 0 and int(idx.max()) < 64 and int(counts.sum()) == 40
    w, idx, _ = mg.muon_route(x, 8, score="sigmoid", groups=4, top_groups=2)
    assert 7 not in idx[2].tolist() and bool(torch.isfinite(w[2]).all()) and bool(torch.isnan(w[3]).all())


@pytest.mark.parametrize("ld,shift", [(104, 0), (101, 0), (128, 4), (128, 3)])
def test_strided_rows(ld, shift):
    for dtype in (torch.float32, torch.bfloat16):
        x, xt = grid_logits(50, 96, ld + shift, dtype)
        base = torch.full((50, ld), 55.0, device=DEV, dtype=dtype)
        view = base[:, shift:shift + 96]
        view.copy_(xt)
        check(x, view, 6, None, "softmax", 3, 2)


def test_gradient_against_differences():
    rng = np.random.RandomState(3)
    x = rng.standard_normal((4, 24))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            w, idx, _ = route64(x, 5, None, score, 1, 1, renorm, 1.5)
            d = rng.standard_normal(idx.shape)

            def f(y):
                s = scores64(y, score)
                v = np.take_along_axis(s, idx, 1)
                if renorm:
                    v = v / v.sum(1, keepdims=True)
                return (v * 1.5 * d).sum()

            got = mg.muon_route_backward(torch.tensor(d, device=DEV, dtype=torch.float32),
                                         torch.tensor(x, device=DEV, dtype=torch.float32),
                                         torch.tensor(idx, device=DEV), score=score, renormalize=renorm, scale=1.5)
            h = 1e-5
            for i in range(4):
                for j in range(24):
                    y = x.copy()
                    y[i, j] += h
                    z = x.copy()
                    z[i, j] -= h
                    num = (f(y) - f(z)) / (2 * h)
                    # 8 TOL max|d| s (see above) is at most 1e-4; fp32 inputs and the
                    # differences (h^2, 1e-16 / h) add less than 1e-6
                    assert abs(float(got[i, j]) - num) <= 1e-4


def test_counts_of_many_tokens_streams_and_graph():
    x = torch.randn(20000, 384, device=DEV)
    w, idx, counts = mg.muon_route(x, 8, score="sigmoid", groups=8, top_groups=4)
    assert torch.equal(counts.long(), torch.bincount(idx.reshape(-1), minlength=384))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w2, i2, c2 = mg.muon_route(x, 8, score="sigmoid", groups=8, top_groups=4, stream=s)
    s.synchronize()
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(counts, c2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w3, i3, c3 = mg.muon_route(x, 8, score="sigmoid", groups=8, top_groups=4)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx, i3) and torch.equal(w, w3) and torch.equal(counts, c3)


def test_no_tokens():
    w, idx, counts = mg.muon_route(torch.empty(0, 16, device=DEV), 2)
    assert w.shape == (0, 2) and counts.tolist() == [0] * 16
    assert mg.muon_route_backward(w, torch.empty(0, 16, device=DEV), idx).shape == (0, 16)


def test_refusals():
    x = torch.randn(4, 16, device=DEV)
    for kw, what in (({"top_k": 0}, "top_k"), ({"top_k": 17}, "top_k"), ({"top_k": 2, "groups": 3}, "groups"),
                     ({"top_k": 2, "groups": 4, "top_groups": 5}, "top_groups"),
                     ({"top_k": 6, "groups": 4, "top_groups": 1}, "below top_k"),
                     ({"top_k": 2, "scale": math.nan}, "scale")):
        with pytest.raises(mg.MuonError, match=what):
            mg.muon_route(x, **kw)
    with pytest.raises(mg.MuonError, match="experts"):
        mg.muon_route(torch.randn(2, 1025, device=DEV), 2)
    with pytest.raises(ValueError, match="score"):
        mg.muon_route(x, 2, score="relu")
    with pytest.raises(ValueError, match="bias"):
        mg.muon_route(x, 2, bias=torch.zeros(15, device=DEV))
    with pytest.raises(ValueError, match="2-D CUDA"):
        mg.muon_route(torch.randn(4, 16), 2)
    with pytest.raises(ValueError, match="rows of logits"):
        mg.muon_route(torch.randn(16, 4, device=DEV).t(), 2)
    w, idx, _ = mg.muon_route(x, 2)
    with pytest.raises(ValueError, match="d_weights"):
        mg.muon_route_backward(w[:3], x, idx)
    with pytest.raises(ValueError, match="chosen"):
        mg.muon_route_backward(w, x, idx.long())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k,groups,top_groups", [(384, 8, 8, 4), (384, 16, 1, 1), (40, 4, 1, 1), (96, 6, 3, 2), (64, 20, 1, 1),
                                                   (12, 12, 1, 1)])
def test_many_tokens_as_few(e, k, groups, top_groups, score):
    """A long call takes tokens in pairs; each comes out as in a short call, next to
    rows of equal values, masked ones and ones that are not numbers."""
    t = 15001
    _, x = grid_logits(t, e, e + k, torch.float32)
    gen = torch.Generator(device=DEV).manual_seed(e)
    kind = torch.randint(0, 12, (t,), generator=gen, device=DEV)
    x[kind == 0] = 0.25                                  # all equal
    x[kind == 1] = -math.inf
    x[kind == 2] = torch.where(torch.rand(x[kind == 2].shape, generator=gen, device=DEV) < 0.8, -math.inf, 1.0)
    x[kind == 3, e // 2] = math.nan
    x[kind == 4] = x[kind == 4].round()                  # many equal
    x[kind == 5] *= 1e36
    bias = torch.round(torch.randn(e, generator=gen, device=DEV) * 8) / 64
    kw = dict(bias=bias, score=score, groups=groups, top_groups=top_groups, scale=2.5)
    for renorm in (True, False):
        w, idx, counts = mg.muon_route(x, k, renormalize=renorm, **kw)
        parts = [mg.muon_route(p, k, renormalize=renorm, **kw) for p in x.split(1000)]
        assert torch.equal(idx, torch.cat([p[1] for p in parts]))
        assert torch.equal(counts, torch.stack([p[2] for p in parts]).sum(0).int())
        few = torch.cat([p[0] for p in parts])
        assert torch.equal(w.isnan(), few.isnan())
        assert bool(((w - few).abs() <= TOL * few.abs() + 1e-37).logical_or(w.isnan()).all())
