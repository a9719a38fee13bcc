"""Global gradient norm and clipping against sums in 64 bits.

Tolerances: squares are summed in fp32 over at most 128 elements (two chains of
64), so a sum is off by at most 64 * 2^-24 of itself and its root by half of that;
the norm is rounded to fp32 once more.  A clipped fp32 element adds the
factor's and the product's roundings; a bf16 one rounds to 2^-9 of itself, and
the factor's error can move it across one rounding boundary (2^-8)."""
import math

import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"
NORM_TOL = 32 * 2.0 ** -24 + 2.0 ** -23
F32_TOL = NORM_TOL + 4 * 2.0 ** -24
BF16_TOL = 2.0 ** -8 + F32_TOL


def grads(shapes, seed, std=1e-3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(s, generator=g, device=DEV) * std).to(dt) for s, dt in shapes]


def norm64(G):
    return math.sqrt(sum(float(t.double().pow(2).sum()) for t in G))


B, F = torch.bfloat16, torch.float32
LISTS = {
    "one_element": [((1,), F)],
    "odd": [((7,), B), ((13, 3), F), ((1001,), B), ((16385,), F)],
    "tile_edges": [((16384,), B), ((8192,), F), ((16383,), B), ((8193,), F), ((32768 + 5,), B)],
    "empty_among": [((0,), F), ((5,), B), ((0, 4), B), ((129,), F)],
    "mixed": [((64, 256), F), ((2048, 640), B), ((6144,), F), ((300, 700), B)],
    "many": [((33 + i % 5, 17), F if i % 3 else B) for i in range(700)],
}


@pytest.mark.parametrize("name", list(LISTS))
def test_norm_and_clip_match_64_bits(name):
    G = grads(LISTS[name], 3)
    want = norm64(G)
    got = mg.muon_grad_norm(G)
    assert got.shape == () and got.dtype == torch.float32
    assert abs(float(got) - want) <= NORM_TOL * want
    for max_norm in (0.25 * want, 4 * want):
        out = [torch.full_like(t, 7.0) for t in G]
        keep = [t.clone() for t in G]
        n = mg.muon_grad_clip(G, max_norm, out=out)
        assert torch.equal(n, got)                       # the same partial sums in the same order
        assert all(torch.equal(a, b) for a, b in zip(G, keep))
        by = min(1.0, max_norm / (want + 1e-6))
        for a, b in zip(out, G):
            tol = BF16_TOL if a.dtype == B else F32_TOL
            ref = b.double() * by
            assert bool(((a.double() - ref).abs() <= tol * ref.abs() + 1e-44).all())
        n = mg.muon_grad_clip(G, max_norm)               # in place
        assert all(torch.equal(a, b) for a, b in zip(G, out))
        G = keep


def test_range_of_fp32_is_kept():
    for v in (3e38, 1e25, 1e-30, 1e-40):
        G = [torch.full((5000,), v, device=DEV), torch.zeros(9000, dtype=B, device=DEV)]
        want = norm64(G)
        got = float(mg.muon_grad_norm(G))
        if want > 3.4028235e38:
            assert got == math.inf
        else:
            assert abs(got - want) <= NORM_TOL * want + 2e-45
    # unaligned views take the other path
    for v in (1e25, 1e-30):
        x = torch.full((5001,), v, device=DEV)[1:]
        want = norm64([x])
        assert abs(float(mg.muon_grad_norm([x])) - want) <= NORM_TOL * want


def test_nothing_zero_and_not_finite():
    assert float(mg.muon_grad_norm([])) == 0.0
    z = [torch.zeros(100, device=DEV)]
    assert float(mg.muon_grad_clip(z, 1.0)) == 0.0 and float(z[0].abs().max()) == 0.0
    for bad in (math.inf, -math.inf, math.nan):
        for dt in (F, B):
            x = torch.ones(40000, device=DEV, dtype=dt)
            x[12345] = bad
            n = float(mg.muon_grad_norm([torch.ones(3, device=DEV), x]))
            assert math.isnan(n) if math.isnan(bad) else n == math.inf
            y = x.clone()
            mg.muon_grad_clip([y], 1.0)
            assert math.isnan(float(y[12345]))           # inf * 0 and NaN * anything
            assert math.isnan(float(y[0])) if math.isnan(bad) else float(y[0]) == 0.0


@pytest.mark.parametrize("shift", [1, 2, 3, 4, 7, 8])
def test_views_at_any_element(shift):
    for dt in (F, B):
        base = grads([((40011,), dt)], shift)[0]
        x = base[shift:]
        want = norm64([x])
        assert abs(float(mg.muon_grad_norm([x])) - want) <= NORM_TOL * want
        first = base[:shift].clone()
        mg.muon_grad_clip([x], 0.5 * want)
        assert torch.equal(base[:shift], first)
        assert abs(norm64([x]) - 0.5 * want) <= 2e-3 * want


def test_more_squares_than_fp32_counts():
    x = torch.full((1 << 28,), 1e-3, device=DEV, dtype=B)
    want = norm64([x[:1024]]) * math.sqrt(x.numel() / 1024)
    assert abs(float(mg.muon_grad_norm([x])) - want) <= NORM_TOL * want


def test_same_bits_on_every_call_and_stream():
    G = grads([((2048, 3000), B), ((777,), F)], 9)
    first = mg.muon_grad_norm(G)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        other = mg.muon_grad_norm(G, stream=s)
        s.synchronize()
        assert torch.equal(first, other)


def test_capture_in_a_graph():
    G = grads([((512, 512), B), ((100,), F)], 11)
    out = [torch.empty_like(t) for t in G]
    mg.muon_grad_clip(G, 0.1, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = mg.muon_grad_clip(G, 0.1, out=out)
    for t in G:
        t.mul_(3.0)
    graph.replay()
    want = norm64(G)
    assert abs(float(n) - want) <= NORM_TOL * want
    assert abs(norm64(out) - 0.1) <= 1e-3


def test_refusals():
    x = torch.ones(8, device=DEV)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mg.muon_grad_norm([torch.ones(8)])
    with pytest.raises(ValueError, match="contiguous"):
        mg.muon_grad_norm([torch.ones(8, 8, device=DEV).t()[:, :3]])
    with pytest.raises(ValueError, match="CUDA tensor"):
        mg.muon_grad_norm([torch.ones(8, device=DEV, dtype=torch.float16)])
    with pytest.raises(ValueError, match="one tensor for each"):
        mg.muon_grad_clip([x], 1.0, out=[])
    with pytest.raises(ValueError, match="dtype and number"):
        mg.muon_grad_clip([x], 1.0, out=[torch.ones(7, device=DEV)])
    for bad in (-1.0, math.nan, math.inf):
        with pytest.raises(mg.MuonError, match="max_norm"):
            mg.muon_grad_clip([x], bad)
    assert float(x.sum()) == 8.0
