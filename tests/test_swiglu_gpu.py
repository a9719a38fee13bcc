"""The gated activation and its gradient against 64 bits, and against differences."""
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = 2.0 ** -8


def pair(rows, cols, dtype, how, gen, scale=3.0):
    if how == "joined":
        both = (torch.randn(rows, 2 * cols, generator=gen, device="cuda") * scale).to(dtype)
        return both[:, :cols], both[:, cols:]
    if how == "shifted":
        big = (torch.randn(2, rows * cols + 1, generator=gen, device="cuda") * scale).to(dtype)
        return big[0, 1:].view(rows, cols), big[1, :-1].view(rows, cols)
    return tuple((torch.randn(rows, cols, generator=gen, device="cuda") * scale).to(dtype) for _ in range(2))


def s_off(g):
    """Relative error of 1 / (1 + __expf(-g)): the exponential is off by 2 + 1.173 |g| units of 2^-23,
    the sum by half a unit, the quotient by 2."""
    return (2 + 1.173 * g.abs()) * 2 * U + U + 4 * U


def check(out, want, off):
    assert out.isfinite().all() == want.isfinite().all()
    if out.dtype == torch.bfloat16:
        off = off + HALF * (want.abs() + off) + 2.0 ** -134       # half of bf16's smallest step at most
    assert ((out.double() - want).abs() <= off).all()


SIZES = [(1, 1), (1, 7), (3, 5), (8, 2048), (5, 130), (33, 1301), (257, 64), (1000, 520), (2, 40000)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", ["plain", "joined", "shifted"])
def test_forward_and_backward(rows, cols, dtype, how):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    gate, up = pair(rows, cols, dtype, how, gen)
    d, _ = pair(rows, cols, dtype, how, gen, 0.1)
    g, u, dd = gate.double(), up.double(), d.double()
    s = torch.sigmoid(g)
    # below 2^-126 the quotient is 0
    tiny = 2.0 ** -126
    out = mg.muon_swiglu(gate, up)
    want = g * s * u
    check(out, want, want.abs() * (s_off(g) + 2 * U) + (g * u).abs() * tiny)
    d_gate, d_up = mg.muon_swiglu_backward(d, gate, up)
    want = dd * g * s
    check(d_up, want, want.abs() * (s_off(g) + 2 * U) + (dd * g).abs() * tiny)
    f = 1 + g * (1 - s)
    want = dd * u * s * f
    off = (dd * u).abs() * (s * (s_off(g) * f.abs() + g.abs() * (s * s_off(g) + U) + 4 * U * f.abs()) + tiny * (1 + g.abs()))
    check(d_gate, want, off)
    both = mg.muon_swiglu_backward(d, gate, up, joined=True)
    assert torch.equal(both, torch.cat([d_gate, d_up], 1)) and both.is_contiguous()


def test_ends_of_the_range():
    g = torch.tensor([[-1e30, -200.0, -104.0, -88.5, -87.0, -0.0, 0.0, 88.0, 200.0, 1e30, float("inf"), float("nan")]], device="cuda")
    u = torch.ones_like(g)
    out = mg.muon_swiglu(g, u)
    fine = g.isfinite()
    want = g.double() * torch.sigmoid(g.double())
    assert ((out.double() - want).abs() <= want.abs() * (s_off(g.double().clamp(-100, 100)) + 2 * U) +
            g.double().abs().clamp(max=1e3) * 2.0 ** -126)[fine].all()
    assert out[0, -2] == float("inf") and out[0, -1].isnan()
    d_gate, d_up = mg.muon_swiglu_backward(u, g, u)
    assert d_gate[fine].isfinite().all() and d_up[fine].isfinite().all()
    # far out the derivative of gate / (1 + exp(-gate)) is 0 and 1
    assert (d_gate[0, :2] == 0).all() and (d_gate[0, 8:10] == 1).all()


def test_gradient_against_differences():
    gen = torch.Generator(device="cuda").manual_seed(1)
    gate, up = pair(7, 9, torch.float32, "plain", gen)
    d = torch.randn(7, 9, generator=gen, device="cuda")
    d_gate, d_up = mg.muon_swiglu_backward(d, gate, up)
    h = 2.0 ** -6
    # central differences of the fp32 kernel: h^2 / 6 times the third derivative (below 1 for x / (1 + exp(-x)))
    # and the forward's rounding over 2 h
    size = (d * up).abs().double()
    by_gate = (d.double() * (mg.muon_swiglu(gate + h, up).double() - mg.muon_swiglu(gate - h, up).double())) / (2 * h)
    assert ((by_gate - d_gate.double()).abs() <= size * (h * h / 6 + 64 * U * (1 + gate.abs().double()) ** 2 / (2 * h))).all()
    by_up = (d.double() * (mg.muon_swiglu(gate, up + h).double() - mg.muon_swiglu(gate, up - h).double())) / (2 * h)
    assert ((by_up - d_up.double()).abs() <= (d * gate).abs().double() * (up.abs().double() + 1) * 64 * U *
            (1 + gate.abs().double()) / (2 * h)).all()


def test_empty_and_refusals():
    z = torch.zeros(0, 8, device="cuda")
    assert mg.muon_swiglu(z, z).shape == (0, 8)
    a = torch.zeros(4, 8, device="cuda")
    for bad in (a[:3], a.bfloat16(), a.t(), a[0], a.cpu()):
        with pytest.raises(ValueError):
            mg.muon_swiglu(a, bad)
        with pytest.raises(ValueError):
            mg.muon_swiglu_backward(bad, a, a)
    with pytest.raises(ValueError):
        mg.muon_swiglu(a.half(), a.half())
