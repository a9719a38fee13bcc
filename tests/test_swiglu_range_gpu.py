"""The gated activation in fp32 over the whole range of the gate keeps fp32's bits."""
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gates(rows, cols, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.empty(rows, cols, device="cuda").uniform_(-79, 40, generator=gen)
    g[::2] = torch.randn(g[::2].shape, generator=gen, device="cuda") * 4
    up = torch.randn(rows, cols, generator=gen, device="cuda")
    d = torch.randn(rows, cols, generator=gen, device="cuda")
    return g, up + torch.sign(up) * 2.0 ** -6, d + torch.sign(d) * 2.0 ** -6     # products stay above the smallest numbers


def within(out, want, off):
    assert ((out.double() - want).abs() <= off).all(), float(((out.double() - want).abs() / want.abs()).max())


@pytest.mark.parametrize("rows,cols", [(64, 520), (33, 1301), (8, 2048)])
def test_fp32_keeps_its_bits(rows, cols):
    """The exponential is off by one unit in the last place, 2 U of its value, or 2 U e / (1 + e) of 1 + e; the sum, the
    quotient and each product that follows by half a unit, U."""
    g, up, d = gates(rows, cols, rows)
    x, u, y = g.double(), up.double(), d.double()
    s = 1 / (1 + torch.exp(-x))
    more = 1 + 2.0 ** -20                            # products of the errors
    want = x * s * u
    within(mg.muon_swiglu(g, up), want, want.abs() * (2 + 1 + 1 + 1) * U * more)
    d_gate, d_up = mg.muon_swiglu_backward(d, g, up)
    want = y * x * s
    within(d_up, want, want.abs() * (2 + 1 + 1 + 1 + 1) * U * more)
    # s by 4 U; in 1 + x (1 - s) that error times s |x|, the difference's and the sum's roundings; three products
    f = 1 + x * (1 - s)
    off = 4 * U * f.abs() + x.abs() * (4 * U * s + U * (1 - s)) + U * f.abs() + 3 * U * f.abs()
    within(d_gate, y * u * s * f, (y * u * s).abs() * off * more)


def test_fp32_up_to_where_the_exponential_ends():
    """1 + exp(-gate) is finite down to -88.7; from -87.3 on its inverse has 2^-149 as its unit."""
    g = torch.linspace(-88.7, -78, 257, device="cuda")[None]
    up, d = torch.full_like(g, 2.0 ** 126), torch.full_like(g, 2.0 ** 20)
    x = g.double()
    s = 1 / (1 + torch.exp(-x))
    # 4 U for s as above and U for a product; those with powers of two are exact
    want = x * s * 2.0 ** 126
    within(mg.muon_swiglu(g, up), want, want.abs() * 5.01 * U + 2.0 ** (126 - 150))
    d_gate, d_up = mg.muon_swiglu_backward(d, g, torch.full_like(g, 2.0 ** 100))
    want = x * s * 2.0 ** 20
    within(d_up, want, want.abs() * 5.01 * U + (x.abs() + 1) * 2.0 ** (20 - 150))
    want = s * (1 + x * (1 - s)) * 2.0 ** 120
    within(d_gate, want, want.abs() * 6.01 * U + x.abs() * 2.0 ** (120 - 150))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [24, 12])                   # one type's runs of 16 bytes, and elements of views below
def test_ends_of_both_types(dtype, cols):
    """Gates whose exponential is 0 or infinite: the result is gate * up, or zero."""
    ends = [-3e38, -1e30, -200.0, -104.0, 0.0, -0.0, 104.0, 200.0, 1e30, 3e38, float("inf"), float("nan")]
    g = torch.tensor([ends * (cols // 12)] * 3, device="cuda").to(dtype)
    both = torch.empty(3, 2 * cols + 1, dtype=dtype, device="cuda")
    for gate, one in ((g, torch.ones_like(g)), (both[:, :cols].copy_(g), both[:, cols + 1:].fill_(1))):
        out = mg.muon_swiglu(gate, one).float()
        want = torch.where(g.float() > 0, g.float(), torch.zeros_like(out))
        assert torch.equal(out.nan_to_num(7.0, float("inf"), -float("inf")), torch.where(g.isnan(), 7.0, want))
        d_gate, d_up = (t.float() for t in mg.muon_swiglu_backward(one, gate, one))
        fine = g.isfinite() & (g.abs() > 1)
        assert torch.equal(d_gate[fine], (g.float() > 0).float()[fine]) and torch.equal(d_up[fine], want[fine])
        assert (d_gate[(g == 0)] == 0.5).all() and (d_up[g == 0] == 0).all() and d_gate[g.isnan()].isnan().all()
