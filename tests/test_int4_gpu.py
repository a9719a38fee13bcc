"""Weights of 4 bits: their rounding, and products with them, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = 2.0 ** -8


def codes_of(m):
    """Codes as whole numbers (.., rows, cols up to 128)."""
    c = m.codes.to(torch.int64)
    q = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    return torch.where(q > 7, q - 16, q)


def values(m):
    """What a weight stands for, in 64 bits."""
    return (codes_of(m).double() * m.scale.double().transpose(-1, -2).repeat_interleave(m.block, -1))[..., :m.cols]


@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (16, 128), (5, 129), (2, 70, 300), (64, 1000), (3, 33, 6144)])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rounding(shape, block, dtype):
    gen = torch.Generator(device="cuda").manual_seed(sum(shape) + block)
    w = (torch.randn(shape, generator=gen, device="cuda") * 0.02).to(dtype)
    w.view(-1)[0] = 0
    m = mg.muon_int4_quantize_weight(w, block)
    up = -(-shape[-1] // 128) * 128
    assert m.codes.shape == (*shape[:-1], up // 2) and m.scale.shape == (*shape[:-2], up // block, shape[-2])
    p = torch.nn.functional.pad(w.float(), (0, up - shape[-1])).unflatten(-1, (-1, block))
    scale = (p.abs().amax(-1) / 7.0).to(torch.bfloat16)
    assert torch.equal(m.scale, scale.transpose(-1, -2))
    by = scale.float()[..., None]
    q = torch.where(by > 0, p / by, torch.zeros_like(p)).round().clamp(-7, 7).flatten(-2)
    assert torch.equal(codes_of(m), q.long())
    # half a step, and what the largest loses to a scale that bf16 rounds down: 7 * 2^-8 of a step
    step = m.scale.double().transpose(-1, -2).repeat_interleave(block, -1)[..., :shape[-1]]
    assert ((values(m) - w.double()).abs() <= step * 0.5 * (1 + 1e-6)).all()


def test_rounding_of_odd_values():
    w = torch.zeros(6, 256, device="cuda")
    w[0, 5] = float("nan")
    w[1, 130] = float("inf")
    w[2, 7] = 1e-44                                  # the scale rounds to zero
    w[3, :128] = 3.4e38
    w[4, 64] = -7.0
    m = mg.muon_int4_quantize_weight(w, 64)
    s = m.scale.t()                                  # rows x blocks
    assert s[0, 0].isnan() and (s[0, 1:] == 0).all() and s[1, 2].isnan() and (s[1, :2] == 0).all()
    assert (s[2] == 0).all() and (codes_of(m)[2] == 0).all()
    assert s[3].isfinite().all() and (codes_of(m)[3, :128] == 7).all()
    assert codes_of(m)[4, 64] == -7 and s[4, 1] == 1
    y = mg.muon_int4_linear(torch.ones(1, 256, device="cuda"), m)
    assert y[0, :2].isnan().all() and (y[0, 2] == 0) and y[0, 4] == -7 and y[0, 5] == 0


def weight(shape, block, gen, whole=False):
    n, up = shape[-2], -(-shape[-1] // 128) * 128
    codes = torch.randint(0, 256, (*shape[:-1], up // 2), generator=gen, device="cuda", dtype=torch.uint8)
    keep = torch.arange(up, device="cuda") < shape[-1]
    codes &= (keep[0::2] * 15 + keep[1::2] * 240).to(torch.uint8)
    if whole:
        scale = torch.ones(*shape[:-2], up // block, n, device="cuda")
        scale *= 2.0 ** torch.randint(-1, 2, scale.shape, generator=gen, device="cuda")
    else:
        scale = torch.rand(*shape[:-2], up // block, n, generator=gen, device="cuda") * 0.01 + 1e-3
    return mg.Int4Matrix(codes, scale.to(torch.bfloat16), block, shape[-1])


def expected(x, m, offsets=None):
    """(result, largest rounding error of its sums) in 64 bits."""
    w, parts = values(m), 1 if x.dtype == torch.bfloat16 else 3
    k = m.cols
    # a product of 16 columns adds 16 terms and the sum before, each cut at 2^-23 of the largest at most; blocks of
    # `block` columns take block / 16 of them for each part of x, their sums and the warps' one rounding each; what
    # fp32 has past three parts of 8 bits is below 2^-24 of it
    off = m.block / 16 * parts * 17 * 2 * U + (k / m.block + 10) * U + U
    if offsets is None:
        return x.double() @ w.t(), off * (x.double().abs() @ w.abs().t())
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    e = torch.zeros_like(y)
    bounds = offsets.tolist()
    for g, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        y[lo:hi] = x[lo:hi].double() @ w[g].t()
        e[lo:hi] = off * (x[lo:hi].double().abs() @ w[g].abs().t())
    return y, e


def check(out, want, off):
    if out.dtype == torch.bfloat16:
        off = off + HALF * (want.abs() + off)
    assert ((out.double() - want).abs() <= off).all()


def rows(t, k, dtype, how, gen):
    ld = {"plain": k, "odd": k + 1, "even": k + 8}[how]
    x = torch.full((t, ld), float("nan"), dtype=dtype, device="cuda")[:, :k]
    return x.copy_(torch.randn(t, k, generator=gen, device="cuda"))


SINGLE = [(1, 1, 1), (1, 16, 128), (1, 6144, 256), (2, 100, 130), (7, 33, 1000), (8, 64, 384), (9, 48, 640), (16, 129, 2048),
          (17, 200, 96), (33, 520, 1300), (64, 250, 512), (65, 256, 1281), (130, 70, 257), (300, 140, 200), (5, 17, 6144)]


@pytest.mark.parametrize("t,n,k", SINGLE)
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", ["plain", "odd", "even"])
def test_product_of_one_weight(t, n, k, block, dtype, how):
    gen = torch.Generator(device="cuda").manual_seed(t + n + k)
    m = weight((n, k), block, gen)
    x = rows(t, k, dtype, how, gen)
    want, off = expected(x, m)
    check(mg.muon_int4_linear(x, m), want, off)
    check(mg.muon_int4_linear(x, m, out_dtype=torch.float32), want, off)


@pytest.mark.parametrize("t,n,k", [(1, 40, 384), (8, 150, 6144), (20, 150, 1024), (70, 300, 640), (200, 128, 256)])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_whole_numbers_are_exact(t, n, k, block, dtype):
    """Sums of whole halves below 2^23 have one value in fp32, in any order."""
    gen = torch.Generator(device="cuda").manual_seed(k)
    m = weight((n, k), block, gen, whole=True)
    x = torch.randint(-20, 21, (t, k), generator=gen, device="cuda").to(dtype)
    want, _ = expected(x, m)
    assert torch.equal(mg.muon_int4_linear(x, m, out_dtype=torch.float32).double(), want)


# counts of rows for each group, after rows of no group
GROUPS = [(0, [1]), (3, [0, 0, 2, 0]), (0, [8, 1, 0, 9, 17]), (5, [0] * 40), (0, [1] * 70), (2, [3, 0, 30, 1, 64, 65, 0]),
          (0, [0] * 300 + [5] + [0] * 211), (7, [130, 0, 1]), (0, [2] * 96)]


@pytest.mark.parametrize("lead,counts", GROUPS)
@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tail", [0, 3])
def test_product_of_experts(lead, counts, block, dtype, tail):
    gen = torch.Generator(device="cuda").manual_seed(len(counts))
    n, k = 72, 300
    t = lead + sum(counts) + tail
    m = weight((len(counts), n, k), block, gen)
    offsets = torch.tensor(lead + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    x = rows(t, k, dtype, "plain", gen)
    x[:lead] = float("nan")                          # rows of no expert: zero, whatever they hold
    if tail:
        x[-tail:] = float("inf")
    out = mg.muon_int4_linear(x, m, offsets=offsets, out_dtype=torch.float32)
    assert (out[:lead] == 0).all() and (out[t - tail:] == 0).all()
    want, off = expected(torch.where(x.isfinite(), x, torch.zeros_like(x)), m, offsets)
    check(out, want, off)


def test_offsets_that_leave_the_rows_are_clamped():
    gen = torch.Generator(device="cuda").manual_seed(5)
    m = weight((4, 40, 256), 64, gen)
    x = rows(20, 256, torch.bfloat16, "plain", gen)
    for bad, clamped in (([-5, 3, 2, 9, 50], [0, 3, 3, 9, 20]), ([6, 2, 4, 8, 30], [6, 6, 6, 8, 20]),
                         ([30, 40, 50, 60, 70], [20] * 5), ([9, 8, 7, 6, 5], [9] * 5)):
        out = mg.muon_int4_linear(x, m, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        want = mg.muon_int4_linear(x, m, offsets=torch.tensor(clamped, dtype=torch.int32, device="cuda"))
        assert torch.equal(out, want), bad


def test_large_small_and_odd_inputs():
    gen = torch.Generator(device="cuda").manual_seed(6)
    m = weight((32, 256), 128, gen, whole=True)
    for big in (3.3895313892515355e38, 2.0 ** -100, 1.5 + 2.0 ** -23, 3.4028234663852886e38):
        x = torch.zeros(2, 256, device="cuda")
        x[0, 3], x[1, 200] = big, -big
        w = values(m)
        want = torch.stack([w[:, 3] * x[0, 3].double(), w[:, 200] * x[1, 200].double()])
        got = mg.muon_int4_linear(x, m, out_dtype=torch.float32)
        fits = want.abs() < 3.4e38
        assert ((got.double() - want).abs() <= want.abs() * 4 * U)[fits].all(), big
    x = torch.ones(3, 256, device="cuda")
    x[1, 9], x[2, 9] = float("inf"), float("nan")
    got = mg.muon_int4_linear(x, m, out_dtype=torch.float32)
    assert got[0].isfinite().all() and got[2].isnan().all()
    w = values(m)[:, 9]
    assert (got[1][w > 0] == float("inf")).all() and (got[1][w < 0] == -float("inf")).all() and got[1][w == 0].isnan().all()


def test_empty_and_refusals():
    gen = torch.Generator(device="cuda").manual_seed(7)
    m = weight((40, 256), 64, gen)
    x = rows(4, 256, torch.bfloat16, "plain", gen)
    assert mg.muon_int4_linear(x[:0], m).shape == (0, 40)
    s = weight((3, 40, 256), 64, gen)
    off = torch.tensor([0, 1, 2, 4], dtype=torch.int32, device="cuda")
    for bad in (x[:, :255], x.half(), x.cpu(), x.t(), x[0]):
        with pytest.raises(ValueError):
            mg.muon_int4_linear(bad, m)
    for bad in (m._replace(codes=m.codes[:, :64]), m._replace(scale=m.scale.float()), m._replace(scale=m.scale[:2]),
                m._replace(cols=300), m._replace(block=128), m._replace(codes=m.codes.to(torch.int8)), s):
        with pytest.raises(ValueError):
            mg.muon_int4_linear(x, bad)
    for bad in (off[:3], off.long(), off.cpu()):
        with pytest.raises(ValueError):
            mg.muon_int4_linear(x, s, offsets=bad)
    with pytest.raises(ValueError):
        mg.muon_int4_linear(x, m, out_dtype=torch.float16)
    for bad, block in ((torch.zeros(4, 8, device="cuda"), 16), (torch.zeros(4, 8, device="cuda").t(), 32),
                       (torch.zeros(4, device="cuda"), 32), (torch.zeros(4, 8, device="cuda").half(), 32)):
        with pytest.raises(ValueError):
            mg.muon_int4_quantize_weight(bad, block)
