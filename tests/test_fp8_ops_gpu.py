"""8-bit block codes, and the products of linear layers on them.

Codes and scales are compared bit for bit with the definition.  The products are
compared with sums in 64 bits over the values that the codes stand for.  A
product of two E4M3 values is exact in fp32; a sum of r of them in fp32 in any
order is off by at most r * 2^-23 of the sum of their magnitudes (2^-23: an
addition may truncate), and a bf16 result rounds to 2^-8 of itself at most."""
import math

import numpy as np
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def up(n):
    return (n + 127) // 128 * 128


def exponents(amax):
    """e of the definition for an array of block maxima (64 bits)."""
    out = np.zeros(amax.shape, np.int64)
    at = amax > 0
    out[at] = np.ceil(np.log2(amax[at] / 448.0)).astype(np.int64)
    # log2 is inexact near a power of two: settle by the definition itself
    for _ in range(2):
        out[at & (amax > 448.0 * 2.0 ** out)] += 1
        out[at & (amax <= 448.0 * 2.0 ** (out - 1))] -= 1
    return np.clip(out, -127, 127)


def e4m3(v):
    """Codes of 64-bit values of magnitude at most 448, nearest even."""
    a = np.abs(v)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6)
    q = np.rint(a / 2.0 ** (e - 3)) * 2.0 ** (e - 3)
    return np.copysign(q, v)


def pad(x, r, c):
    return np.pad(x, ((0, -x.shape[0] % 128 if r else 0), (0, -x.shape[1] % 128 if c else 0)))


def row_blocks(x):
    p = pad(x, False, True)
    b = p.reshape(p.shape[0], -1, 128)
    e = exponents(np.abs(b).max(-1))
    v = e4m3(b * 2.0 ** -e[..., None].astype(np.float64))
    return v.reshape(p.shape), e.T


def bounds_of(offsets, rows):
    return [(0, rows)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def col_blocks(x, bounds):
    """Codes and exponents of the groups' padded rows, one under the other."""
    vs, es = [], []
    for lo, hi in bounds:
        if hi > lo:
            p = pad(x[lo:hi], True, True)
            v, e = row_blocks(p.T.copy())
            vs.append(v.T)
            es.append(e)
    return np.concatenate(vs), np.concatenate(es)


def weight_blocks(w):
    p = pad(w, True, True)
    b = p.reshape(p.shape[0] // 128, 128, p.shape[1] // 128, 128)
    e = exponents(np.abs(b).max((1, 3)))
    v = e4m3(b * 2.0 ** -e[:, None, :, None].astype(np.float64))
    return v.reshape(p.shape)[:w.shape[0]], e


def data(rows, cols, seed, dtype=BF, blocks=True):
    """Magnitudes that vary by row, by column and by block of 128, so that a
    scale taken from a neighbour shows."""
    rng = np.random.RandomState(seed)
    x = rng.standard_normal((rows, cols))
    x *= np.exp2(rng.randint(-6, 7, (rows, 1))) * np.exp2(rng.randint(-6, 7, (1, cols)))
    if blocks:
        x *= np.kron(np.exp2(rng.randint(-8, 9, (up(rows) // 128, up(cols) // 128))), np.ones((128, 128)))[:rows, :cols]
    t = torch.tensor(x, dtype=dtype)
    return t.double().numpy(), t.to(DEV)


def host(codes):
    return codes.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 6144), (3, 130), (128, 128), (129, 257), (300, 520), (77, 1000)])
def test_codes_of_rows_and_columns(rows, cols, dtype):
    x, xt = data(rows, cols, rows + cols, dtype)
    r, c = mg.muon_fp8_quantize(xt, row=True, col=True)
    v, e = row_blocks(x)
    assert np.array_equal(host(r.codes), v) and np.array_equal(r.scale.cpu().numpy(), e + 127)
    v, e = col_blocks(x, [(0, rows)])
    n = v.shape[0]
    assert np.array_equal(host(c.codes)[:n], v) and np.array_equal(c.scale.cpu().numpy()[:n // 128], e + 127)
    # each alone gives the same
    r1, none = mg.muon_fp8_quantize(xt)
    assert none is None and torch.equal(r1.codes.view(torch.uint8), r.codes.view(torch.uint8))
    none, c1 = mg.muon_fp8_quantize(xt, row=False, col=True)
    assert none is None and torch.equal(c1.codes.view(torch.uint8)[:n], c.codes.view(torch.uint8)[:n])


@pytest.mark.parametrize("offsets", [[0, 5, 5, 200, 328, 328, 400], [0, 400], [0] * 40 + [400], [0, 1, 2, 3, 400],
                                     [0, 128, 256, 400], [3, 100, 390]])
def test_codes_of_groups(offsets):
    x, xt = data(400, 300, 7)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    r, c = mg.muon_fp8_quantize(xt, row=True, col=True, offsets=off)
    v, e = col_blocks(x, bounds_of(offsets, 400))
    n = v.shape[0]
    assert c.codes.shape[0] >= n
    assert np.array_equal(host(c.codes)[:n], v) and np.array_equal(c.scale.cpu().numpy()[:n // 128], e + 127)
    lo, hi = offsets[0], offsets[-1]
    v, e = row_blocks(x)
    assert np.array_equal(host(r.codes)[lo:hi], v[lo:hi])
    assert np.array_equal(r.scale.cpu().numpy()[:, lo:hi], e[:, lo:hi] + 127)


def test_codes_of_weights():
    for shape in ((1, 1), (520, 1300), (3, 200, 129), (2, 128, 256)):
        rows, cols = shape[-2:]
        parts = [data(rows, cols, 11 + i) for i in range(shape[0] if len(shape) == 3 else 1)]
        wt = torch.stack([p[1] for p in parts]) if len(shape) == 3 else parts[0][1]
        m = mg.muon_fp8_quantize_weight(wt)
        for i, (w, _) in enumerate(parts):
            v, e = weight_blocks(w)
            assert np.array_equal(host(m.codes[i] if len(shape) == 3 else m.codes), v)
            assert np.array_equal((m.scale[i] if len(shape) == 3 else m.scale).cpu().numpy(), e + 127)


def test_scale_boundaries():
    # maxima at and next to 448 * 2^e, subnormal and largest numbers, zeros
    tops = [448.0, np.nextafter(np.float32(448), np.float32(1e9)), np.nextafter(np.float32(448), np.float32(0)), 1.0, 0.0,
            1.75, 2.0 ** -126, 2.0 ** -130, 2.0 ** -149, 1.75 * 2.0 ** -140, 3.4028235e38, 1.75 * 2.0 ** 127, 2.0 ** 127]
    x = np.zeros((len(tops), 256), np.float32)
    for i, t in enumerate(tops):
        x[i, 5] = t
        x[i, 6] = -t / 3
        x[i, 200] = t / 7
    r, _ = mg.muon_fp8_quantize(torch.tensor(x, device=DEV))
    v, e = row_blocks(x.astype(np.float64))
    assert np.array_equal(r.scale.cpu().numpy(), e + 127)
    assert np.array_equal(host(r.codes), v)


def test_not_finite_elements_stay_visible():
    x = torch.ones(4, 256, device=DEV)
    x[1, 3], x[2, 130], x[3, 200] = math.inf, math.nan, -math.inf
    r, c = mg.muon_fp8_quantize(x, col=True)
    for codes in (r.codes, c.codes[:4]):
        bad = torch.isnan(codes.float())
        assert int(bad.sum()) == 3 and bool(bad[1, 3]) and bool(bad[2, 130]) and bool(bad[3, 200])
    w = mg.muon_fp8_quantize_weight(torch.ones(40, 256, device=DEV))
    y = mg.muon_fp8_linear(x, w)
    assert bool(torch.isnan(y[1:]).all()) and bool((y[0] == 256).all())


def test_strided_input_and_ones():
    base = torch.randn(50, 401, device=DEV).to(BF)
    for lo, hi in ((0, 256), (1, 301), (16, 316)):
        view = base[:, lo:hi]
        a, ac = mg.muon_fp8_quantize(view, col=True)
        b, bc = mg.muon_fp8_quantize(view.contiguous(), col=True)
        assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scale, b.scale)
        n = 128
        assert torch.equal(ac.codes.view(torch.uint8)[:n], bc.codes.view(torch.uint8)[:n])


# ---------------------------------------------------------------- products --
def near(got, a, b, red):
    """got against a @ b in 64 bits, with the tolerance of the head of the file."""
    ref = a @ b
    tol = red * 2.0 ** -23 * (np.abs(a) @ np.abs(b)) + (2.0 ** -8 * np.abs(ref) if got.dtype == BF else 2.0 ** -23 * np.abs(ref))
    return bool(np.all(np.abs(got.double().cpu().numpy() - ref) <= tol + 1e-40))


def values_row(x):
    v, e = row_blocks(x)
    return (v.reshape(x.shape[0], -1, 128) * 2.0 ** e.T[..., None].astype(np.float64)).reshape(v.shape)[:, :x.shape[1]]


def values_weight(w):
    v, e = weight_blocks(w)
    s = np.kron(2.0 ** e.astype(np.float64), np.ones((128, 128)))
    return (v * s[:v.shape[0]])[:, :w.shape[1]]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 256, 128), (5, 300, 130), (33, 64, 512), (256, 256, 640), (257, 513, 384),
                                   (640, 200, 1000), (1001, 520, 1300), (300, 2049, 257), (64, 128, 4100)])
def test_single_layer(t, n, k, out):
    x, xt = data(t, k, t + k)
    w, wt = data(n, k, n + k + 1)
    dy, dyt = data(t, n, t + n + 2)
    m = mg.muon_fp8_quantize_weight(wt)
    y = mg.muon_fp8_linear(xt, m, out_dtype=out)
    assert y.dtype == out and y.shape == (t, n)
    wv = values_weight(w)
    assert near(y, values_row(x), wv.T, k)
    dx, dw = mg.muon_fp8_linear_backward(dyt, xt, m, dx_dtype=out, dw_dtype=out)
    assert near(dx, values_row(dy), wv, n)
    assert dw.shape == (n, k)
    assert near(dw, values_row(dy.T.copy()), values_row(x.T.copy()).T, t)
    assert mg.muon_device_status() == 0


GROUPS = {
    "uneven": ([0, 3, 3, 140, 141, 397, 700], 700),
    "one": ([0, 50], 50),
    "first_and_last_empty": ([0, 0, 100, 229, 229], 229),
    "one_token_each": (list(range(41)), 40),
    "all_in_one_of_many": ([0] * 30 + [300] * 11, 300),
    "exact_tiles": ([0, 256, 512, 640], 640),
    "room_left": ([0, 17, 90], 128),
}


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("n,k", [(300, 200), (128, 640), (257, 384)])
def test_experts(name, n, k):
    offsets, t = GROUPS[name]
    g = len(offsets) - 1
    x, xt = data(t, k, t + k)
    dy, dyt = data(t, n, t + n)
    parts = [data(n, k, 100 + i) for i in range(g)]
    m = mg.muon_fp8_quantize_weight(torch.stack([p[1] for p in parts]))
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    q, _ = mg.muon_fp8_quantize(xt)
    y = torch.full((t, n), 77.0, dtype=BF, device=DEV)
    mg.muon_fp8_product("forward", q, m, offsets=off, out=y)
    dx, dw = mg.muon_fp8_linear_backward(dyt, xt, m, offsets=off, dw_dtype=F32)
    assert dw.shape == (g, n, k)
    xv, dyv = values_row(x), values_row(dy)
    for i, (lo, hi) in enumerate(zip(offsets[:-1], offsets[1:])):
        wv = values_weight(parts[i][0])
        assert near(y[lo:hi], xv[lo:hi], wv.T, k), i
        assert near(dx[lo:hi], dyv[lo:hi], wv, n), i
        if hi > lo:
            assert near(dw[i], values_row(dy[lo:hi].T.copy()), values_row(x[lo:hi].T.copy()).T, hi - lo), i
        else:
            assert int(torch.count_nonzero(dw[i])) == 0
    assert bool((y[offsets[-1]:] == 77.0).all())         # rows of no expert are left alone
    assert mg.muon_device_status() == 0


def test_no_tokens():
    m = mg.muon_fp8_quantize_weight(torch.randn(3, 64, 96, device=DEV))
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    x, dy = torch.empty(0, 96, device=DEV, dtype=BF), torch.empty(0, 64, device=DEV, dtype=BF)
    assert mg.muon_fp8_linear(x, m, offsets=off).shape == (0, 64)
    dx, dw = mg.muon_fp8_linear_backward(dy, x, m, offsets=off)
    assert dx.shape == (0, 96) and dw.shape == (3, 64, 96) and int(torch.count_nonzero(dw)) == 0


def test_offsets_out_of_range_are_clamped():
    x, xt = data(200, 256, 1)
    parts = [data(64, 256, 50 + i) for i in range(3)]
    m = mg.muon_fp8_quantize_weight(torch.stack([p[1] for p in parts]))
    dy, dyt = data(200, 64, 2)
    # descending, negative and past the end: expert 0 has rows 0-149, 1 none, 2 rows 150-199
    off = torch.tensor([-5, 150, 90, 999], dtype=torch.int32, device=DEV)
    y = mg.muon_fp8_linear(xt, m, offsets=off)
    xv = values_row(x)
    assert near(y[:150], xv[:150], values_weight(parts[0][0]).T, 256)
    assert near(y[150:], xv[150:], values_weight(parts[2][0]).T, 256)
    _, dw = mg.muon_fp8_linear_backward(dyt, xt, m, offsets=off, dw_dtype=F32)
    assert near(dw[0], values_row(dy[:150].T.copy()), values_row(x[:150].T.copy()).T, 150)
    assert int(torch.count_nonzero(dw[1])) == 0
    assert near(dw[2], values_row(dy[150:].T.copy()), values_row(x[150:].T.copy()).T, 50)


def test_output_rows_of_any_stride():
    x, xt = data(70, 200, 3)
    w, wt = data(90, 200, 4)
    m = mg.muon_fp8_quantize_weight(wt)
    q, _ = mg.muon_fp8_quantize(xt)
    for ld, shift in ((90, 0), (101, 3), (128, 1)):
        base = torch.full((70, ld), 5.0, dtype=BF, device=DEV)
        mg.muon_fp8_product("forward", q, m, out=base[:, shift:shift + 90])
        assert near(base[:, shift:shift + 90], values_row(x), values_weight(w).T, 200)
        rest = torch.ones(ld, dtype=torch.bool)
        rest[shift:shift + 90] = False
        assert bool((base[:, rest.to(DEV)] == 5.0).all())


def test_more_tiles_than_the_persistent_grid():
    """Many tiles per pair of SMs: both accumulators and every ring wrap many times."""
    t, n, k = 4096, 2560, 384
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(t, k, generator=g, device=DEV).to(BF)
    w = torch.randn(n, k, generator=g, device=DEV)
    m = mg.muon_fp8_quantize_weight(w)
    y = mg.muon_fp8_linear(x, m, out_dtype=F32)
    q, _ = mg.muon_fp8_quantize(x)
    xv = torch.ldexp(q.codes.float().view(t, -1, 128), (q.scale.t().int() - 127).unsqueeze(-1)).view(t, k)
    e = (m.scale.int() - 127).repeat_interleave(128, 0).repeat_interleave(128, 1)
    wv = torch.ldexp(m.codes.float(), e)
    ref = xv.double() @ wv.double().t()
    tol = k * 2.0 ** -23 * (xv.abs().double() @ wv.abs().double().t()) + 2.0 ** -23 * ref.abs()
    assert bool(((y.double() - ref).abs() <= tol).all())
    again = mg.muon_fp8_linear(x, m, out_dtype=F32)
    assert torch.equal(y, again)                         # no order that changes
    assert mg.muon_device_status() == 0


def test_streams_and_graph():
    x, xt = data(300, 256, 8)
    w, wt = data(200, 256, 9)
    m = mg.muon_fp8_quantize_weight(wt)
    y = mg.muon_fp8_linear(xt, m)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = mg.muon_fp8_linear(xt, m, stream=s)
    s.synchronize()
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3 = mg.muon_fp8_linear(xt, m)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y3)


def test_refusals():
    x = torch.randn(8, 256, device=DEV).to(BF)
    w = mg.muon_fp8_quantize_weight(torch.randn(64, 256, device=DEV))
    ws = mg.muon_fp8_quantize_weight(torch.randn(2, 64, 256, device=DEV))
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="stacked weight"):
        mg.muon_fp8_linear(x, ws)
    with pytest.raises(ValueError, match="stacked weight"):
        mg.muon_fp8_linear(x, w, offsets=off)
    with pytest.raises(ValueError, match="offsets"):
        mg.muon_fp8_linear(x, ws, offsets=off[:2])
    with pytest.raises(ValueError, match="offsets"):
        mg.muon_fp8_linear(x, ws, offsets=off.long())
    with pytest.raises(ValueError, match="expected"):
        mg.muon_fp8_linear(x[:, :128], w)
    with pytest.raises(ValueError, match="scale"):
        mg.muon_fp8_linear(x, w._replace(scale=w.scale[:, :1]))
    with pytest.raises(ValueError, match="codes"):
        mg.muon_fp8_linear(x, w._replace(codes=w.codes.view(torch.uint8)))
    with pytest.raises(ValueError, match="kind"):
        q, _ = mg.muon_fp8_quantize(x)
        mg.muon_fp8_product("forward", q._replace(kind="col"), w)
    with pytest.raises(ValueError, match="product must be"):
        mg.muon_fp8_product("backward", q, w)
    with pytest.raises(ValueError, match="needs tokens"):
        mg.muon_fp8_product("grad_weight", q, q)
    with pytest.raises(ValueError, match="2-D CUDA"):
        mg.muon_fp8_linear(x.cpu(), w)
    with pytest.raises(ValueError, match="rows of x"):
        mg.muon_fp8_quantize(x.t())
    with pytest.raises(ValueError, match="dy"):
        mg.muon_fp8_linear_backward(x, x, w)


def dequantized(m):
    """What an Fp8Matrix ("row" or "block") stands for, in 64 bits on the device."""
    if m.kind == "row":
        t = m.codes.shape[0]
        return torch.ldexp(m.codes.double().view(t, -1, 128), (m.scale.t().int() - 127).unsqueeze(-1)).view(t, -1)[:, :m.cols]
    e = (m.scale.int() - 127).repeat_interleave(128, -2).repeat_interleave(128, -1)
    return torch.ldexp(m.codes.double(), e[..., :m.codes.shape[-2], :])[..., :m.cols]


@pytest.mark.parametrize("offsets", [None, [0, 700, 700, 1301, 2600], [0, 30, 2560, 2600], [0, 1024, 1500, 2500],
                                     [7, 520, 1033, 2599]])
@pytest.mark.parametrize("out", [BF, F32])
def test_many_tiles_of_large_groups(offsets, out):
    """Sizes at which two pairs of SMs share the weight's tiles: uneven, empty and
    small groups, column tiles that come out empty, rows and columns past the end."""
    t, inner, red = 2600, 3001, 640
    g = 1 if offsets is None else len(offsets) - 1
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(31)
    spread = torch.exp2(torch.randint(-6, 7, (t, 1), generator=gen, device=DEV).float())
    x = (torch.randn(t, red, generator=gen, device=DEV) * spread).to(BF)
    q, _ = mg.muon_fp8_quantize(x)
    xv = dequantized(q)
    for product, shape in (("forward", (inner, red)), ("grad_input", (red, inner))):
        w = torch.randn(g, *shape, generator=gen, device=DEV)
        m = mg.muon_fp8_quantize_weight(w if offsets is not None else w[0])
        wv = dequantized(m)
        y = torch.full((t, inner), 55.0, dtype=out, device=DEV)
        mg.muon_fp8_product(product, q, m, offsets=off, out=y)
        for i, (lo, hi) in enumerate(bounds_of(offsets, t)):
            b = wv if offsets is None else wv[i]
            b = b.t() if product == "forward" else b
            ref = xv[lo:hi] @ b
            tol = red * 2.0 ** -23 * (xv[lo:hi].abs() @ b.abs()) + (2.0 ** -8 if out == BF else 2.0 ** -23) * ref.abs()
            assert bool(((y[lo:hi].double() - ref).abs() <= tol).all()), (product, i)
        if offsets is not None:
            assert bool((y[:offsets[0]] == 55.0).all()) and bool((y[offsets[-1]:] == 55.0).all())
    assert mg.muon_device_status() == 0


@pytest.mark.parametrize("inner", [301, 302, 303, 304, 290, 513])
def test_columns_behind_the_output_stay(inner):
    """Rows that start on 16 bytes and end elsewhere: what lies between the last
    column and the next row is not the product's."""
    gen = torch.Generator(device=DEV).manual_seed(inner)
    t, red, ld = 160, 300, (inner + 8) // 8 * 8
    q, _ = mg.muon_fp8_quantize(torch.randn(t, red, generator=gen, device=DEV).to(BF))
    for product, shape in (("forward", (inner, red)), ("grad_input", (red, inner))):
        m = mg.muon_fp8_quantize_weight(torch.randn(*shape, generator=gen, device=DEV))
        for out in (BF, F32):
            y = mg.muon_fp8_product(product, q, m, out_dtype=out)
            wide = torch.full((t, ld), 55.0, dtype=out, device=DEV)
            mg.muon_fp8_product(product, q, m, out=wide[:, :inner])
            assert torch.equal(wide[:, :inner], y) and bool((wide[:, inner:] == 55.0).all()), (product, out)
    assert mg.muon_device_status() == 0


@pytest.mark.parametrize("t,inner,red", [(4100, 2500, 2100), (2500, 4611, 2048)])
def test_one_weight_shared_by_many_tiles(t, inner, red):
    """One weight, many column tiles and a long reduction: clusters of two pairs of
    SMs, with an odd number of full column tiles and edges in every direction."""
    gen = torch.Generator(device=DEV).manual_seed(t)
    x = torch.randn(t, red, generator=gen, device=DEV).to(BF)
    q, _ = mg.muon_fp8_quantize(x)
    xv = dequantized(q)
    for product, shape in (("forward", (inner, red)), ("grad_input", (red, inner))):
        m = mg.muon_fp8_quantize_weight(torch.randn(*shape, generator=gen, device=DEV))
        b = dequantized(m).t() if product == "forward" else dequantized(m)
        for off in (None, torch.tensor([100, t - 77], dtype=torch.int32, device=DEV)):
            lo, hi = (0, t) if off is None else (100, t - 77)
            w = m if off is None else mg.Fp8Matrix(m.codes[None], m.scale[None], "block", m.cols)
            y = torch.full((t, inner), 55.0, dtype=F32, device=DEV)
            mg.muon_fp8_product(product, q, w, offsets=off, out=y)
            ref = xv[lo:hi] @ b
            tol = red * 2.0 ** -23 * (xv[lo:hi].abs() @ b.abs()) + 2.0 ** -23 * ref.abs()
            assert bool(((y[lo:hi].double() - ref).abs() <= tol).all()), product
            assert bool((y[:lo] == 55.0).all()) and bool((y[hi:] == 55.0).all())
    assert mg.muon_device_status() == 0


def test_backward_on_streams_in_a_graph_and_one_after_the_other():
    """Both products of a layer's gradients may run side by side, and whatever
    follows on the stream comes after both."""
    gen = torch.Generator(device=DEV).manual_seed(77)
    t, n, k, g = 900, 520, 640, 5
    off = torch.tensor([0, 100, 100, 420, 800, 900], dtype=torch.int32, device=DEV)
    x = torch.randn(t, k, generator=gen, device=DEV).to(BF)
    dy = torch.randn(t, n, generator=gen, device=DEV).to(BF)
    m = mg.muon_fp8_quantize_weight(torch.randn(g, n, k, generator=gen, device=DEV))
    dx, dw = mg.muon_fp8_linear_backward(dy, x, m, offsets=off)
    # each alone
    only, none = mg.muon_fp8_linear_backward(dy, x, m, offsets=off, need_dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = mg.muon_fp8_linear_backward(dy, x, m, offsets=off, need_dx=False)
    assert none is None and torch.equal(only, dw)
    # operands of two types take a launch each
    _, w32 = mg.muon_fp8_linear_backward(dy, x.float(), m, offsets=off)
    assert torch.equal(w32, dw)
    for _ in range(20):                                  # consumers right behind
        a, b = mg.muon_fp8_linear_backward(dy, x, m, offsets=off)
        assert torch.equal(a + 0, dx) and torch.equal(b + 0, dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = mg.muon_fp8_linear_backward(dy, x, m, offsets=off, stream=s)
    s.synchronize()
    assert torch.equal(a, dx) and torch.equal(b, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = mg.muon_fp8_linear_backward(dy, x, m, offsets=off)
        c, d = a * 2, b * 2
    for _ in range(3):
        c.zero_()
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, dx) and torch.equal(b, dw) and torch.equal(c, dx * 2) and torch.equal(d, dw * 2)
    assert mg.muon_device_status() == 0


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("product,t,inner,red", [
    ("forward", 40, 5000, 2100), ("forward", 300, 700, 3001), ("forward", 700, 301, 4500), ("forward", 9, 256, 4096),
    ("grad_input", 40, 2000, 4200), ("grad_input", 300, 700, 6200), ("grad_input", 500, 301, 8200),
    ("grad_weight", 700, 300, 4100), ("grad_weight", 301, 513, 6200), ("grad_weight", 130, 520, 8200)])
def test_few_tiles_and_a_long_reduction(product, t, inner, red, out):
    """Sizes at which two, three or four pairs of SMs share a tile's reduction, with
    edges in every direction, output rows of a stride, and the same bits each time.
    (Of the weight gradient `t` is the rows, `red` the tokens.)"""
    gen = torch.Generator(device=DEV).manual_seed(red)
    x = (torch.randn(t, red, generator=gen, device=DEV) *
         torch.exp2(torch.randint(-6, 7, (1, red), generator=gen, device=DEV).float())).to(BF)
    b = torch.randn(red, inner, generator=gen, device=DEV).to(BF)
    if product == "grad_weight":
        _, p = mg.muon_fp8_quantize(x.t().contiguous(), row=False, col=True)
        _, m = mg.muon_fp8_quantize(b, row=False, col=True)
        # the same blocks of 128 tokens as rows' blocks of the transposed operands
        pv = dequantized(mg.muon_fp8_quantize(x)[0])
        mv = dequantized(mg.muon_fp8_quantize(b.t().contiguous())[0]).t()
        extra = {"tokens": red}
    else:
        p, _ = mg.muon_fp8_quantize(x)
        m = mg.muon_fp8_quantize_weight(b.t().contiguous() if product == "forward" else b)
        pv, mv = dequantized(p), dequantized(m)
        mv = mv.t() if product == "forward" else mv
        extra = {}
    ref = pv @ mv
    tol = red * 2.0 ** -23 * (pv.abs() @ mv.abs()) + (2.0 ** -8 if out == BF else 2.0 ** -23) * ref.abs()
    y = torch.full((t, inner), 55.0, dtype=out, device=DEV)
    first = mg.muon_fp8_product(product, p, m, out=y, **extra).clone()
    assert bool(((first.double() - ref).abs() <= tol).all())
    for _ in range(5):
        assert torch.equal(mg.muon_fp8_product(product, p, m, out=y, **extra), first)
    if product != "grad_weight":
        wide = torch.full((t, inner + 3), 55.0, dtype=out, device=DEV)
        mg.muon_fp8_product(product, p, m, out=wide[:, :inner])
        assert torch.equal(wide[:, :inner], first) and bool((wide[:, inner:] == 55.0).all())
    assert mg.muon_device_status() == 0


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("t,n,k", [(512, 300, 500), (500, 301, 500), (512, 1024, 1024), (256, 2048, 4100), (130, 520, 2000),
                                   (700, 130, 130), (1000, 2047, 2048), (65, 256, 6144)])
def test_narrow_tiles(t, n, k, out):
    """Sizes that are cut into column tiles of 64 or 128, some with slices of the reduction."""
    test_few_tiles_and_a_long_reduction("forward", t, n, k, out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("at", range(9))
def test_codes_of_windows(at, dtype):
    """A window of a larger matrix that starts and ends anywhere, in edge tiles in
    every direction: what lies around it shows in no code and no scale."""
    for rows, cols, ld in ((150, 131, 143), (150, 137, 160), (97, 263, 264), (260, 120, 129)):
        _, part = data(rows, cols, at + cols, dtype)
        whole = torch.full((at + rows * ld + 7,), math.nan, dtype=dtype, device=DEV)
        x = whole.as_strided((rows, cols), (ld, 1), at)
        x.copy_(part)
        for row, col in ((True, False), (False, True), (True, True)):
            got, want = mg.muon_fp8_quantize(x, row=row, col=col), mg.muon_fp8_quantize(part, row=row, col=col)
            for g, w in zip(got, want):
                assert (g is None) == (w is None)
                if g is not None:
                    assert torch.equal(g.codes.view(torch.uint8), w.codes.view(torch.uint8)) and torch.equal(g.scale, w.scale)
