"""What the binding never asks of the entry points between an expert layer's routing
and its result: results with rows apart, on any address, with what lies between them
left alone; and offsets past 32 bits."""
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODE = {torch.bfloat16: 0, torch.float32: 1}
MARK = -1234.0


def room(rows, cols, dtype, gap, shift):
    """(whole buffer, rows x cols view with `gap` elements between rows, `shift` elements in), all MARK."""
    ld = cols + gap
    buf = torch.full((rows * ld + shift + 16,), MARK, dtype=dtype, device=DEV)
    return buf, buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]


def only_written(buf, view):
    """Nothing of the buffer but the view has changed."""
    left = buf.clone()
    left.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(MARK)
    return bool((left == MARK).all())


@pytest.fixture(scope="module")
def L():
    return mg.lib()


def ok(rc):
    assert rc == 0, mg.lib().muon_last_error()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [5, 64, 260, 1301])
@pytest.mark.parametrize("gap,shift", [(3, 1), (8, 0), (1, 4)])
def test_rows_apart(L, dtype, cols, gap, shift):
    gen = torch.Generator(device=DEV).manual_seed(cols)
    tokens, top_k = 37, 3
    chosen = torch.randint(-1, 6, (tokens, top_k), generator=gen, device=DEV, dtype=torch.int32)
    plan = mg.muon_sort_tokens(chosen, 4, first=1)
    x = torch.randn(tokens, cols, generator=gen, device=DEV).to(dtype)
    y = torch.randn(tokens * top_k, cols, generator=gen, device=DEV).to(dtype)
    w = torch.randn(tokens, top_k, generator=gen, device=DEV)
    place, offs = plan.place.data_ptr(), plan.offsets.data_ptr()
    code, n = CODE[dtype], tokens * top_k
    buf, out = room(n, cols, dtype, gap, shift)
    ok(L.muon_dispatch_tokens(x.data_ptr(), code, tokens, cols, cols, top_k, place, offs, 4, out.data_ptr(), cols + gap, None))
    assert torch.equal(out, mg.muon_dispatch_tokens(x, plan)) and only_written(buf, out)
    buf, out = room(tokens, cols, dtype, gap, shift)
    ok(L.muon_combine_tokens(y.data_ptr(), code, cols, tokens, cols, top_k, place, offs, 4, w.data_ptr(), out.data_ptr(), code,
                             cols + gap, None))
    assert torch.equal(out, mg.muon_combine_tokens(y, plan, w)) and only_written(buf, out)
    buf, dy = room(n, cols, dtype, gap, shift)
    dw = torch.empty(tokens, top_k, device=DEV)
    ok(L.muon_combine_tokens_backward(x.data_ptr(), code, cols, y.data_ptr(), code, cols, tokens, cols, top_k, place, offs, 4,
                                      w.data_ptr(), dy.data_ptr(), cols + gap, dw.data_ptr(), None))
    # aligned rows are added up four entries at a time, these one at a time: the same products, rounded alike
    want_dy, want_dw = mg.muon_combine_tokens_backward(x, y, plan, w)
    assert torch.equal(dy, want_dy) and only_written(buf, dy)
    size = (y.double()[plan.place.long()] * x.double()[:, None]).abs().sum(-1)
    assert ((dw - want_dw).double().abs() <= 2 * cols * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 9), (7, 130), (40, 264)])
@pytest.mark.parametrize("gap,shift", [(3, 1), (8, 0), (0, 3)])
def test_gated_apart(L, dtype, rows, cols, gap, shift):
    g, u, d = (torch.randn(rows, cols, device=DEV).to(dtype) for _ in range(3))
    buf, out = room(rows, cols, dtype, gap, shift)
    ok(L.muon_swiglu(g.data_ptr(), cols, u.data_ptr(), cols, CODE[dtype], rows, cols, out.data_ptr(), cols + gap, None))
    assert torch.equal(out, mg.muon_swiglu(g, u)) and only_written(buf, out)
    buf1, dg = room(rows, cols, dtype, gap, shift)
    buf2, du = room(rows, cols, dtype, gap + 2, shift + 1)
    ok(L.muon_swiglu_backward(d.data_ptr(), cols, g.data_ptr(), cols, u.data_ptr(), cols, CODE[dtype], rows, cols, dg.data_ptr(),
                              cols + gap, du.data_ptr(), cols + gap + 2, None))
    want = mg.muon_swiglu_backward(d, g, u)
    assert torch.equal(dg, want[0]) and torch.equal(du, want[1]) and only_written(buf1, dg) and only_written(buf2, du)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,gap,shift", [(33, 5, 1), (64, 8, 0)])
def test_four_bits_apart(L, dtype, n, gap, shift):
    k, tokens = 200, 11
    m = mg.muon_int4_quantize_weight(torch.randn(3, n, k, device=DEV), 32)
    x = torch.randn(tokens, k, device=DEV).to(torch.bfloat16)
    offs = torch.tensor([2, 4, 4, 9], dtype=torch.int32, device=DEV)
    buf, out = room(tokens, n, dtype, gap, shift)
    # scales from an address that is no multiple of 4
    scale = torch.empty(m.scale.numel() + 1, dtype=torch.bfloat16, device=DEV)[1:]
    scale.copy_(m.scale.reshape(-1))
    ok(L.muon_int4_linear(x.data_ptr(), 0, tokens, k, m.codes.data_ptr(), scale.data_ptr(), 32, n, k, 3, offs.data_ptr(),
                          out.data_ptr(), CODE[dtype], n + gap, None))
    assert torch.equal(out, mg.muon_int4_linear(x, m, offsets=offs, out_dtype=dtype)) and only_written(buf, out)


def test_offsets_past_32_bits():
    """2.7e9 elements of rows: the last tokens' against the same tokens by themselves."""
    tokens, top_k, cols, last = 41000, 8, 8192, 40
    x = torch.empty(tokens, cols, dtype=torch.bfloat16, device=DEV)
    x[-last:] = torch.randn(last, cols, device=DEV)
    x[:-last] = 1
    chosen = torch.arange(top_k, dtype=torch.int32, device=DEV).expand(tokens, top_k).contiguous()
    plan = mg.muon_sort_tokens(chosen, top_k)
    assert torch.equal(plan.offsets.cpu(), torch.arange(top_k + 1, dtype=torch.int32) * tokens)
    y = mg.muon_dispatch_tokens(x, plan)
    assert y.numel() > 1 << 31 and torch.equal(y[-last:], x[-last:]) and bool((y[-last - 1] == 1).all())
    w = torch.rand(tokens, top_k, device=DEV)
    few = mg.muon_sort_tokens(chosen[-last:].contiguous(), top_k)
    part = mg.muon_dispatch_tokens(x[-last:], few)
    out = mg.muon_combine_tokens(y, plan, w)
    assert torch.equal(out[-last:], mg.muon_combine_tokens(part, few, w[-last:].contiguous()))
    dy, dw = mg.muon_combine_tokens_backward(out, y, plan, w)
    dy2, dw2 = mg.muon_combine_tokens_backward(out[-last:], part, few, w[-last:].contiguous())
    assert torch.equal(dw[-last:], dw2) and torch.equal(dy[plan.place[-last:].long()], dy2[few.place.long()])
    del dy, out
    g = mg.muon_swiglu(y, y)
    assert torch.equal(g[-last:], mg.muon_swiglu(y[-last:], y[-last:]))
    d_gate, d_up = mg.muon_swiglu_backward(g, y, y)
    e_gate, e_up = mg.muon_swiglu_backward(g[-last:], y[-last:], y[-last:])
    assert torch.equal(d_gate[-last:], e_gate) and torch.equal(d_up[-last:], e_up)


def test_codes_past_32_bits():
    """500 experts' codes take 4.9 GB: the last expert's product against that of a weight by itself."""
    groups, n, k = 500, 1600, 12288
    one = mg.muon_int4_quantize_weight(torch.randn(n, k, device=DEV), 64)
    codes = torch.zeros(groups, n, k // 2, dtype=torch.uint8, device=DEV)
    scale = torch.zeros(groups, k // 64, n, dtype=torch.bfloat16, device=DEV)
    assert codes.numel() > 1 << 32
    codes[-1], scale[-1] = one.codes, one.scale
    x = torch.randn(5, k, device=DEV).to(torch.bfloat16)
    offs = torch.zeros(groups + 1, dtype=torch.int32, device=DEV)
    offs[1:] = 2
    offs[-1] = 5
    out = mg.muon_int4_linear(x, mg.Int4Matrix(codes, scale, 64, k), offsets=offs)
    assert bool((out[:2] == 0).all()) and torch.equal(out[2:], mg.muon_int4_linear(x[2:], one))
