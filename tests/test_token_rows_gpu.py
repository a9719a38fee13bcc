"""Entries sorted by expert, tokens' rows to the experts and, weighted, back, and
their gradients, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}      # half a step, relative
U = 2.0 ** -24


def sorted_by_counting(chosen, experts, first):
    flat = chosen.reshape(-1).astype(np.int64) - first
    flat[(flat < 0) | (flat >= experts)] = -1
    runs = [np.flatnonzero(flat == e) for e in range(-1, experts)]
    order = np.concatenate(runs)
    place = np.empty_like(order)
    place[order] = np.arange(order.size)
    return order, place.reshape(chosen.shape), np.cumsum([r.size for r in runs])


def check_sort(chosen, experts, first=0, **kw):
    plan = mg.muon_sort_tokens(torch.tensor(chosen, dtype=torch.int32, device="cuda"), experts, first=first, **kw)
    want = sorted_by_counting(chosen, experts, first)
    for got, w in zip(plan, want):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), w)
    return plan


# one block (up to 4096 entries), its last chunk, two launches, uneven last run, more entries than 128 blocks' chunks
@pytest.mark.parametrize("tokens,top_k,experts", [(0, 8, 4), (1, 1, 1), (1, 8, 384), (3, 5, 7), (31, 1, 2), (2048, 1, 5),
                                                  (2049, 1, 33), (1024, 4, 1024), (1025, 4, 96), (4097, 1, 512), (5000, 3, 511),
                                                  (6001, 1, 1024), (33000, 8, 60), (70001, 4, 600)])
def test_sort_against_counting(tokens, top_k, experts):
    rng = np.random.RandomState(tokens + experts)
    chosen = rng.randint(-1, experts, (tokens, top_k))
    check_sort(chosen, experts)
    # a rank's share in the middle: numbers below, above and negative are no expert's here
    first = experts // 3
    chosen = rng.randint(-3, 2 * experts + 2, (tokens, top_k))
    check_sort(chosen, max(1, experts // 2), first)


@pytest.mark.parametrize("tokens", [300, 9000])
def test_sort_of_one_kind(tokens):
    check_sort(np.full((tokens, 2), 3), 8)          # every entry one expert's
    check_sort(np.full((tokens, 2), -1), 8)         # none
    check_sort(np.full((tokens, 2), 7), 3, 4)       # all of others
    check_sort(np.full((tokens, 2), 6), 3, 4)       # the last
    worst = np.array([[-2 ** 31, 2 ** 31 - 1]] * tokens)
    check_sort(worst, 1024, 0)
    check_sort(worst, 4, 1 << 30)


def test_sort_agrees_with_the_layers_sort():
    from muon_newton_schulz_step_gb300 import experts
    logits = torch.randn(700, 24, device="cuda")
    logits[5] = -float("inf")
    _, chosen, counts = mg.muon_route(logits, 3)
    order, offsets = experts.sort_tokens(chosen, counts)
    plan = mg.muon_sort_tokens(chosen, 24)
    assert torch.equal(plan.order.long(), order) and torch.equal(plan.offsets, offsets)


def a_plan(tokens, top_k, experts, held, seed=0):
    """A plan with some entries of no expert (and one token of none)."""
    rng = np.random.RandomState(seed)
    chosen = np.stack([rng.permutation(experts)[:top_k] for _ in range(tokens)]) if tokens else np.zeros((0, top_k), int)
    if tokens > 2:
        chosen[tokens // 2] = -1
    c = torch.tensor(chosen, dtype=torch.int32, device="cuda")
    return mg.muon_sort_tokens(c, held)


def matrix(rows, cols, dtype, gen, how):
    """rows x cols: contiguous, rows apart by an odd or even stride, or from an odd element on."""
    ld = {"plain": cols, "odd": cols + 3, "even": cols + 8, "shifted": cols + 5}[how]
    big = torch.full((rows * ld + 8,), float("nan"), dtype=dtype, device="cuda")
    at = 1 if how == "shifted" else 0
    m = big[at:at + rows * ld].view(rows, ld)[:, :cols]
    m.copy_(torch.randn(rows, cols, generator=gen, device="cuda"))
    return m


SHAPES = [(1, 1, 1, 1), (1, 8, 1, 16), (5, 3, 7, 9), (17, 4, 130, 8), (9, 32, 64, 40), (64, 2, 513, 6), (33, 6, 1301, 12),
          (3, 8, 6144, 16), (40, 9, 264, 20), (0, 4, 16, 4), (50, 3, 12, 5),
          (21, 5, 1300, 9), (6, 2, 4, 3)]


@pytest.mark.parametrize("tokens,top_k,cols,experts", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", ["plain", "odd", "even", "shifted"])
def test_dispatch_copies_rows(tokens, top_k, cols, experts, dtype, how):
    experts = max(experts, top_k)
    gen = torch.Generator(device="cuda").manual_seed(tokens + cols)
    plan = a_plan(tokens, top_k, experts, (experts + 1) // 2)
    x = matrix(tokens, cols, dtype, gen, how)
    if tokens > 2:
        x[tokens // 2] = float("nan")               # a token of no expert: its row goes nowhere
    out = mg.muon_dispatch_tokens(x, plan)
    want = x[plan.order.long() // top_k].clone()
    want[:int(plan.offsets[0])] = 0
    assert out.dtype == dtype and torch.equal(out, want)


@pytest.mark.parametrize("tokens,top_k,cols,experts", SHAPES)
@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, None), (torch.float32, None), (torch.bfloat16, torch.float32),
                                             (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("how", ["plain", "shifted"])
def test_combine_against_64_bits(tokens, top_k, cols, experts, dtype, out_dtype, weighted, how):
    experts = max(experts, top_k)
    gen = torch.Generator(device="cuda").manual_seed(tokens * 3 + cols)
    plan = a_plan(tokens, top_k, experts, (experts + 1) // 2)
    y = matrix(tokens * top_k, cols, dtype, gen, how)
    held = plan.place >= plan.offsets[0]
    y[:int(plan.offsets[0])] = float("nan")         # rows of no expert are not read
    w = torch.randn(tokens, top_k, generator=gen, device="cuda") if weighted else None
    if weighted:
        w[~held] = float("inf")                     # nor their weights
    out = mg.muon_combine_tokens(y, plan, w, out_dtype=out_dtype)
    assert out.dtype == (out_dtype or dtype) and out.shape == (tokens, cols)
    rows = y.double()[plan.place.long()]
    terms = torch.where(held[..., None], rows * (w.double()[..., None] if weighted else 1.0), torch.zeros_like(rows))
    want, size = terms.sum(1), terms.abs().sum(1)
    # top_k fused multiply-adds, then one rounding of the result
    sum_off = top_k * U * size
    off = sum_off + (HALF[out.dtype] * (want.abs() + sum_off) if out.dtype == torch.bfloat16 else 0.0)
    assert ((out.double() - want).abs() <= off).all()


def test_combine_of_infinite_and_nan_rows():
    plan = a_plan(8, 2, 4, 4)
    y = torch.ones(16, 24, device="cuda")
    t = 1
    y[plan.place[t, 0].long(), 3] = float("inf")
    y[plan.place[t, 1].long(), 4] = float("nan")
    out = mg.muon_combine_tokens(y, plan, torch.full((8, 2), 0.5, device="cuda"))
    assert out[t, 3] == float("inf") and out[t, 4].isnan()
    keep = torch.ones(8, 24, dtype=torch.bool, device="cuda")
    keep[t, 3:5] = False
    assert out[keep].isfinite().all()


@pytest.mark.parametrize("tokens,top_k,cols,experts", SHAPES)
@pytest.mark.parametrize("d_dtype,dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                           (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("how", ["plain", "shifted"])
def test_combine_backward_against_64_bits(tokens, top_k, cols, experts, d_dtype, dtype, how):
    experts = max(experts, top_k)
    gen = torch.Generator(device="cuda").manual_seed(tokens * 5 + cols)
    plan = a_plan(tokens, top_k, experts, (experts + 1) // 2)
    y = matrix(tokens * top_k, cols, dtype, gen, how)
    y[:int(plan.offsets[0])] = float("nan")
    d = matrix(tokens, cols, d_dtype, gen, how)
    if tokens > 2:
        d[tokens // 2] = float("nan")               # a token of no expert passes nothing on
    w = torch.randn(tokens, top_k, generator=gen, device="cuda")
    held = plan.place >= plan.offsets[0]
    w[~held] = float("nan")
    dy, dw = mg.muon_combine_tokens_backward(d, y, plan, w)
    rows, dd = y.double()[plan.place.long()], d.double()[:, None, :].expand(-1, top_k, -1)
    terms = torch.where(held[..., None], rows * dd, torch.zeros_like(rows))
    assert dw.dtype == torch.float32 and (dw[~held] == 0).all()
    assert ((dw.double() - terms.sum(-1)).abs() <= cols * U * terms.abs().sum(-1)).all()
    want = torch.zeros(tokens * top_k, cols, dtype=torch.float64, device="cuda")
    prod = torch.where(held[..., None], w.double()[..., None] * dd, torch.zeros_like(rows))
    want[plan.place.long().reshape(-1)] = prod.reshape(-1, cols)
    # a product in fp32, then y's type
    off = want.abs() * (U + (HALF[dtype] * (1 + U) if dtype == torch.bfloat16 else 0.0))
    assert dy.dtype == dtype and ((dy.double() - want).abs() <= off).all()
    # one of the two alone gives the same bits
    assert torch.equal(mg.muon_combine_tokens_backward(d, y, plan, w, need_dw=False)[0], dy)
    assert torch.equal(mg.muon_combine_tokens_backward(d, y, plan, w, need_dy=False)[1], dw)


def test_combine_backward_without_weights_is_dispatch():
    plan = a_plan(50, 3, 8, 4)
    d, y = torch.randn(50, 40, device="cuda"), torch.randn(150, 40, device="cuda")
    dy, dw = mg.muon_combine_tokens_backward(d, y, plan)
    assert dw is None and torch.equal(dy, mg.muon_dispatch_tokens(d, plan))


def test_gradients_against_differences():
    """fp32 differences of the weighted sum: f is linear in y and in the weights, so a central
    difference of step 1 is exact but for the rounding of the sums."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    plan = a_plan(6, 2, 5, 3)
    y = torch.randn(12, 20, generator=gen, device="cuda")
    y[:int(plan.offsets[0])] = 0
    w = torch.randn(6, 2, generator=gen, device="cuda")
    d = torch.randn(6, 20, generator=gen, device="cuda")
    dy, dw = mg.muon_combine_tokens_backward(d, y, plan, w)

    def f(y, w):
        return float((mg.muon_combine_tokens(y, plan, w).double() * d.double()).sum())

    size = float(d.abs().sum()) * float(y.abs().max() + 1) * (float(w.abs().max()) + 1) * 2
    for t, j in ((0, 0), (2, 1), (3, 0), (5, 1)):
        e = torch.zeros_like(w)
        e[t, j] = 1
        assert abs((f(y, w + e) - f(y, w - e)) / 2 - float(dw[t, j])) <= 8 * U * size
        r = int(plan.place[t, j])
        e = torch.zeros_like(y)
        e[r, 7] = 1
        assert abs((f(y + e, w) - f(y - e, w)) / 2 - float(dy[r, 7])) <= 8 * U * size


def test_refusals_on_the_device():
    plan = a_plan(4, 2, 4, 4)
    x = torch.zeros(4, 8, device="cuda")
    y = torch.zeros(8, 8, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    with pytest.raises(ValueError):
        mg.muon_sort_tokens(plan.place.long(), 4)
    with pytest.raises(ValueError, match="contiguous"):
        mg.muon_sort_tokens(torch.zeros(4, 4, dtype=torch.int32, device="cuda")[:, :2], 4)
    with pytest.raises(ValueError):
        mg.muon_sort_tokens(plan.place, 0)
    with pytest.raises(mg.MuonError):
        mg.muon_sort_tokens(plan.place, 1025)
    with pytest.raises(mg.MuonError):
        mg.muon_sort_tokens(plan.place, 4, first=-1)
    for bad in (x[:3], x.half(), x.t()):
        with pytest.raises(ValueError):
            mg.muon_dispatch_tokens(bad, plan)
    for bad in (y[:7], y.double()):
        with pytest.raises(ValueError):
            mg.muon_combine_tokens(bad, plan)
    for bad in (w[:3], w.bfloat16(), torch.zeros(2, 4, device="cuda").t()):
        with pytest.raises(ValueError):
            mg.muon_combine_tokens(y, plan, bad)
    with pytest.raises(ValueError):
        mg.muon_combine_tokens(y, plan, w, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mg.muon_combine_tokens_backward(x[:, :7], y, plan, w)
    with pytest.raises(ValueError):
        mg.muon_combine_tokens(y, plan._replace(offsets=plan.offsets.long()))
    with pytest.raises(ValueError):
        mg.muon_combine_tokens(y, plan._replace(place=plan.place.t()))
