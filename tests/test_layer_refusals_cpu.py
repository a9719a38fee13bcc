"""Refusals of the operators between an expert layer's routing and its result, and
of the products with weights of 4 bits, without a GPU: the binding refuses host
tensors and wrong types, the C ABI bad sizes and pointers (fake addresses:
validation reads none)."""
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg
from muon_newton_schulz_step_gb300 import build as cuda_build

OK, INVALID, UNSUPPORTED, CUDA, OOM = range(5)
A = 1 << 20


@pytest.fixture(scope="module")
def L():
    cuda_build.build()
    return mg.lib()


def test_binding_refuses_host_tensors_and_wrong_types():
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    plan = mg.TokenPlan(i.reshape(-1), i, torch.zeros(3, dtype=torch.int32))
    w4 = mg.Int4Matrix(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.bfloat16), 128, 8)
    for call in (lambda: mg.muon_sort_tokens(i, 2), lambda: mg.muon_dispatch_tokens(x, plan),
                 lambda: mg.muon_combine_tokens(x, plan), lambda: mg.muon_combine_tokens_backward(x, x, plan),
                 lambda: mg.muon_swiglu(x, x), lambda: mg.muon_swiglu_backward(x, x, x),
                 lambda: mg.muon_int4_quantize_weight(x), lambda: mg.muon_int4_linear(x, w4)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    for bad in (None, (i, i, i), [1]):
        with pytest.raises(ValueError, match="TokenPlan"):
            mg.muon_combine_tokens(x, bad)
        with pytest.raises(ValueError, match="Int4Matrix"):
            mg.muon_int4_linear(x, bad)
    with pytest.raises(ValueError, match="stacked weight"):
        mg.muon_int4_linear(x, w4, offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="block of 32, 64 or 128"):
        mg.muon_int4_linear(x, w4._replace(block=16))


def test_sort_arguments(L):
    def sort(chosen=A, n=100, first=0, experts=8, ws=None, wsb=0, order=A, place=A, offsets=A):
        return L.muon_sort_tokens(chosen, n, first, experts, ws, wsb, order, place, offsets, None)

    for kw in (dict(n=-1), dict(n=(1 << 30) + 1), dict(first=-1), dict(first=(1 << 30) + 1), dict(chosen=None),
               dict(chosen=A + 2), dict(order=None), dict(place=None), dict(offsets=None), dict(offsets=A + 1)):
        assert sort(**kw) == INVALID, kw
    assert sort(experts=0) == UNSUPPORTED and sort(experts=1025) == UNSUPPORTED
    big = 1 << 20
    need = L.muon_sort_tokens_workspace_bytes(big, 8)
    assert need > 0 and need % (9 * 4) == 0
    assert sort(n=big) == INVALID                              # no workspace
    assert sort(n=big, ws=A, wsb=need - 1) == OOM
    assert sort(n=big, ws=A + 4, wsb=need) == INVALID
    assert L.muon_sort_tokens_workspace_bytes(8, 384) == 0     # one block
    for n, e in ((-1, 8), (8, 0), (8, 1025), ((1 << 30) + 1, 8)):
        assert L.muon_sort_tokens_workspace_bytes(n, e) == 0


def test_rows_arguments(L):
    def dispatch(x=A, dtype=0, tokens=4, cols=8, ld=8, top_k=2, place=A, offsets=A, groups=3, out=2 * A, ldo=8):
        return L.muon_dispatch_tokens(x, dtype, tokens, cols, ld, top_k, place, offsets, groups, out, ldo, None)

    def combine(y=A, dtype=0, ld=8, tokens=4, cols=8, top_k=2, place=A, offsets=A, groups=3, w=A, out=2 * A, odt=0, ldo=8):
        return L.muon_combine_tokens(y, dtype, ld, tokens, cols, top_k, place, offsets, groups, w, out, odt, ldo, None)

    def back(d=A, ddt=0, ldd=8, y=2 * A, dtype=0, ld=8, tokens=4, cols=8, top_k=2, place=A, offsets=A, groups=3, w=A,
             dy=3 * A, lddy=8, dw=A):
        return L.muon_combine_tokens_backward(d, ddt, ldd, y, dtype, ld, tokens, cols, top_k, place, offsets, groups, w, dy,
                                              lddy, dw, None)

    common = (dict(dtype=2), dict(tokens=-1), dict(tokens=1 << 30), dict(cols=0), dict(cols=(1 << 24) + 1), dict(ld=7),
              dict(top_k=0), dict(top_k=33), dict(place=None), dict(place=A + 2), dict(offsets=None), dict(groups=0),
              dict(groups=1025))
    for call in (dispatch, combine, back):
        for kw in common:
            assert call(**kw) == INVALID, (call.__name__, kw)
        assert call(tokens=0, place=None, offsets=None) == OK
    for kw in (dict(x=None), dict(x=A + 1), dict(out=None), dict(ldo=7)):
        assert dispatch(**kw) == INVALID, kw
    for kw in (dict(y=None), dict(out=None), dict(odt=9), dict(ldo=7), dict(w=A + 2)):
        assert combine(**kw) == INVALID, kw
    for kw in (dict(d=None), dict(ddt=5), dict(ldd=7), dict(y=None), dict(lddy=7), dict(dw=A + 2), dict(w=A + 1),
               dict(dy=2 * A)):
        assert back(**kw) == INVALID, kw
    assert back(dy=None, dw=None) == OK                         # nothing is asked for


def test_swiglu_arguments(L):
    def forward(g=A, ldg=8, u=2 * A, ldu=8, dtype=1, rows=4, cols=8, out=3 * A, ldo=8):
        return L.muon_swiglu(g, ldg, u, ldu, dtype, rows, cols, out, ldo, None)

    for kw in (dict(g=None), dict(g=A + 2), dict(u=None), dict(out=None), dict(ldg=7), dict(ldu=7), dict(ldo=7),
               dict(dtype=4), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(cols=0)):
        assert forward(**kw) == INVALID, kw
    assert forward(g=None, u=None, out=None, rows=0) == OK

    def backward(d=A, ldd=8, g=A, ldg=8, u=2 * A, ldu=8, dtype=0, rows=4, cols=8, dg=3 * A, lddg=8, du=4 * A, lddu=8):
        return L.muon_swiglu_backward(d, ldd, g, ldg, u, ldu, dtype, rows, cols, dg, lddg, du, lddu, None)

    for kw in (dict(d=None), dict(g=None), dict(u=None), dict(dg=None), dict(du=None), dict(ldd=7), dict(lddg=7),
               dict(lddu=7), dict(dtype=-1), dict(rows=-1), dict(cols=0)):
        assert backward(**kw) == INVALID, kw
    assert backward(d=None, g=None, u=None, dg=None, du=None, rows=0) == OK


def test_int4_arguments(L):
    def quantize(w=A, dtype=0, batch=1, rows=4, cols=8, block=32, codes=A, scale=A):
        return L.muon_int4_quantize_weight(w, dtype, batch, rows, cols, block, codes, scale, None)

    for kw in (dict(w=None), dict(w=A + 1), dict(dtype=3), dict(batch=-1), dict(batch=513), dict(rows=0), dict(cols=0),
               dict(block=16), dict(block=256), dict(codes=None), dict(codes=A + 8), dict(scale=None), dict(scale=A + 1)):
        assert quantize(**kw) == INVALID, kw
    assert quantize(batch=0, w=None, codes=None, scale=None) == OK

    def linear(x=A, dtype=0, tokens=4, ld=8, codes=A, scale=A, block=128, n=8, k=8, groups=1, offsets=None, out=2 * A, odt=0,
               ldo=8):
        return L.muon_int4_linear(x, dtype, tokens, ld, codes, scale, block, n, k, groups, offsets, out, odt, ldo, None)

    for kw in (dict(x=None), dict(x=A + 1), dict(dtype=3), dict(tokens=-1), dict(ld=7), dict(codes=None), dict(codes=A + 4),
               dict(scale=None), dict(block=0), dict(n=0), dict(k=0), dict(groups=0), dict(groups=513, offsets=A),
               dict(groups=2), dict(offsets=A + 2), dict(out=None), dict(odt=2), dict(ldo=7)):
        assert linear(**kw) == INVALID, kw
    assert linear(tokens=0, x=None, out=None) == OK
