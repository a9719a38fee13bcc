"""Refusals of the operators around the step, without a GPU: the binding refuses
host tensors and wrong types, the C ABI bad sizes, options and pointers (fake
addresses: validation reads none)."""
import ctypes
import math

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
    x = torch.zeros(4, 8)
    for call in (lambda: mg.muon_grad_norm([x]), lambda: mg.muon_grad_clip([x], 1.0), lambda: mg.muon_route(x, 2),
                 lambda: mg.muon_route_backward(x, x, x), lambda: mg.muon_fp8_quantize(x),
                 lambda: mg.muon_fp8_quantize_weight(x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    for bad in (3, None, [1.0]):
        with pytest.raises(ValueError, match="CUDA tensor"):
            mg.muon_grad_norm([bad])
    w = mg.Fp8Matrix(torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(1, 1, dtype=torch.uint8), "block", 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mg.muon_fp8_linear(x, w)
    with pytest.raises(ValueError, match='kind "block"'):
        mg.muon_fp8_linear(x, w._replace(kind="row"))
    with pytest.raises(ValueError, match="stacked weight"):
        mg.muon_fp8_linear(x, w, offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="score"):
        mg._route_opts(2, "relu", 1, 1, True, 1.0)


def test_scores_and_sizes_of_scratch(L):
    assert [mg.muon_fp8_padded_rows(r, g) for r, g in ((0, 3), (1, 1), (128, 1), (129, 1), (200, 3), (2, 100))] == \
        [0, 128, 256, 256, 512, 256]
    n = (ctypes.c_longlong * 3)(5, 0, 1 << 33)
    assert L.muon_grad_norm_workspace_bytes(n, 3) >= 8
    assert L.muon_grad_norm_workspace_bytes((ctypes.c_longlong * 1)(-1), 1) == 0
    # enough for the codes and scales, whatever the alignment inside
    for t, k in ((9, 1), (100, 129), (8192, 6144)):
        assert L.muon_fp8_linear_workspace_bytes(t, 6144, k, 0) >= t * (k + k / 128)
    assert L.muon_fp8_linear_workspace_bytes(1, 6144, 6144, 0) == 0
    assert L.muon_fp8_linear_workspace_bytes(1, 6144, 6144, 1) > 0
    assert L.muon_fp8_linear_backward_workspace_bytes(100, 64, 32, 4, 0, 0) == 0


def test_gradient_norm_arguments(L):
    vp = ctypes.c_void_p
    G, n, d = (vp * 1)(A), (ctypes.c_longlong * 1)(100), (ctypes.c_int * 1)(1)

    def norm(G=G, n=n, d=d, count=1, ws=A, wsb=1 << 20, out=A):
        return L.muon_grad_norm(G, n, d, count, ws, wsb, out, None)

    assert norm(count=-1) == INVALID
    assert norm(G=None) == INVALID
    assert norm(out=None) == INVALID
    assert norm(n=(ctypes.c_longlong * 1)(-5)) == INVALID
    assert norm(d=(ctypes.c_int * 1)(7)) == INVALID
    assert norm(G=(vp * 1)(0)) == INVALID
    assert norm(G=(vp * 1)(A + 2)) == INVALID                # fp32 at 2 bytes
    assert norm(ws=None) == INVALID
    assert norm(wsb=8) == OOM
    for bad in (-1.0, math.nan, math.inf):
        assert L.muon_grad_clip(G, None, n, d, 1, bad, A, 1 << 20, A, None) == INVALID
    assert b"max_norm" in L.muon_last_error()


def test_route_arguments(L):
    def route(logits=A, dtype=1, tokens=4, experts=16, ld=16, weights=A, chosen=A, counts=A, **opts):
        o = mg._RouteOpts()
        L.muon_route_opts_init(ctypes.byref(o))
        assert (o.top_k, o.groups, o.top_groups, o.score, o.renormalize, o.scale) == (1, 1, 1, 0, 1, 1.0)
        for k, v in opts.items():
            setattr(o, k, v)
        return L.muon_route(logits, dtype, tokens, experts, ld, None, ctypes.byref(o), weights, chosen, counts, None)

    for kw in (dict(dtype=3), dict(tokens=-1), dict(ld=15), dict(logits=None), dict(logits=A + 2), dict(weights=None),
               dict(chosen=None), dict(counts=None), dict(top_k=0), dict(top_k=17), dict(groups=3), dict(groups=0),
               dict(groups=4, top_groups=5), dict(groups=8, top_groups=1, top_k=3), dict(score=2), dict(renormalize=2),
               dict(scale=math.inf)):
        assert route(**kw) == INVALID, kw
    assert route(experts=0) == UNSUPPORTED and route(experts=1025, ld=1025) == UNSUPPORTED
    # 31 groups leave one lane each, and a lane holds 32 experts
    assert route(experts=31 * 33, ld=31 * 33, groups=31, top_groups=31) == UNSUPPORTED
    assert L.muon_route(A, 1, 4, 16, 16, None, None, A, A, A, None) == INVALID


def test_fp8_arguments(L):
    q = L.muon_fp8_quantize
    assert q(A, 1, -1, 8, 8, 1, None, A, A, None, None, None) == INVALID
    assert q(A, 1, 4, 0, 8, 1, None, A, A, None, None, None) == INVALID
    assert q(A, 1, 4, 8, 7, 1, None, A, A, None, None, None) == INVALID
    assert q(A, 1, 4, 8, 8, 0, None, A, A, None, None, None) == INVALID
    assert q(A, 1, 4, 8, 8, 513, A, A, A, None, None, None) == INVALID
    assert q(A, 1, 4, 8, 8, 2, None, A, A, None, None, None) == INVALID     # two groups without offsets
    assert q(A, 1, 4, 8, 8, 1, None, None, None, None, None, None) == INVALID
    assert q(A, 1, 4, 8, 8, 1, None, A, None, None, None, None) == INVALID
    assert q(A, 1, 4, 8, 8, 1, None, A + 8, A, None, None, None) == INVALID
    assert q(A + 2, 1, 4, 8, 8, 1, None, A, A, None, None, None) == INVALID
    assert q(A, 1, 0, 8, 8, 1, None, None, None, None, None, None) == OK     # no rows: nothing to do
    p = L.muon_fp8_product
    assert p(5, A, A, A, A, 4, 8, 8, 1, None, A, 0, 8, None) == INVALID
    assert p(0, A, A, A, A, 4, 8, 8, 1, None, A, 0, 7, None) == INVALID
    assert p(0, A, A, A, A, 4, 8, 8, 1, None, None, 0, 8, None) == INVALID
    assert p(0, A + 1, A, A, A, 4, 8, 8, 1, None, A, 0, 8, None) == INVALID
    assert p(0, A, None, A, A, 4, 8, 8, 1, None, A, 0, 8, None) == INVALID
    assert p(2, A, A + 1, A, A, 4, 8, 8, 1, None, A, 0, 8, None) == INVALID
    assert p(0, A, A, A, A, 4, 1 << 25, 8, 1, None, A, 0, 1 << 25, None) == INVALID
    assert p(0, None, None, None, None, 0, 8, 8, 1, None, A, 0, 8, None) == OK
    lin = L.muon_fp8_linear
    assert lin(A, 0, 4, 7, A, A, 8, 8, 1, None, None, 0, A, 0, 8, None) == INVALID
    assert lin(A, 0, 4, 8, A, A, 8, 8, 1, None, None, 0, A, 0, 7, None) == INVALID
    assert lin(A, 0, 4, 8, None, A, 8, 8, 1, None, None, 0, A, 0, 8, None) == INVALID
    assert lin(A, 0, 100, 8, A, A, 8, 8, 1, None, None, 0, A, 0, 8, None) == INVALID      # no workspace
    assert lin(A, 0, 100, 8, A, A, 8, 8, 1, None, A, 64, A, 0, 8, None) == OOM
    assert lin(None, 0, 0, 8, A, A, 8, 8, 1, None, None, 0, None, 0, 8, None) == OK
    w = L.muon_fp8_quantize_weight
    assert w(A, 1, -1, 8, 8, A, A, None) == INVALID and w(A, 1, 1, 8, 8, A, None, None) == INVALID
    assert w(A, 1, 0, 8, 8, None, None, None) == OK
