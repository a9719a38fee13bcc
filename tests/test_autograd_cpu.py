"""The experts' layers refuse a second derivative, which their kernels do not have.

The kernels are replaced by stand-ins on the CPU that, as the kernels do, return
gradients without a graph of their own."""
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg
from muon_newton_schulz_step_gb300 import experts


@pytest.fixture
def layers(monkeypatch):
    def route(logits, top_k, **kw):
        return logits.detach()[:, :top_k] ** 2, torch.arange(top_k, dtype=torch.int32).expand(len(logits), -1), \
            torch.full((logits.shape[1],), len(logits), dtype=torch.int32)

    def route_backward(d, logits, chosen, **kw):
        g = torch.zeros_like(logits).detach()
        g[:, :d.shape[1]] = (2 * logits[:, :d.shape[1]] * d).detach()
        return g

    def linear(x, w, offsets=None, out_dtype=None):
        return x.detach() @ w.codes.t()

    def linear_backward(dy, x, w, offsets=None, **kw):
        return dy.detach() @ w.codes, dy.detach().t() @ x.detach()

    monkeypatch.setattr(experts, "muon_route", route)
    monkeypatch.setattr(experts, "muon_route_backward", route_backward)
    monkeypatch.setattr(experts, "muon_fp8_linear", linear)
    monkeypatch.setattr(experts, "muon_fp8_linear_backward", linear_backward)
    monkeypatch.setattr(experts, "muon_fp8_quantize_weight",
                        lambda w: mg.Fp8Matrix(w.clone(), torch.ones(1), "block", w.shape[1]))
    return experts


def of_route(layers, x):
    return layers.route(x, 2)[0]


def of_linear(layers, x):
    return layers.Fp8Linear(torch.ones(3, 4, requires_grad=True))(x)


@pytest.mark.parametrize("layer", [of_route, of_linear])
def test_second_derivative_is_refused(layers, layer):
    x = torch.randn(5, 4, requires_grad=True)
    g, = torch.autograd.grad((layer(layers, x) ** 2).sum() + (x ** 3).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives"):
        torch.autograd.grad(g.sum(), x)


def test_mixed_second_derivative_of_a_weight_is_refused(layers):
    x = torch.randn(5, 4, requires_grad=True)
    lin = layers.Fp8Linear(torch.ones(3, 4, requires_grad=True))
    dx, = torch.autograd.grad(lin(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives"):
        torch.autograd.grad((dx ** 2).sum() + (lin.weight ** 2).sum(), lin.weight)
    dw, = torch.autograd.grad(lin(x).sum(), lin.weight, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives"):
        torch.autograd.grad((dw ** 2).sum() + (x ** 2).sum(), x)


@pytest.mark.parametrize("layer", [of_route, of_linear])
def test_first_derivative_is_the_same_with_a_graph(layers, layer):
    x = torch.randn(5, 4, requires_grad=True)
    a, = torch.autograd.grad((layer(layers, x) ** 2).sum(), x, create_graph=True)
    b, = torch.autograd.grad((layer(layers, x) ** 2).sum(), x)
    assert torch.equal(a.detach(), b)
