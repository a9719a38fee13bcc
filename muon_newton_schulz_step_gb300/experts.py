"""Mixture-of-experts layers on the library's operators, for autograd.

Routing (``route``), the order of the tokens by expert (``sort_tokens``) and
linear layers on 8-bit operands (``Fp8Linear`` holds a weight and its codes):
what a layer of experts runs in front of the optimizer step ("Domyn is training
a 1T-parameter MoE on Europe's Jupiter supercomputer, and published the
recipe", table "The model and the machine": 384 experts, 8 chosen).  The
arithmetic runs in the library's kernels; torch supplies memory, the sort and
the graph.  The layers have first derivatives alone: a second one is refused.
"""
import torch

from . import (muon_fp8_linear, muon_fp8_linear_backward, muon_fp8_quantize_weight, muon_route,
               muon_route_backward)

__all__ = ["route", "sort_tokens", "Fp8Linear"]


class _Underived(torch.autograd.Function):
    """A gradient as it is, made of ``sources`` by kernels that have no derivative:
    going back through it is an error.  (torch's ``once_differentiable`` does not tie
    the gradient to its sources, and ``torch.autograd.grad`` then leaves this path out
    without a word.)"""

    @staticmethod
    def forward(ctx, grad, *sources):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the experts' layers have first derivatives alone: no gradient of their gradients")


def _underived(grad, *sources):
    """``grad`` of ``sources``; without create_graph nothing to do."""
    return grad if grad is None or not torch.is_grad_enabled() else _Underived.apply(grad, *sources)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, top_k, score, groups, top_groups, renormalize, scale):
        weights, chosen, counts = muon_route(logits, top_k, bias=bias, score=score, groups=groups,
                                             top_groups=top_groups, renormalize=renormalize, scale=scale)
        ctx.save_for_backward(logits, chosen)
        ctx.how = dict(score=score, renormalize=renormalize, scale=scale)
        ctx.mark_non_differentiable(chosen, counts)
        return weights, chosen, counts

    @staticmethod
    def backward(ctx, d_weights, _chosen, _counts):
        logits, chosen = ctx.saved_tensors
        with torch.no_grad():
            d = muon_route_backward(d_weights.contiguous(), logits, chosen, **ctx.how)
        return (_underived(d, d_weights, logits),) + (None,) * 7


def route(logits, top_k, *, bias=None, score="softmax", groups=1, top_groups=None, renormalize=True, scale=1.0):
    """``muon_route`` with a gradient for the logits: (weights, chosen experts,
    tokens of each expert).  The bias steers the choice and gets no gradient."""
    return _Route.apply(logits, bias, top_k, score, groups, top_groups, bool(renormalize), float(scale))


def sort_tokens(chosen, counts):
    """The places of ``chosen`` (tokens x top_k) sorted by expert, and the
    experts' offsets among them (int32, experts + 1): place p of the result
    holds entry order[p], that is token order[p] // top_k.  Entries without an
    expert (-1) come first and belong to no group."""
    order = torch.argsort(chosen.reshape(-1), stable=True)
    ends = torch.cumsum(counts, 0, dtype=torch.int32)
    first = order.numel() - ends[-1:]
    return order, torch.cat([first, first + ends]).to(torch.int32)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, codes, offsets):
        ctx.save_for_backward(x, offsets)
        ctx.codes = codes
        ctx.weight = weight
        return muon_fp8_linear(x, codes, offsets=offsets, out_dtype=x.dtype)

    @staticmethod
    def backward(ctx, dy):
        x, offsets = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[:2]
        with torch.no_grad():
            dx, dw = muon_fp8_linear_backward(dy.contiguous(), x, ctx.codes, offsets=offsets, need_dx=need_dx,
                                              need_dw=need_dw, dx_dtype=x.dtype, dw_dtype=ctx.weight.dtype)
        return _underived(dx, dy, ctx.weight), _underived(dw, dy, x), None, None


class Fp8Linear:
    """A linear layer's weight (out x in, or stacked over experts) and its 8-bit
    codes.  ``layer(x, offsets)`` is x W^T with gradients for both;
    ``layer.update()`` makes the codes anew after a step changed the weight."""

    def __init__(self, weight):
        self.weight = weight
        self.codes = None
        self.update()

    @torch.no_grad()
    def update(self):
        self.codes = muon_fp8_quantize_weight(self.weight.detach())

    def __call__(self, x, offsets=None):
        return _Linear.apply(x, self.weight, self.codes, offsets)
