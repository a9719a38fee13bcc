"""Mixture-of-experts layers on the library's operators, for autograd.

Routing (``route``), the order of the tokens by expert (``plan_tokens``, or
``sort_tokens`` by torch alone), their rows on the way to the experts and back
(``dispatch``, ``combine``), the gated activation (``swiglu``) and linear layers on
8-bit operands (``Fp8Linear`` holds a weight and its codes), for serving on weights of
4 bits (``Int4Linear``): what a layer of experts runs in front of the optimizer step ("Domyn is training
a 1T-parameter MoE on Europe's Jupiter supercomputer, and published the
recipe", table "The model and the machine": 384 experts, 8 chosen).  The
arithmetic runs in the library's kernels; torch supplies memory, the sort and
the graph.  The layers have first derivatives alone: a second one is refused.
"""
import torch

from . import (TokenPlan, muon_combine_tokens, muon_combine_tokens_backward, muon_dispatch_tokens, muon_fp8_linear,
               muon_fp8_linear_backward, muon_fp8_quantize_weight, muon_int4_linear, muon_int4_quantize_weight,
               muon_route, muon_route_backward, muon_sort_tokens, muon_swiglu, muon_swiglu_backward)

__all__ = ["route", "sort_tokens", "plan_tokens", "dispatch", "combine", "swiglu", "Fp8Linear", "Int4Linear"]


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


def plan_tokens(chosen, experts, first=0):
    """``muon_sort_tokens``: where the rows of ``chosen`` (tokens x top_k, of ``route``) lie,
    sorted by expert, for the ``experts`` experts from ``first`` on that are held here."""
    return muon_sort_tokens(chosen, experts, first=first)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, *plan):
        ctx.save_for_backward(*plan)
        return muon_dispatch_tokens(x, TokenPlan(*plan))

    @staticmethod
    def backward(ctx, d):
        with torch.no_grad():
            dx = muon_combine_tokens(d.contiguous(), TokenPlan(*ctx.saved_tensors))
        return _underived(dx, d), None, None, None


def dispatch(x, plan):
    """The tokens' rows sorted by expert (``muon_dispatch_tokens``), with a gradient for x."""
    return _Dispatch.apply(x, *plan)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, out_dtype, *plan):
        ctx.save_for_backward(y, weights, *plan)
        return muon_combine_tokens(y, TokenPlan(*plan), weights, out_dtype=out_dtype)

    @staticmethod
    def backward(ctx, d):
        y, weights, *plan = ctx.saved_tensors
        need_dy, need_dw = ctx.needs_input_grad[:2]
        with torch.no_grad():
            dy, dw = muon_combine_tokens_backward(d.contiguous(), y, TokenPlan(*plan), weights, need_dy=need_dy,
                                                  need_dw=need_dw)
        sources = (d, y) if weights is None else (d, y, weights)
        return (_underived(dy, *sources), _underived(dw, *sources)) + (None,) * 4


def combine(y, plan, weights=None, *, out_dtype=None):
    """The experts' rows back at their tokens, weighted and added up (``muon_combine_tokens``),
    with gradients for y and the weights."""
    return _Combine.apply(y, weights, out_dtype, *plan)


class _Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up):
        ctx.save_for_backward(gate, up)
        return muon_swiglu(gate, up)

    @staticmethod
    def backward(ctx, d):
        gate, up = ctx.saved_tensors
        with torch.no_grad():
            d_gate, d_up = muon_swiglu_backward(d.contiguous(), gate, up)
        return _underived(d_gate, d, gate, up), _underived(d_up, d, gate, up)


class _SwigluJoined(torch.autograd.Function):
    @staticmethod
    def forward(ctx, both):
        ctx.save_for_backward(both)
        return muon_swiglu(*both.chunk(2, -1))

    @staticmethod
    def backward(ctx, d):
        both, = ctx.saved_tensors
        with torch.no_grad():
            d_both = muon_swiglu_backward(d.contiguous(), *both.chunk(2, -1), joined=True)
        return _underived(d_both, d, both)


def swiglu(gate, up=None):
    """gate / (1 + exp(-gate)) * up (``muon_swiglu``) with gradients for both; without ``up``
    gate holds both, rows x 2 cols, gate before up, as one product makes them."""
    if up is not None:
        return _Swiglu.apply(gate, up)
    if gate.dim() != 2 or gate.shape[1] % 2:
        raise ValueError("without up, gate must have an even number of columns: gate's, then up's")
    return _SwigluJoined.apply(gate)


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


class Int4Linear:
    """A weight (out x in, or stacked over experts) in 4 bits, for serving: ``layer(x,
    offsets)`` is x W^T in x's type.  There are no gradients: neither for the weight, of which
    the codes alone are kept, nor for x.  ``layer.update(weight)`` puts another weight of the
    shape in its place, in the memory that is there: graphs captured of the layer go on with it."""

    def __init__(self, weight, block=128):
        with torch.no_grad():
            self.codes = muon_int4_quantize_weight(weight.detach(), block)

    @torch.no_grad()
    def update(self, weight):
        new = muon_int4_quantize_weight(weight.detach(), self.codes.block)
        if new.cols != self.codes.cols or new.codes.shape != self.codes.codes.shape:
            raise ValueError("the weight must be of the shape that the layer was made with")
        self.codes.codes.copy_(new.codes)
        self.codes.scale.copy_(new.scale)

    def __call__(self, x, offsets=None):
        if torch.is_grad_enabled() and x.requires_grad:
            raise RuntimeError("a layer of 4 bits has no gradients: call it under torch.no_grad()")
        return muon_int4_linear(x, self.codes, offsets=offsets, out_dtype=x.dtype)
