"""The operators together: a mixture-of-experts layer and its training step."""
import math
import os
import sys

import pytest
import torch

import muon_newton_schulz_step_gb300 as mg
from muon_newton_schulz_step_gb300 import experts
from muon_newton_schulz_step_gb300.optim import MuonAdamW

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
DEV = "cuda"


def layer_reference(layer, h):
    """The same layer without rounding to 8 bits, expert by expert, in fp32."""
    logits = h @ layer.router.t()
    s = torch.sigmoid(logits)
    with torch.no_grad():
        _, chosen, _ = mg.muon_route(logits.detach(), layer.top_k, bias=layer.bias, score="sigmoid", groups=layer.groups,
                                     top_groups=layer.top_groups)
    w = s.gather(1, chosen.long())
    w = w / w.sum(1, keepdim=True)
    out = torch.zeros_like(h)
    for e in range(layer.router.shape[0]):
        t, k = (chosen == e).nonzero(as_tuple=True)
        x = h[t]
        a = torch.nn.functional.silu(x @ layer.gate.weight[e].float().t()) * (x @ layer.up.weight[e].float().t())
        out = out.index_add(0, t, (a @ layer.down.weight[e].float().t()) * w[t, k, None])
    return out


def test_layer_and_gradients_are_near_the_unrounded_ones():
    """E4M3 keeps 3 bits of fraction: an operand is off by at most 2^-4 of itself,
    2^-4 / sqrt(3) in the mean square at worst (4 % measured on normal data for one
    operand).  A result of two rounded operands is then off by at most
    2 * 2^-4 / sqrt(3) = 7.3 % in the 2-norm, three products in a row by 22 %."""
    import moe_layer_step

    layer = moe_layer_step.MoeLayer(seed=3)
    h = torch.randn(300, 512, device=DEV).to(torch.bfloat16)
    out, counts = layer(h)
    assert int(counts.sum()) == 300 * layer.top_k
    d = torch.randn_like(out)
    out.backward(d)
    got = [layer.router.grad] + [w.weight.grad.float() for w in layer.layers]
    layer.router.grad = None
    for w in layer.layers:
        w.weight.grad = None
    ref = layer_reference(layer, h.float())
    ref.backward(d)
    want = [layer.router.grad] + [w.weight.grad.float() for w in layer.layers]
    assert float((out.detach() - ref.detach()).norm() / ref.detach().norm()) < 0.22
    for a, b in zip(got, want):
        assert float((a - b).norm() / b.norm()) < 0.22


def test_training_steps_reduce_the_loss():
    import moe_layer_step

    losses, norms = moe_layer_step.train(steps=12, tokens=512)
    assert all(math.isfinite(v) for v in losses + norms)
    assert losses[-1] < 0.8 * losses[0]
    assert mg.muon_device_status() == 0


def test_tokens_without_an_expert_pass_nothing():
    logits = torch.randn(40, 8, device=DEV)
    logits[::4] = -math.inf                              # every fourth token is padding
    w, chosen, counts = experts.route(logits, 2)
    order, offsets = experts.sort_tokens(chosen, counts)
    assert offsets.tolist()[0] == 20 and offsets.tolist()[-1] == 80
    flat = chosen.reshape(-1)[order]
    assert bool((flat[:20] == -1).all()) and bool((flat[20:].diff() >= 0).all())
    x = torch.randn(80, 128, device=DEV).to(torch.bfloat16).requires_grad_(True)
    lin = experts.Fp8Linear(torch.randn(8, 64, 128, device=DEV).to(torch.bfloat16).requires_grad_(True))
    y = lin(x, offsets)
    y.backward(torch.ones_like(y))
    assert int(torch.count_nonzero(y[:20])) == 0 and int(torch.count_nonzero(x.grad[:20])) == 0
    assert int(torch.count_nonzero(y[20:])) > 0
    assert bool(torch.isfinite(lin.weight.grad).all())


def test_optimizer_clips_by_the_global_norm():
    torch.manual_seed(1)
    shapes = [(64, 128), (96,), (300, 200)]
    ps = [torch.nn.Parameter(torch.randn(s, device=DEV)) for s in shapes]
    qs = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    grads = [torch.randn(s, device=DEV) for s in shapes]
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    a = MuonAdamW([{"params": ps}], max_grad_norm=0.5)
    b = MuonAdamW([{"params": qs}])
    for p, q, g in zip(ps, qs, grads):
        p.grad = g.clone()
        q.grad = g * (0.5 / (norm + 1e-6))
    a.step()
    b.step()
    assert abs(float(a.grad_norm) - norm) <= 1e-5 * norm and b.grad_norm is None
    for p, q, g, s in zip(ps, qs, grads, shapes):
        # the factor is off by 1e-5 at most; Muon and AdamW do not change with the gradient's size
        assert float((p.grad - q.grad).norm()) <= 2e-5 * float(q.grad.norm())
        assert float((p - q).detach().norm()) <= 2e-3 * float(q.detach().norm())
