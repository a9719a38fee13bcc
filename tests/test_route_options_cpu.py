"""Routing options reach the kernel by value, whatever carries them."""
import torch

import muon_newton_schulz_step_gb300 as mg


def options(top_k=8, groups=1, top_groups=None, renormalize=True, scale=1.0):
    o, _ = mg._route_opts(top_k, "softmax", groups, top_groups, renormalize, scale)
    return o.top_k, o.groups, o.top_groups, o.renormalize, o.scale


def test_a_scale_changed_in_place_is_seen():
    scale = torch.tensor(1.0)
    assert options(scale=scale) == (8, 1, 1, 1, 1.0)
    scale.mul_(3.0)
    assert options(scale=scale) == (8, 1, 1, 1, 3.0)


def test_counts_and_flags_changed_in_place_are_seen():
    k, on = torch.tensor(4), torch.tensor(True)
    assert options(top_k=k, groups=k, renormalize=on) == (4, 4, 4, 1, 1.0)
    k.fill_(2)
    on.fill_(False)
    assert options(top_k=k, groups=k, renormalize=on) == (2, 2, 2, 0, 1.0)


def test_the_same_values_share_their_options():
    assert mg._route_opts(8, "sigmoid", 4, 2, True, 2.5)[0] is mg._route_opts(8, "sigmoid", 4, 2, True, 2.5)[0]


def test_the_gradient_takes_the_scale_of_its_forward(monkeypatch):
    """Kernels replaced by stand-ins: what counts is the scale that each call receives."""
    from muon_newton_schulz_step_gb300 import experts

    seen = []

    def forward(logits, top_k, *, scale, **kw):
        seen.append(float(scale))
        return logits[:, :top_k] * 1.0, torch.zeros(len(logits), top_k, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)

    def backward(d, logits, chosen, *, scale, **kw):
        seen.append(float(scale))
        return torch.zeros_like(logits)

    monkeypatch.setattr(experts, "muon_route", forward)
    monkeypatch.setattr(experts, "muon_route_backward", backward)
    scale = torch.tensor(1.0)
    w, _, _ = experts.route(torch.zeros(3, 4, requires_grad=True), 2, scale=scale)
    scale.mul_(3.0)
    w.sum().backward()
    assert seen == [1.0, 1.0]
