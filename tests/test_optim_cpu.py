"""MuonAdamW's options outlive copies, pickles and saved state, without a GPU."""
import copy
import pickle

import torch

from muon_newton_schulz_step_gb300 import optim
from muon_newton_schulz_step_gb300.optim import MuonAdamW


def make(**kw):
    return MuonAdamW([torch.nn.Parameter(torch.zeros(4, 4))], **kw)


def test_copies_and_pickles_keep_the_clipping():
    for again in (copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))):
        a = again(make(max_grad_norm=0.5))
        assert a.max_grad_norm == 0.5 and a.grad_norm is None
        b = again(make())
        assert b.max_grad_norm is None
        assert b.step() is None                          # no gradients: nothing to launch


def test_a_copy_clips(monkeypatch):
    calls = []
    monkeypatch.setattr(optim, "muon_grad_clip", lambda G, max_norm: calls.append((len(G), max_norm)) or torch.tensor(2.0))
    monkeypatch.setattr(optim, "muon_step_ex", lambda *a, **kw: None)
    a = copy.deepcopy(make(max_grad_norm=0.25))
    for p in a.param_groups[0]["params"]:
        p.grad = torch.ones_like(p)
    a.step()
    assert calls == [(1, 0.25)] and float(a.grad_norm) == 2.0
    b = pickle.loads(pickle.dumps(a))
    assert b.max_grad_norm == 0.25 and float(b.grad_norm) == 2.0


def test_pickles_from_before_the_option_step_without_it():
    old = make()
    state = old.__getstate__()
    for name in ("max_grad_norm", "grad_norm"):
        state.pop(name, None)
    new = MuonAdamW.__new__(MuonAdamW)
    new.__setstate__(state)
    assert new.max_grad_norm is None and new.step() is None
