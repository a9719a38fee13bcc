"""The short allocation is found good by the first result, and serves from then on."""
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg

pytestmark = pytest.mark.gpu


def test_first_result_tries_the_short_allocation(monkeypatch):
    a = torch.randn(3, 5, device="cuda")
    want = mg.muon_swiglu(a, a)
    monkeypatch.setattr(mg, "_allocate", mg._first_allocation)
    assert torch.equal(mg.muon_swiglu(a, a), want)
    assert mg._allocate is mg._empty_strided
    monkeypatch.setattr(mg, "_empty_strided", lambda sizes, strides: None)
    monkeypatch.setattr(mg, "_allocate", mg._first_allocation)
    assert torch.equal(mg.muon_swiglu(a, a), want) and mg._allocate is None
    assert torch.equal(mg.muon_swiglu(a, a), want)
