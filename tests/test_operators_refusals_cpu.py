"""What is no 8-bit weight is refused by name, before anything of it is used; no GPU."""
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg


def weight():
    return mg.Fp8Matrix(torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(1, 1, dtype=torch.uint8), "block", 8)


@pytest.mark.parametrize("bad", [None, torch.zeros(4, 8), (1, 2, "block", 8), weight()._replace(codes=None),
                                 weight()._replace(scale=[0])])
def test_what_is_no_weight_is_refused(bad):
    x = torch.zeros(4, 8)
    for call in (lambda: mg.muon_fp8_linear(x, bad), lambda: mg.muon_fp8_linear_backward(x, x, bad),
                 lambda: mg.muon_fp8_product("forward", bad, bad), lambda: mg.muon_fp8_product("grad_input", bad, bad),
                 lambda: mg.muon_fp8_product("grad_weight", bad, bad, tokens=4)):
        with pytest.raises(ValueError):
            call()
