"""Where torch's short allocation is missing, fails or gives something else, results come from torch.empty."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
asked = []
empty = torch.empty
def recorded(*a, device=None, **kw):
    asked.append(device)
    return empty(*a, **kw)
def refuses(sizes, strides, dtype, device):             # another signature
    raise AssertionError("never called")
def on_the_host(sizes, strides, dtype):
    return torch.zeros(sizes, dtype=dtype)
guards = torch._C._dynamo.guards
if %(how)r == "None":
    if hasattr(guards, "_empty_strided_cuda"):
        del guards._empty_strided_cuda
else:
    guards._empty_strided_cuda = %(how)s
import muon_newton_schulz_step_gb300 as mg
torch.empty = recorded
for _ in range(2):
    t, v = mg._new_rows(5, 7, torch.float32), mg._new_vector(9, torch.int32)
    assert t.shape == (5, 7) and t.dtype == torch.float32 and v.shape == (9,) and v.dtype == torch.int32
assert asked == ["cuda"] * 4, asked
print("allocated")
"""


@pytest.mark.parametrize("how", ["None", "refuses", "on_the_host"])
def test_results_come_from_torch_empty(how):
    r = subprocess.run([sys.executable, "-c", PROGRAM % {"how": how}], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "allocated" in r.stdout, r.stderr[-2000:]
