"""Every operator around the step is captured in a CUDA graph by the first call
of it that a process makes (nothing warmed up), and the replay gives what a call gives."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import torch
import muon_newton_schulz_step_gb300 as mg
gen = torch.Generator(device="cuda").manual_seed(7)
def randn(*shape): return torch.randn(*shape, generator=gen, device="cuda")
def bf(*shape): return randn(*shape).to(torch.bfloat16)
"""
CALLS = {
    "route": ("x = randn(20000, 384); run = lambda: mg.muon_route(x, 8, score='sigmoid', groups=8, top_groups=4)"),
    "route_backward": ("x, d = randn(700, 100), randn(700, 4)\n"
                       "c = torch.arange(2800, device='cuda', dtype=torch.int32).reshape(700, 4) % 100\n"
                       "run = lambda: (mg.muon_route_backward(d, x, c, renormalize=False),)"),
    "quantize": "x = bf(300, 700); run = lambda: sum((tuple(m[:2]) for m in mg.muon_fp8_quantize(x, col=True)), ())",
    "weight": "x = bf(3, 300, 700); run = lambda: mg.muon_fp8_quantize_weight(x)[:2]",
    "linear": ("x, w = bf(600, 700), bf(500, 700)\n"
               "run = lambda: (mg.muon_fp8_linear(x, mg.muon_fp8_quantize_weight(w)),)"),
    "linear_backward": ("x, dy, w = bf(600, 700), bf(600, 500), bf(500, 700)\n"
                        "run = lambda: mg.muon_fp8_linear_backward(dy, x, mg.muon_fp8_quantize_weight(w))"),
    "norm": "G = [bf(300, 700), randn(901)]; run = lambda: (mg.muon_grad_norm(G),)",
    "clip": ("G = [bf(300, 700), randn(901)]; O = [torch.empty_like(g) for g in G]\n"
             "run = lambda: (mg.muon_grad_clip(G, 0.5, out=O), *O)"),
}
TAIL = """
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
got = [t.reshape(-1).view(torch.uint8).clone() for t in out]
for a, b in zip(got, run()):
    assert torch.equal(a, b.reshape(-1).view(torch.uint8))
assert mg.muon_device_status() == 0
print("captured")
"""


@pytest.mark.parametrize("name", list(CALLS))
def test_first_call_is_captured(name):
    r = subprocess.run([sys.executable, "-c", HEAD + CALLS[name] + TAIL], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
