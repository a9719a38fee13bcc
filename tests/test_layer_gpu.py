"""The operators between an expert layer's routing and its result, together: for
autograd, as a training layer, as a layer that serves single tokens on weights of 4
bits, on streams and in CUDA graphs."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import muon_newton_schulz_step_gb300 as mg
from muon_newton_schulz_step_gb300 import experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = 2.0 ** -8                                     # half a step of bf16, relative
U = 2.0 ** -24


def routed(tokens, count, top_k, seed=0, masked=True):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    logits = torch.randn(tokens, count, generator=gen, device=DEV)
    if masked:
        logits[::7] = -float("inf")                  # padding
    weights, chosen, _ = mg.muon_route(logits, top_k)
    return weights, chosen


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_are_the_operators(dtype):
    weights, chosen = routed(100, 12, 3)
    plan = experts.plan_tokens(chosen, 8, 2)
    h = torch.randn(100, 48, device=DEV).to(dtype).requires_grad_(True)
    w = weights.clone().requires_grad_(True)
    x = experts.dispatch(h, plan)
    a = experts.swiglu(x)
    y = experts.swiglu(x[:, :24], x[:, 24:])
    assert torch.equal(a, y)
    out = experts.combine(a, plan, w, out_dtype=torch.float32)
    d = torch.randn_like(out)
    out.backward(d)
    da, dw = mg.muon_combine_tokens_backward(d, a.detach(), plan, weights)
    dx = mg.muon_swiglu_backward(da, x.detach()[:, :24], x.detach()[:, 24:], joined=True)
    assert torch.equal(w.grad, dw)
    assert torch.equal(h.grad, mg.muon_combine_tokens(dx, plan)) and h.grad.dtype == dtype
    # the two-argument form through autograd's own slices
    h2 = h.detach().clone().requires_grad_(True)
    x2 = experts.dispatch(h2, plan)
    experts.combine(experts.swiglu(x2[:, :24], x2[:, 24:]), plan, w.detach(), out_dtype=torch.float32).backward(d)
    assert torch.equal(h2.grad, h.grad)


def test_gradients_that_are_views_and_sums():
    weights, chosen = routed(40, 6, 2)
    plan = experts.plan_tokens(chosen, 6)
    h = torch.randn(40, 32, device=DEV, requires_grad=True)
    experts.combine(experts.dispatch(h, plan), plan, weights).sum().backward()     # an expanded gradient
    held = (plan.place >= plan.offsets[0]).float()
    want = (weights * held).sum(1, keepdim=True).expand(-1, 32)
    # two weights of at most 1, added after a rounding each
    assert ((h.grad - want).abs() <= 4 * U).all()
    h.grad = None
    experts.combine(experts.dispatch(h, plan), plan).t().backward(torch.ones(32, 40, device=DEV))
    assert torch.equal(h.grad, held.sum(1, keepdim=True).expand(-1, 32))


def test_second_derivatives_and_gradients_of_4_bits_are_refused():
    weights, chosen = routed(20, 6, 2, masked=False)
    plan = experts.plan_tokens(chosen, 6)
    h = torch.randn(20, 32, device=DEV, requires_grad=True)
    w = weights.clone().requires_grad_(True)
    out = experts.combine(experts.swiglu(experts.dispatch(h, plan)), plan, w)
    g, = torch.autograd.grad(out.square().sum(), h, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives alone"):
        g.sum().backward()
    layer = experts.Int4Linear(torch.randn(16, 32, device=DEV))
    with pytest.raises(RuntimeError, match="no gradients"):
        layer(h)
    with torch.no_grad():
        assert layer(h).dtype == torch.float32
    assert layer(h.detach()).shape == (20, 16)
    with pytest.raises(ValueError, match="even number"):
        experts.swiglu(torch.randn(3, 5, device=DEV))


def test_training_layer_by_kernels():
    """The bounds of the layer by torch hold: the kernels round less."""
    import moe_layer_step
    from tests.test_experts_gpu import layer_reference

    layer = moe_layer_step.MoeLayer(seed=3, fused=True)
    h = torch.randn(300, 512, device=DEV).to(torch.bfloat16)
    out, counts = layer(h)
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
    losses, norms = moe_layer_step.train(steps=3, tokens=200, fused=True)
    assert all(v == v and abs(v) < float("inf") for v in losses + norms)
    assert mg.muon_device_status() == 0


def values(m):
    c = m.codes.to(torch.int64)
    q = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    q = torch.where(q > 7, q - 16, q).double()
    return (q * m.scale.double().transpose(-1, -2).repeat_interleave(m.block, -1))[..., :m.cols]


@pytest.mark.parametrize("tokens", [1, 2, 9])
def test_serving_layer_stage_by_stage(tokens):
    """Each stage against 64 bits from what the stage before it gave."""
    import moe_layer_step

    layer = moe_layer_step.MoeLayer(seed=5)
    h = torch.randn(tokens, 512, device=DEV).to(torch.bfloat16)
    out = layer.serve(h)
    gate_up, down = layer.served
    weights, chosen, _ = mg.muon_route(h.float() @ layer.router.detach().t(), layer.top_k, bias=layer.bias,
                                       score="sigmoid", groups=layer.groups, top_groups=layer.top_groups)
    plan = experts.plan_tokens(chosen, 16)
    x = mg.muon_dispatch_tokens(h, plan)
    both = gate_up(x, plan.offsets)
    a = mg.muon_swiglu(both[:, :256], both[:, 256:])
    y = down(a, plan.offsets)
    for p in range(tokens * layer.top_k):
        entry = int(plan.order[p])
        e = int(chosen.reshape(-1)[entry])
        assert int(plan.offsets[e]) <= p < int(plan.offsets[e + 1])
        assert torch.equal(x[p], h[entry // layer.top_k])
        for v, m, r in ((x, gate_up.codes, both), (a, down.codes, y)):
            w = values(m)[e]
            want, size = w @ v[p].double(), w.abs() @ v[p].double().abs()
            # sums as in the products' own test, then half a step of bf16
            off = (m.block / 16 * 17 * 2 * U + (m.cols / m.block + 10) * U + U) * size
            assert ((r[p].double() - want).abs() <= off + HALF * (want.abs() + off)).all()
    g, u = both[:, :256].double(), both[:, 256:].double()
    want = g * torch.sigmoid(g) * u
    off = want.abs() * ((2 + 1.173 * g.abs()) * 2 * U + 7 * U)
    assert ((a.double() - want).abs() <= off + HALF * (want.abs() + off) + 2.0 ** -126).all()
    rows = y.double()[plan.place.long()] * weights.double()[..., None]
    assert ((out.double() - rows.sum(1)).abs() <= layer.top_k * U * rows.abs().sum(1)).all()


def test_serving_layer_in_a_graph_with_new_tokens():
    import moe_layer_step

    layer = moe_layer_step.MoeLayer(seed=6)
    h = torch.randn(3, 512, device=DEV).to(torch.bfloat16)
    layer.serve(h)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.serve(h)
    torch.cuda.current_stream().wait_stream(s)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    other = torch.randn(3, 512, device=DEV).to(torch.bfloat16)
    with torch.cuda.graph(one):
        a = layer.serve(h)
    with torch.cuda.graph(two):
        b = layer.serve(other)
    for _ in range(3):
        h.copy_(torch.randn(3, 512, device=DEV))
        other.copy_(torch.randn(3, 512, device=DEV))
        one.replay()
        two.replay()
        one.replay()
        assert torch.equal(a, layer.serve(h)) and torch.equal(b, layer.serve(other))


def chain(h, weights, chosen, held, first, w4):
    plan = mg.muon_sort_tokens(chosen, held, first=first)
    x = mg.muon_dispatch_tokens(h, plan)
    both = mg.muon_int4_linear(x, w4, offsets=plan.offsets)
    n = both.shape[1] // 2
    a = mg.muon_swiglu(both[:, :n], both[:, n:])
    out = mg.muon_combine_tokens(a, plan, weights)
    return [*plan, x, both, a, out, *mg.muon_combine_tokens_backward(out, a, plan, weights),
            *mg.muon_swiglu_backward(a, both[:, :n], both[:, n:])]


def same(a, b):
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("tokens", [5, 3000])
def test_streams_and_host_threads(tokens):
    """A stream of one's own, given or current, and two host threads at once."""
    weights, chosen = routed(tokens, 12, 3)
    h = torch.randn(tokens, 256, device=DEV).to(torch.bfloat16)
    w4 = mg.muon_int4_quantize_weight(torch.randn(8, 128, 256, device=DEV), 64)
    want = chain(h, weights, chosen, 8, 2, w4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = chain(h, weights, chosen, 8, 2, w4)
    s.synchronize()
    same(got, want)
    plan = mg.muon_sort_tokens(chosen, 8, first=2, stream=s)
    x = mg.muon_dispatch_tokens(h, plan, stream=s)
    both = mg.muon_int4_linear(x, w4, offsets=plan.offsets, stream=s)
    a = mg.muon_swiglu(both[:, :64], both[:, 64:], stream=s.cuda_stream)
    out = mg.muon_combine_tokens(a, plan, weights, stream=s)
    back = mg.muon_combine_tokens_backward(out, a, plan, weights, stream=s)
    gated = mg.muon_swiglu_backward(a, both[:, :64], both[:, 64:], stream=s)
    s.synchronize()
    same([*plan, x, both, a, out, *back, *gated], want)
    results = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                results[i] = chain(h, weights, chosen, 8, 2, w4)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for r in results:
        same(r, want)


HEAD = """
import torch
import muon_newton_schulz_step_gb300 as mg
from muon_newton_schulz_step_gb300 import experts
gen = torch.Generator(device="cuda").manual_seed(7)
def randn(*shape): return torch.randn(*shape, generator=gen, device="cuda")
def bf(*shape): return randn(*shape).to(torch.bfloat16)
def ints(n, *shape): return torch.randint(-1, n, shape, generator=gen, device="cuda", dtype=torch.int32)
"""
CALLS = {
    "sort": "c = ints(96, 9000, 8); run = lambda: mg.muon_sort_tokens(c, 96)",
    "sort_few": "c = ints(96, 9, 8); run = lambda: mg.muon_sort_tokens(c, 50, first=10)",
    "rows": ("c, x, y, w = ints(9, 300, 4), bf(300, 100), bf(1200, 100), randn(300, 4)\n"
             "p = mg.TokenPlan(*(t.clone() for t in mg.muon_sort_tokens(c, 9)))\n"
             "run = lambda: (mg.muon_dispatch_tokens(x, p), mg.muon_combine_tokens(y, p, w),\n"
             "               *mg.muon_combine_tokens_backward(x, y, p, w))"),
    "swiglu": ("g, u, d = bf(300, 700), bf(300, 700), bf(300, 700)\n"
               "run = lambda: (mg.muon_swiglu(g, u), *mg.muon_swiglu_backward(d, g, u))"),
    "int4": "w, x = bf(500, 700), bf(3, 700); run = lambda: (mg.muon_int4_linear(x, mg.muon_int4_quantize_weight(w, 32)),)",
    "layer": ("c, w, W = ints(8, 200, 2), randn(200, 2), bf(8, 64, 32).requires_grad_()\n"
              "h, lin = bf(200, 64).requires_grad_(), experts.Fp8Linear(bf(8, 64, 64).requires_grad_())\n"
              "def run():\n"
              "    p = experts.plan_tokens(c, 8)\n"
              "    y = experts.combine(experts.swiglu(lin(experts.dispatch(h, p), p.offsets)), p, w)\n"
              "    return (y.detach(), *torch.autograd.grad(y.float().square().sum(), (h, lin.weight)))"),
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
    """Captured by the first call that a process makes, nothing warmed up; the layer with its backward pass."""
    r = subprocess.run([sys.executable, "-c", HEAD + CALLS[name] + TAIL], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_example_runs():
    r = subprocess.run([sys.executable, "examples/moe_layer_step.py", "--steps", "2", "--fused", "--serve"], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "4 bits" in r.stdout, r.stderr[-2000:]


def test_results_where_torch_lacks_the_short_allocation(monkeypatch):
    weights, chosen = routed(50, 12, 3)
    h = torch.randn(50, 256, device=DEV).to(torch.bfloat16)
    w4 = mg.muon_int4_quantize_weight(torch.randn(8, 128, 256, device=DEV), 64)
    want = chain(h, weights, chosen, 8, 2, w4)
    monkeypatch.setattr(mg, "_allocate", None)
    got = chain(h, weights, chosen, 8, 2, w4)
    same(got, want)
    assert [t.stride() for t in got] == [t.stride() for t in want]


def test_profile_names_the_kernels():
    weights, chosen = routed(50, 12, 3)
    h = torch.randn(50, 256, device=DEV).to(torch.bfloat16)
    mg.muon_profile_enable(True)
    try:
        chain(h, weights, chosen, 8, 2, mg.muon_int4_quantize_weight(torch.randn(8, 128, 256, device=DEV), 64))
        torch.cuda.synchronize()
        seen = {k["name"]: k["launches"] for k in mg.muon_profile_read()}
    finally:
        mg.muon_profile_enable(False)
    for name in ("token_sort", "dispatch", "combine", "combine_backward", "swiglu", "swiglu_backward", "int4_quantize",
                 "int4_linear"):
        assert seen[name] == 1, (name, seen)
