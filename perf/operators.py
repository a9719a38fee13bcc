"""Timed cases of the training operators around the optimizer step.

Five operators of one mixture-of-experts training step, in the order in which
the step runs them: routing tokens to experts, its gradient, the experts' 8-bit
products, their gradients, and the global gradient norm with clipping in front
of the weight update.  ``run`` computes them in a plain form (elementary torch
operations in 32 bits, rounded once at the end) or, where ``own`` is true, by
the calls that a program makes of this package.  Sizes are those of the
package's workloads (hidden size 6144, expert width 2048, 384 experts with 96
on a rank, 8 chosen for each token) or generic.

Definitions (E4M3 operands with one power-of-two scale for each block of 128):

  scale of a block     2^e, e the smallest integer with max|x| <= 448 * 2^e
                       (0 where the block is zero), stored as the byte e + 127
  code of an element   x * 2^-e rounded to E4M3, nearest even
  "row" blocks         128 columns of one row;  "col" blocks: 128 rows of one
                       column, counted from the first row of each group;
                       "block" blocks: 128 x 128
"""
import math

import numpy as np
import torch

own = False

HIDDEN, WIDTH, EXPERTS, LOCAL, TOP = 6144, 2048, 384, 96, 8


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # the gradients of one layer's experts (96 x gate, up, down): the norm alone, as logged each step
        {"name": "norm_layer", "op": "norm", "count": 288, "rows": WIDTH, "cols": HIDDEN, "dtype": "bf16", "vectors": 0},
        # norm weights and a few small matrices: a call whose latency counts
        {"name": "clip_small", "op": "clip", "count": 8, "rows": 64, "cols": 256, "dtype": "f32", "vectors": 4},
        # eight experts' gradients and some vectors, with the clipping taking effect
        {"name": "clip_experts", "op": "clip", "count": 24, "rows": WIDTH, "cols": HIDDEN, "dtype": "bf16", "vectors": 6},
        # one generated token through the router
        {"name": "route_token", "op": "route", "tokens": 1, "experts": EXPERTS, "top_k": TOP, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "renormalize": True, "scale": 2.5},
        # a whole sequence through the router
        {"name": "route_sequence", "op": "route", "tokens": 32768, "experts": EXPERTS, "top_k": TOP, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "renormalize": True, "scale": 2.5},
        # gradient of the softmax router over a sequence, weights not renormalised: a dense gradient
        {"name": "route_grad_sequence", "op": "route_grad", "tokens": 32768, "experts": EXPERTS, "top_k": TOP,
         "dtype": "bf16", "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "renormalize": False,
         "scale": 1.0},
        # a small odd batch and an odd number of experts
        {"name": "route_grad_odd", "op": "route_grad", "tokens": 513, "experts": 60, "top_k": 4, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 1, "top_groups": 1, "renormalize": True, "scale": 1.0},
        # one generated token through one projection: bound by the weight's bytes
        {"name": "linear_token", "op": "linear", "tokens": 1, "out": HIDDEN, "inner": HIDDEN, "groups": 0},
        # a dense projection over a batch of sequences
        {"name": "linear_dense", "op": "linear", "tokens": 8192, "out": HIDDEN, "inner": HIDDEN, "groups": 0},
        # the gate projections of a rank's 96 experts, tokens sorted by expert, uneven counts
        {"name": "linear_experts", "op": "linear", "tokens": 32768, "out": WIDTH, "inner": HIDDEN, "groups": LOCAL},
        # gradients of a dense projection with odd sizes
        {"name": "linear_grad_odd", "op": "linear_grad", "tokens": 1001, "out": 520, "inner": 1300, "groups": 0},
        # gradients of the experts' projections: the input's and 96 weights'
        {"name": "linear_grad_experts", "op": "linear_grad", "tokens": 32768, "out": WIDTH, "inner": HIDDEN,
         "groups": LOCAL},
    ]


def _spread(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, min(hi, n))
    return n + 1 if n == 3072 and n < hi else n


def draw(rng):
    op = rng.choice(["norm", "clip", "route", "route_grad", "linear", "linear_grad"])
    if op in ("norm", "clip"):
        dtype = rng.choice(["bf16", "f32"])
        most = 48 if op == "clip" else 288 if dtype == "bf16" else 144
        return {"op": op, "count": _spread(rng, 1, most), "rows": _spread(rng, 1, WIDTH),
                "cols": _spread(rng, 1, HIDDEN), "dtype": dtype, "vectors": rng.randint(0, 8)}
    if op in ("route", "route_grad"):
        experts = _spread(rng, 8, EXPERTS)
        groups = rng.choice([1, 2, 4, 8])
        experts -= experts % groups
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(TOP, experts // groups * top_groups))
        return {"op": op, "tokens": _spread(rng, 1, 32768), "experts": experts, "top_k": top_k,
                "dtype": rng.choice(["bf16", "f32"]), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.choice([True, False]), "groups": groups, "top_groups": top_groups,
                "renormalize": rng.choice([True, False]), "scale": rng.choice([1.0, 2.5])}
    groups = rng.choice([0, 0, _spread(rng, 2, LOCAL)])
    tokens = _spread(rng, 1, 32768 if groups else 8192)
    return {"op": op, "tokens": tokens, "out": _spread(rng, 64, WIDTH if groups else HIDDEN),
            "inner": _spread(rng, 64, HIDDEN), "groups": groups}


# ------------------------------------------------------------------ inputs --
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _shapes(case):
    return [(case["rows"], case["cols"])] * case["count"] + [(HIDDEN,)] * case["vectors"]


def _counts(case, seed):
    """Tokens of each expert: a multinomial over uneven popularities."""
    groups, tokens = case["groups"], case["tokens"]
    rng = np.random.RandomState(seed % (1 << 31))
    p = np.exp(0.5 * rng.standard_normal(groups))
    return rng.multinomial(tokens, p / p.sum())


def _first(v):
    """Indices in descending order of the values, equal ones by ascending index."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices


def _choice64(case, logits, bias):
    """Biased scores in 64 bits, with the experts of the groups that are left out at -inf, and the group scores."""
    x = logits.double()
    s = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    sel = s + bias.double() if bias is not None else s
    t, e = sel.shape
    g = case["groups"]
    if g == 1:
        return s, sel, None
    by = sel.view(t, g, e // g)
    gs = by.topk(min(2, e // g), -1).values.sum(-1)
    order = _first(gs)[:, :case["top_groups"]]
    keep = torch.zeros(t, g, dtype=torch.bool, device=x.device).scatter_(1, order, True)
    return s, by.masked_fill(~keep[..., None], -math.inf).reshape(t, e), gs


def _near(case, logits, bias):
    """Tokens whose choice turns on a difference that 32 bits cannot be trusted with (equal inputs are no such case)."""
    k = case["top_k"]
    _, sel, gs = _choice64(case, logits, bias)
    v = sel.sort(-1, descending=True).values[:, :k + 1]
    gap = v[:, :-1] - v[:, 1:]
    tight = (gap < 1e-5 * v[:, :-1].abs().clamp_min(1e-3)) & (v[:, :-1] > -math.inf)
    if bias is None:
        tight &= gap > 0
    bad = tight.any(-1)
    if gs is not None:
        w = gs.sort(-1, descending=True).values
        n = case["top_groups"]
        if n < case["groups"]:
            bad |= (w[:, n - 1] - w[:, n]) < 1e-5
    return bad


def _logits(case, gen):
    t, e = case["tokens"], case["experts"]
    popular = torch.randn(e, generator=gen, device="cuda") * 0.5
    bias = torch.randn(e, generator=gen, device="cuda") * 0.02 if case["bias"] else None
    logits = (torch.randn(t, e, generator=gen, device="cuda") + popular).to(_dtype(case))
    for _ in range(40):
        bad = _near(case, logits, bias)
        again = (torch.randn(t, e, generator=gen, device="cuda") + popular).to(logits.dtype)
        logits = torch.where(bad[:, None], again, logits)
    return logits, bias


def _exponent(amax):
    """e of the definition above, from max|x| of each block."""
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    return torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-127, 127)


def _pad(x, dims):
    """x with zeros up to multiples of 128 in the last two dimensions (dims says which)."""
    r, c = x.shape[-2:]
    return torch.nn.functional.pad(x, (0, -c % 128 if dims[1] else 0, 0, -r % 128 if dims[0] else 0))


def _weight(w):
    """A weight kept in 8 bits, as its owner lays it out once: codes [.., rows, cols up to 128] and scale bytes."""
    p = _pad(w.float(), (True, True))
    r, c = p.shape[-2:]
    b = p.reshape(*p.shape[:-2], r // 128, 128, c // 128, 128)
    e = _exponent(b.abs().amax((-3, -1)))
    q = torch.ldexp(b, -e[..., :, None, :, None]).reshape(p.shape)[..., :w.shape[-2], :]
    return q.to(torch.float8_e4m3fn).contiguous(), (e + 127).to(torch.uint8).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op in ("norm", "clip"):
        grads = []
        for i, s in enumerate(_shapes(case)):
            dt = _dtype(case) if len(s) == 2 else torch.float32
            grads.append((torch.randn(s, generator=gen, device="cuda", dtype=dt)).mul_(1e-3 * (1 + i % 5)))
        state["grads"] = grads
        if op == "clip":
            state["out"] = [torch.empty_like(g) for g in grads]
            # about half of the norm that these gradients have
            state["max_norm"] = 1e-3 * math.sqrt(sum(g.numel() for g in grads))
        return state
    if op in ("route", "route_grad"):
        state["logits"], state["bias"] = _logits(case, gen)
        if op == "route_grad":
            s, sel, _ = _choice64(case, state["logits"], state["bias"])
            state["chosen"] = _first(sel)[:, :case["top_k"]].to(torch.int32).contiguous()
            state["grad"] = torch.randn(state["chosen"].shape, generator=gen, device="cuda") * 1e-2
        return state
    t, n, k, g = case["tokens"], case["out"], case["inner"], case["groups"]
    channel = torch.exp(0.5 * torch.randn(k, generator=gen, device="cuda"))
    state["x"] = (torch.randn(t, k, generator=gen, device="cuda") * channel).to(torch.bfloat16)
    if g:
        parts = [_weight(torch.randn(n, k, generator=gen, device="cuda") * 0.02) for _ in range(g)]
        state["w"], state["w_scale"] = torch.stack([p[0].view(torch.uint8) for p in parts]).view(
            torch.float8_e4m3fn), torch.stack([p[1] for p in parts])
        counts = _counts(case, seed)
        state["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        state["most"] = int(counts.max())
    else:
        state["w"], state["w_scale"] = _weight(torch.randn(n, k, generator=gen, device="cuda") * 0.02)
        state["offsets"] = None
        state["most"] = t
    if op == "linear_grad":
        size = torch.exp(0.5 * torch.randn(t, 1, generator=gen, device="cuda"))
        state["dy"] = (torch.randn(t, n, generator=gen, device="cuda") * size * 1e-3).to(torch.bfloat16)
    return state


# -------------------------------------------------------------- plain forms --
def _norm(grads):
    return torch.stack([g.float().square().sum() for g in grads]).sum().sqrt()


def _scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _route(case, logits, bias):
    s = _scores(logits.float(), case["score"])
    sel = s if bias is None else s + bias
    t, e = s.shape
    g = case["groups"]
    if g > 1:
        by = sel.view(t, g, e // g)
        gs = by.sort(-1, descending=True).values[..., :2].sum(-1)
        order = _first(gs)[:, :case["top_groups"]]
        keep = torch.zeros(t, g, dtype=torch.bool, device=s.device).scatter_(1, order, True)
        sel = torch.where(keep[..., None], by, by.new_full((), -math.inf)).reshape(t, e)
    chosen = _first(sel)[:, :case["top_k"]]
    w = s.gather(1, chosen)
    if case["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    counts = torch.zeros(e, dtype=torch.int32, device=s.device)
    counts.index_add_(0, chosen.reshape(-1), torch.ones(chosen.numel(), dtype=torch.int32, device=s.device))
    return w * case["scale"], chosen.to(torch.int32), counts


def _route_grad(case, logits, chosen, grad):
    s = _scores(logits.float(), case["score"])
    at = chosen.long()
    c = s.gather(1, at)
    d = grad * case["scale"]
    if case["renormalize"]:
        total = c.sum(-1, keepdim=True)
        d = (d - (d * c).sum(-1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, at, d)
    if case["score"] == "sigmoid":
        dx = ds * s * (1.0 - s)
    else:
        dx = s * (ds - (ds * s).sum(-1, keepdim=True))
    return dx.to(logits.dtype)


def _values(q, scale):
    """What a weight's codes and scale bytes stand for, in 32 bits."""
    e = scale.to(torch.int32) - 127
    e = e.repeat_interleave(128, -2).repeat_interleave(128, -1)[..., :q.shape[-2], :]
    return torch.ldexp(q.float(), e)


def _by_rows(x):
    """x rounded to E4M3 with a scale for each 128 columns of a row, as the values that stand for."""
    c = x.shape[-1]
    p = _pad(x.float(), (False, True))
    b = p.view(*p.shape[:-1], -1, 128)
    e = _exponent(b.abs().amax(-1, keepdim=True))
    return torch.ldexp(torch.ldexp(b, -e).to(torch.float8_e4m3fn).float(), e).view(p.shape)[..., :c]


def _by_cols(x):
    return _by_rows(x.transpose(-1, -2)).transpose(-1, -2)


def _spots(state):
    """Where each row of the sorted tokens lies when every expert's rows get the same room."""
    off = state["offsets"].long()
    row = torch.arange(state["x"].shape[0], device=off.device)
    g = torch.bucketize(row, off[1:], right=True)
    return g * state["most"] + row - off[g]


def _room(state, x):
    """[groups, most rows of a group, cols] with zeros where a group has fewer rows."""
    g = state["offsets"].numel() - 1
    r = x.new_zeros(g * state["most"], x.shape[1])
    return r.index_copy_(0, _spots(state), x).view(g, state["most"], -1)


def _linear(state):
    x, w = _by_rows(state["x"]), _values(state["w"], state["w_scale"])[..., :state["x"].shape[1]]
    if state["offsets"] is None:
        return (x @ w.t()).to(torch.bfloat16)
    y = torch.bmm(_room(state, x), w.transpose(1, 2))
    return y.view(-1, w.shape[1])[_spots(state)].to(torch.bfloat16)


def _linear_grad(state):
    x, dy = state["x"].float(), state["dy"].float()
    w = _values(state["w"], state["w_scale"])[..., :x.shape[1]]
    if state["offsets"] is None:
        return (_by_rows(dy) @ w).to(torch.bfloat16), (_by_cols(dy).t() @ _by_cols(x)).to(torch.bfloat16)
    dx = torch.bmm(_room(state, _by_rows(dy)), w).view(-1, x.shape[1])[_spots(state)]
    dw = torch.bmm(_by_cols(_room(state, dy)).transpose(1, 2), _by_cols(_room(state, x)))
    return dx.to(torch.bfloat16), dw.to(torch.bfloat16)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(case, op, state)
    if op == "norm":
        return _norm(state["grads"])
    if op == "clip":
        norm = _norm(state["grads"])
        by = (state["max_norm"] / (norm + 1e-6)).clamp_max(1.0)
        return [norm] + [(g.float() * by).to(g.dtype) for g in state["grads"]]
    if op == "route":
        return _route(case, state["logits"], state["bias"])
    if op == "route_grad":
        return _route_grad(case, state["logits"], state["chosen"], state["grad"])
    return _linear(state) if op == "linear" else _linear_grad(state)


def _run_own(case, op, state):
    import muon_newton_schulz_step_gb300 as mg

    if op == "norm":
        return mg.muon_grad_norm(state["grads"])
    if op == "clip":
        return [mg.muon_grad_clip(state["grads"], state["max_norm"], out=state["out"])] + state["out"]
    if op == "route":
        return mg.muon_route(state["logits"], case["top_k"], bias=state["bias"], score=case["score"],
                             groups=case["groups"], top_groups=case["top_groups"],
                             renormalize=case["renormalize"], scale=case["scale"])
    if op == "route_grad":
        return mg.muon_route_backward(state["grad"], state["logits"], state["chosen"], score=case["score"],
                                      renormalize=case["renormalize"], scale=case["scale"])
    w = mg.Fp8Matrix(state["w"], state["w_scale"], "block", case["inner"])
    if op == "linear":
        return mg.muon_fp8_linear(state["x"], w, offsets=state["offsets"])
    return mg.muon_fp8_linear_backward(state["dy"], state["x"], w, offsets=state["offsets"])


# -------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        size = 2 if case["dtype"] == "bf16" else 4
        n, v = case["count"] * case["rows"] * case["cols"], case["vectors"] * HIDDEN
        return {"bytes": (n * size + v * 4) * (1 if op == "norm" else 2), "flops": (n + v) * (2 if op == "norm" else 3)}
    if op in ("route", "route_grad"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        size = 2 if case["dtype"] == "bf16" else 4
        if op == "route":
            return {"bytes": t * e * size + t * k * 8 + e * (8 if case["bias"] else 4), "flops": t * e * 4}
        return {"bytes": 2 * t * e * size + t * k * 8, "flops": t * e * 6}
    t, n, k = case["tokens"], case["out"], case["inner"]
    g = min(t, case["groups"]) or 1
    if op == "linear":
        return {"bytes": t * k * 2 + g * n * k + t * n * 2, "flops": 2 * t * n * k}
    g_all = case["groups"] or 1
    return {"bytes": t * (2 * k + n) * 2 + g * n * k + g_all * n * k * 2, "flops": 4 * t * n * k}


# ------------------------------------------------------------------- exact --
def _e4m3_64(v):
    """The nearest E4M3 value (ties to even) of 64-bit values of at most 448."""
    a = v.abs()
    step = torch.exp2((torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3).clamp_min(-9))
    return torch.round(v / step) * step


def _scaled_64(x, dim):
    """x in 64 bits, rounded to E4M3 with one power of two for each 128 along `dim`."""
    out = torch.empty_like(x)
    for lo in range(0, x.shape[dim], 128):
        b = x.narrow(dim, lo, min(128, x.shape[dim] - lo))
        top = b.abs().amax(dim, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0))
        s = torch.where(top > 0, torch.exp2(e), torch.ones_like(top))
        out.narrow(dim, lo, b.shape[dim]).copy_(_e4m3_64(b / s) * s)
    return out


def _weight_64(q, scale, k):
    s = torch.exp2(scale.double() - 127)
    rows = torch.arange(q.shape[-2], device=q.device) // 128
    cols = torch.arange(k, device=q.device) // 128
    return q[..., :k].double() * s[..., rows[:, None], cols[None, :]]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "clip"):
        total = 0.0
        for g in state["grads"]:
            for part in g.reshape(-1).split(1 << 26):
                total += float(part.double().pow(2).sum())
        norm = torch.tensor(math.sqrt(total), dtype=torch.float64, device="cuda")
        if op == "norm":
            return norm
        by = min(1.0, state["max_norm"] / (math.sqrt(total) + 1e-6))
        return [norm] + [g.double() * by for g in state["grads"]]
    if op == "route":
        s, sel, _ = _choice64(case, state["logits"], state["bias"])
        chosen = _first(sel)[:, :case["top_k"]]
        w = torch.take_along_dim(s, chosen, 1)
        if case["renormalize"]:
            w = w / w.sum(-1, keepdim=True)
        return w * case["scale"], chosen.to(torch.int32), torch.bincount(
            chosen.reshape(-1), minlength=case["experts"]).to(torch.int32)
    if op == "route_grad":
        x = state["logits"].double().requires_grad_(True)
        s = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
        w = torch.take_along_dim(s, state["chosen"].long(), 1)
        if case["renormalize"]:
            w = w / w.sum(-1, keepdim=True)
        return torch.autograd.grad((w * case["scale"] * state["grad"].double()).sum(), x)[0]
    x, off = state["x"].double(), state["offsets"]
    bounds = [0, x.shape[0]] if off is None else off.tolist()
    if op == "linear":
        y = x.new_empty(x.shape[0], case["out"])
        for g, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            if hi > lo:
                w = _weight_64(state["w"] if off is None else state["w"][g],
                               state["w_scale"] if off is None else state["w_scale"][g], case["inner"])
                y[lo:hi] = _scaled_64(x[lo:hi], 1) @ w.t()
        return y
    dy = state["dy"].double()
    dx = torch.zeros_like(x)
    dw = x.new_zeros(len(bounds) - 1, case["out"], case["inner"])
    for g, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi > lo:
            w = _weight_64(state["w"] if off is None else state["w"][g],
                           state["w_scale"] if off is None else state["w_scale"][g], case["inner"])
            dx[lo:hi] = _scaled_64(dy[lo:hi], 1) @ w
            dw[g] = _scaled_64(dy[lo:hi], 0).t() @ _scaled_64(x[lo:hi], 0)
    return dx, (dw[0] if off is None else dw)
