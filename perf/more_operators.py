"""Timed cases of a mixture-of-experts layer's way from the router to its output.

What the layer runs between routing and its experts' products, and after them,
and the products that serve a few generated tokens: the sort of the routed
entries by expert, the tokens' rows on their way to the experts and, weighted,
back, the gated activation between the projections, the gradients of these, and
products with weights of 4 bits.  ``run`` computes them in a plain form
(elementary torch operations in 32 bits, rounded once at the end) or, where
``own`` is true, by the calls that a program makes of this package.  Sizes are
those of the package's workloads (hidden size 6144, expert width 2048, 384
experts with 96 on a rank, 8 chosen for each token) or generic.

Definitions.  An entry is one choice of one token: entry e of ``chosen`` (tokens x
top_k) is token e // top_k's.  A rank holds the experts first .. first + local - 1;
entries of other experts, or of none (-1), have no row to compute.

  order    entries sorted by expert, equal ones as they come; those of no expert
           held here first
  place    the inverse: where each entry's row lies (tokens x top_k)
  offsets  local + 1: rows offsets[i] .. offsets[i + 1] are expert first + i's
  rows     row place[t, j] is x[t]; rows of no expert here are zero
  back     out[t] = sum over j of weights[t, j] * y[place[t, j]], over entries
           whose expert is held here
  gated    gate / (1 + exp(-gate)) * up
  4 bits   w[n, k] = code[n, k] * scale[k // group, n]; codes are integers from -8
           to 7, two to a byte, the even column in the low half; rows end on a
           multiple of 128 columns, zeros past the last
"""
import math

import numpy as np
import torch

own = False

HIDDEN, WIDTH, EXPERTS, LOCAL, TOP = 6144, 2048, 384, 96, 8


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one generated token's entries: a call whose latency counts
        {"name": "sort_token", "op": "sort", "tokens": 1, "top_k": TOP, "experts": EXPERTS, "first": 0, "local": EXPERTS,
         "padded": False},
        # a long batch's entries on a rank that holds a quarter of the experts, the batch's end padded
        {"name": "sort_sequence", "op": "sort", "tokens": 32768, "top_k": TOP, "experts": EXPERTS, "first": LOCAL,
         "local": LOCAL, "padded": True},
        # a small odd batch in fp32, half of the experts held here
        {"name": "rows_odd", "op": "rows", "tokens": 1001, "top_k": 4, "experts": 60, "first": 30, "local": 30,
         "padded": True, "cols": 1300, "dtype": "f32"},
        # a training batch's rows to the experts
        {"name": "rows_sequence", "op": "rows", "tokens": 8192, "top_k": TOP, "experts": LOCAL, "first": 0, "local": LOCAL,
         "padded": False, "cols": HIDDEN, "dtype": "bf16"},
        # one generated token's eight results, weighted
        {"name": "back_token", "op": "back", "tokens": 1, "top_k": TOP, "experts": EXPERTS, "first": 0, "local": EXPERTS,
         "padded": False, "cols": HIDDEN, "dtype": "bf16", "weighted": True},
        # a training batch's results, weighted
        {"name": "back_sequence", "op": "back", "tokens": 8192, "top_k": TOP, "experts": LOCAL, "first": 0, "local": LOCAL,
         "padded": False, "cols": HIDDEN, "dtype": "bf16", "weighted": True},
        # gradients of an odd batch, rows that start anywhere, half of the experts held here
        {"name": "back_grad_odd", "op": "back_grad", "tokens": 513, "top_k": 6, "experts": 64, "first": 0, "local": 32,
         "padded": True, "cols": 1301, "dtype": "bf16", "weighted": True},
        # gradients of a training batch's weighted sum: the rows' and the weights'
        {"name": "back_grad_sequence", "op": "back_grad", "tokens": 8192, "top_k": TOP, "experts": LOCAL, "first": 0,
         "local": LOCAL, "padded": False, "cols": HIDDEN, "dtype": "bf16", "weighted": True},
        # one generated token's eight experts, gate and up from one product
        {"name": "gated_token", "op": "gated", "rows": TOP, "cols": WIDTH, "dtype": "bf16", "joined": True},
        # gradient of a training batch's gated activation
        {"name": "gated_grad_sequence", "op": "gated_grad", "rows": 8192 * TOP, "cols": WIDTH, "dtype": "bf16",
         "joined": True},
        # one generated token through one projection of 4 bits: bound by the weight's bytes
        {"name": "four_bits_token", "op": "four_bits", "tokens": 1, "out": HIDDEN, "inner": HIDDEN, "groups": 0,
         "block": 128, "dtype": "bf16", "rest": False},
        # a batch of generated tokens through the gate projections of a rank's experts
        {"name": "four_bits_experts", "op": "four_bits", "tokens": 256, "out": WIDTH, "inner": HIDDEN, "groups": LOCAL,
         "block": 32, "dtype": "bf16", "rest": True},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "rows", "back", "back_grad", "gated", "gated_grad", "four_bits", "four_bits"])
    dtype = rng.choice(["bf16", "f32"])
    if op in ("gated", "gated_grad"):
        return {"op": op, "rows": _spread(rng, 1, 8192 * (TOP if dtype == "bf16" else TOP // 2)),
                "cols": _spread(rng, 64, WIDTH), "dtype": dtype, "joined": rng.choice([True, False])}
    if op == "four_bits":
        groups = rng.choice([0, _spread(rng, 2, LOCAL)])
        return {"op": op, "tokens": _spread(rng, 1, 512), "out": _spread(rng, 64, WIDTH if groups else HIDDEN),
                "inner": _spread(rng, 64, HIDDEN), "groups": groups, "block": rng.choice([32, 64, 128]), "dtype": dtype,
                "rest": bool(groups) and rng.choice([True, False])}
    experts = _spread(rng, 8, EXPERTS)
    local = rng.choice([experts, max(1, experts // 2), max(1, experts // 4)])
    case = {"op": op, "tokens": _spread(rng, 1, 32768 if op == "sort" else 8192 if dtype == "bf16" else 4096),
            "top_k": rng.randint(1, TOP), "experts": experts, "first": rng.choice([0, experts - local]), "local": local,
            "padded": rng.choice([True, False])}
    if op != "sort":
        case |= {"cols": _spread(rng, 64, HIDDEN), "dtype": dtype}
    if op in ("back", "back_grad"):
        # without weights the sum is the gradient of the tokens on their way to the experts
        case["weighted"] = op == "back_grad" or rng.choice([True, True, False])
    return case


# ------------------------------------------------------------------ inputs --
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _chosen(case, gen):
    """The experts of each token, distinct, by uneven popularities; -1 for the padding at a batch's end."""
    t, e = case["tokens"], case["experts"]
    popular = _randn(gen, e) * 0.5
    chosen = (_randn(gen, t, e) + popular).topk(case["top_k"], -1).indices.to(torch.int32)
    if case["padded"]:
        chosen[t - t // 16:] = -1
    return chosen.contiguous()


def _four_bits(w, block):
    """A weight kept in 4 bits, as its owner lays it out once: codes (rows, half of cols up to 128) and scales
    (blocks of columns, rows)."""
    w = torch.nn.functional.pad(w, (0, -w.shape[-1] % 128))
    b = w.view(w.shape[0], -1, block)
    scale = (b.abs().amax(-1) / 7.0).to(torch.bfloat16)
    by = scale.float()[..., None]
    q = torch.where(by > 0, b / by, torch.zeros_like(b)).round().clamp(-7, 7).to(torch.int16).view(w.shape[0], -1)
    codes = (q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)
    return codes.to(torch.uint8), scale.t().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op in ("gated", "gated_grad"):
        r, c = case["rows"], case["cols"]
        if case["joined"]:
            both = _randn(gen, r, 2 * c).to(_dtype(case))
            state["gate"], state["up"] = both[:, :c], both[:, c:]
        else:
            state["gate"], state["up"] = _randn(gen, r, c).to(_dtype(case)), _randn(gen, r, c).to(_dtype(case))
        if op == "gated_grad":
            state["d"] = (_randn(gen, r, c) * 1e-2).to(_dtype(case))
        return state
    if op == "four_bits":
        t, n, k, g = case["tokens"], case["out"], case["inner"], case["groups"]
        channel = torch.exp(0.5 * _randn(gen, k))
        state["x"] = (_randn(gen, t, k) * channel).to(_dtype(case))
        parts = [_four_bits(_randn(gen, n, k) * 0.02, case["block"]) for _ in range(g or 1)]
        if g:
            state["codes"], state["scale"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
            rng = np.random.RandomState(seed % (1 << 31))
            p = np.exp(0.5 * rng.standard_normal(g))
            lead = t // 8 if case["rest"] else 0
            counts = rng.multinomial(t - lead, p / p.sum())
            state["offsets"] = torch.tensor(lead + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32,
                                            device="cuda")
            state["most"] = max(1, int(counts.max()))
        else:
            state["codes"], state["scale"] = parts[0]
            state["offsets"] = None
        return state
    state["chosen"] = _chosen(case, gen)
    if op == "sort":
        return state
    # the order that the sort left
    state["order"], state["place"], state["offsets"] = _sort(case, state["chosen"])
    t, c = case["tokens"], case["cols"]
    if op == "rows":
        state["x"] = _randn(gen, t, c).to(_dtype(case))
        return state
    n = t * case["top_k"]
    y = _randn(gen, n, c).to(_dtype(case))
    y[:int(state["offsets"][0])] = 0    # rows of no expert, as the experts' products leave them
    state["y"] = y
    w = torch.rand(t, case["top_k"], generator=gen, device="cuda") + 0.05
    state["weights"] = w / w.sum(-1, keepdim=True) * 2.5 if case["weighted"] else None
    if op == "back_grad":
        state["d"] = (_randn(gen, t, c) * 1e-2).to(_dtype(case))
    return state


# -------------------------------------------------------------- plain forms --
def _sort(case, chosen):
    e = chosen.reshape(-1) - case["first"]
    held = (e >= 0) & (e < case["local"])
    bucket = torch.where(held, e + 1, torch.zeros_like(e))
    order = torch.sort(bucket, stable=True).indices
    place = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device))
    sizes = torch.zeros(case["local"] + 1, dtype=torch.int32, device=e.device)
    sizes.index_add_(0, bucket.long(), torch.ones_like(bucket))
    return (order.to(torch.int32), place.to(torch.int32).view(chosen.shape),
            torch.cumsum(sizes, 0, dtype=torch.int32))


def _held(state):
    """Which places hold a row of an expert that is here."""
    return state["place"] >= state["offsets"][0]


def _rows(state):
    token = state["order"].long() // state["case"]["top_k"]
    out = state["x"][token]
    here = torch.arange(token.numel(), device=token.device) >= state["offsets"][0]
    return torch.where(here[:, None], out, torch.zeros_like(out))


def _taken(state):
    """y's rows of each token in 32 bits (tokens x top_k x cols), zero where there is none."""
    taken = state["y"][state["place"].long()].float()
    return torch.where(_held(state)[..., None], taken, torch.zeros_like(taken))


def _back(state):
    taken = _taken(state)
    if state["weights"] is not None:
        taken = taken * state["weights"][..., None]
    return taken.sum(1).to(state["y"].dtype)


def _back_grad(state):
    d = state["d"].float()
    held = _held(state)
    d_weights = torch.where(held, (_taken(state) * d[:, None, :]).sum(-1), torch.zeros_like(state["weights"]))
    by = torch.where(held, state["weights"], torch.zeros_like(state["weights"])).reshape(-1)
    order = state["order"].long()
    d_y = d[order // state["case"]["top_k"]] * by[order][:, None]
    return d_y.to(state["y"].dtype), d_weights


def _gated(state):
    g, u = state["gate"].float(), state["up"].float()
    return (g / (1.0 + torch.exp(-g)) * u).to(state["gate"].dtype)


def _gated_grad(state):
    g, u, d = state["gate"].float(), state["up"].float(), state["d"].float()
    s = 1.0 / (1.0 + torch.exp(-g))
    dt = state["gate"].dtype
    return (d * u * (s * (1.0 + g * (1.0 - s)))).to(dt), (d * (g * s)).to(dt)


def _values(codes, scale, block, k):
    """What a weight's codes and scales stand for, in 32 bits."""
    c = codes.to(torch.int32)
    q = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    q = ((q ^ 8) - 8).float()
    return (q * scale.float().transpose(-1, -2).repeat_interleave(block, -1))[..., :k]


def _four_bits_product(state):
    case = state["case"]
    x = state["x"].float()
    w = _values(state["codes"], state["scale"], case["block"], case["inner"])
    if state["offsets"] is None:
        return (x @ w.t()).to(torch.bfloat16)
    off, most, g = state["offsets"].long(), state["most"], case["groups"]
    row = torch.arange(x.shape[0], device=x.device)
    group = torch.bucketize(row, off[1:], right=True)
    spot = group * most + row - off[group]
    spot = torch.where(row >= off[0], spot, torch.full_like(spot, g * most))
    room = x.new_zeros(g * most + 1, x.shape[1]).index_copy_(0, spot, x)[:g * most].view(g, most, -1)
    y = torch.bmm(room, w.transpose(1, 2)).view(g * most, -1)
    return torch.cat([y, y.new_zeros(1, y.shape[1])])[spot].to(torch.bfloat16)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(case, op, state)
    if op == "sort":
        return _sort(case, state["chosen"])
    if op == "rows":
        return _rows(state)
    if op == "back":
        return _back(state)
    if op == "back_grad":
        return _back_grad(state)
    if op == "gated":
        return _gated(state)
    if op == "gated_grad":
        return _gated_grad(state)
    return _four_bits_product(state)


def _run_own(case, op, state):
    import muon_newton_schulz_step_gb300 as mg

    if op == "sort":
        return tuple(mg.muon_sort_tokens(state["chosen"], case["local"], first=case["first"]))
    if op == "gated":
        return mg.muon_swiglu(state["gate"], state["up"])
    if op == "gated_grad":
        return mg.muon_swiglu_backward(state["d"], state["gate"], state["up"])
    if op == "four_bits":
        w = mg.Int4Matrix(state["codes"], state["scale"], case["block"], case["inner"])
        return mg.muon_int4_linear(state["x"], w, offsets=state["offsets"])
    plan = mg.TokenPlan(state["order"], state["place"], state["offsets"])
    if op == "rows":
        return mg.muon_dispatch_tokens(state["x"], plan)
    if op == "back":
        return mg.muon_combine_tokens(state["y"], plan, state["weights"])
    return mg.muon_combine_tokens_backward(state["d"], state["y"], plan, state["weights"])


# -------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "four_bits":
        t, n, k = case["tokens"], case["out"], case["inner"]
        g = min(t, case["groups"]) or 1
        size = 2 if case["dtype"] == "bf16" else 4
        up = (k + 127) // 128 * 128
        return {"bytes": t * k * size + g * n * (up // 2 + up // case["block"] * 2) + t * n * 2, "flops": 2 * t * n * k}
    if op == "sort":
        n = case["tokens"] * case["top_k"]
        return {"bytes": 12 * n + 4 * (case["local"] + 1), "flops": n}
    size = 2 if case["dtype"] == "bf16" else 4
    if op in ("gated", "gated_grad"):
        n = case["rows"] * case["cols"]
        return {"bytes": n * size * (3 if op == "gated" else 5), "flops": n * (5 if op == "gated" else 11)}
    t, c, n = case["tokens"], case["cols"], case["tokens"] * case["top_k"]
    # rows that hold something; all of them are written
    some = n * case["local"] // case["experts"]
    if op == "rows":
        return {"bytes": (t + n) * c * size + n * 4, "flops": n * c}
    if op == "back":
        return {"bytes": (some + t) * c * size + n * (8 if case["weighted"] else 4), "flops": 2 * some * c}
    return {"bytes": (t + some + n) * c * size + n * 12, "flops": 3 * some * c}


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("gated", "gated_grad"):
        g, u = state["gate"].double().requires_grad_(True), state["up"].double().requires_grad_(True)
        y = g * torch.sigmoid(g) * u
        if op == "gated":
            return y.detach()
        return torch.autograd.grad(y, (g, u), state["d"].double())
    if op == "four_bits":
        return _exact_four_bits(case, state)
    order, place, offsets = _exact_sort(case, state["chosen"].cpu().numpy())
    if op == "sort":
        return order, place, offsets
    dev = "cuda"
    lead = int(offsets[0])
    order, place = torch.tensor(order, device=dev).long(), torch.tensor(place, device=dev).long()
    token = order // case["top_k"]
    if op == "rows":
        out = state["x"].double()[token]
        out[:lead] = 0
        return out
    y = state["y"].double()
    w = torch.ones(place.shape, dtype=torch.float64, device=dev) if state["weights"] is None else state["weights"].double()
    here = place >= lead
    if op == "back":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=dev)
        for j in range(case["top_k"]):
            out[here[:, j]] += w[here[:, j], j, None] * y[place[here[:, j], j]]
        return out
    d = state["d"].double()
    d_y, d_w = torch.zeros_like(y), torch.zeros_like(w)
    for j in range(case["top_k"]):
        t = here[:, j].nonzero().reshape(-1)
        d_y[place[t, j]] = d[t] * w[t, j, None]
        d_w[t, j] = (d[t] * y[place[t, j]]).sum(-1)
    return d_y, d_w


def _exact_sort(case, chosen):
    """Counting, one expert after the other."""
    flat = chosen.reshape(-1).astype(np.int64) - case["first"]
    flat[(flat < 0) | (flat >= case["local"])] = -1
    runs = [np.flatnonzero(flat == e) for e in range(-1, case["local"])]
    order = np.concatenate(runs)
    place = np.empty_like(order)
    place[order] = np.arange(order.size)
    return (order.astype(np.int32), place.reshape(chosen.shape).astype(np.int32),
            np.cumsum([r.size for r in runs]).astype(np.int32))


def _exact_four_bits(case, state):
    x, off = state["x"].double(), state["offsets"]
    bounds = [0, x.shape[0]] if off is None else off.tolist()
    codes = state["codes"] if off is not None else state["codes"][None]
    scale = state["scale"] if off is not None else state["scale"][None]
    y = x.new_zeros(x.shape[0], case["out"])
    for g, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi > lo:
            low, high = (codes[g] % 16).double(), torch.div(codes[g], 16, rounding_mode="floor").double()
            q = torch.empty(codes.shape[1], 2 * codes.shape[2], dtype=torch.float64, device=x.device)
            q[:, 0::2], q[:, 1::2] = low, high
            q[q > 7] -= 16
            at = torch.arange(case["inner"], device=x.device)
            y[lo:hi] = x[lo:hi] @ (q[:, at] * scale[g].double()[at // case["block"]].t()).t()
    return y
