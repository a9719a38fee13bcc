"""One training step of a small mixture-of-experts layer, end to end.

    python examples/moe_layer_step.py [--steps 20] [--fused] [--serve]

Routes tokens to experts (group-limited, with a balance bias), runs the experts'
gate, up and down projections on 8-bit operands over the tokens sorted by
expert, takes the gradients back through both, clips them by their global norm
and steps: Muon for the experts' matrices, AdamW for the router.  With --fused the
sort, the rows' way to the experts and back and the activation run in the library's
kernels too, each with its gradient; --serve then runs single tokens through the
trained layer on weights of 4 bits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import muon_newton_schulz_step_gb300 as mg  # noqa: E402
from muon_newton_schulz_step_gb300 import experts  # noqa: E402


class MoeLayer:
    def __init__(self, hidden=512, width=256, count=16, top_k=4, groups=4, top_groups=2, seed=0, fused=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.top_k, self.groups, self.top_groups = top_k, groups, top_groups
        self.fused = fused

        def matrix(*shape, std):
            w = torch.randn(*shape, generator=g, device="cuda") * std
            return w.to(torch.bfloat16).requires_grad_(True)

        self.router = (torch.randn(count, hidden, generator=g, device="cuda") * hidden ** -0.5).requires_grad_(True)
        self.bias = torch.zeros(count, device="cuda")
        self.gate = experts.Fp8Linear(matrix(count, width, hidden, std=hidden ** -0.5))
        self.up = experts.Fp8Linear(matrix(count, width, hidden, std=hidden ** -0.5))
        self.down = experts.Fp8Linear(matrix(count, hidden, width, std=width ** -0.5))
        self.layers = (self.gate, self.up, self.down)
        self.momentum = [torch.zeros_like(w.weight, dtype=torch.float32) for w in self.layers]
        self.adam = [torch.zeros_like(self.router), torch.zeros_like(self.router)]
        self.steps = 0
        self.kept = {}                               # weights of 4 bits by block, where it serves

    def __call__(self, h):
        """h: tokens x hidden in bf16; (output, tokens of each expert)."""
        logits = h.float() @ self.router.t()
        weights, chosen, counts = experts.route(logits, self.top_k, bias=self.bias, score="sigmoid", groups=self.groups,
                                                top_groups=self.top_groups)
        if self.fused:
            plan = experts.plan_tokens(chosen, counts.numel())
            x = experts.dispatch(h, plan)
            y = self.down(experts.swiglu(self.gate(x, plan.offsets), self.up(x, plan.offsets)), plan.offsets)
            return experts.combine(y, plan, weights, out_dtype=torch.float32), counts
        order, offsets = experts.sort_tokens(chosen, counts)
        token = order // self.top_k
        x = h[token]
        y = self.down(torch.nn.functional.silu(self.gate(x, offsets)) * self.up(x, offsets), offsets)
        out = torch.zeros(h.shape, dtype=torch.float32, device=h.device)
        return out.index_add(0, token, y.float() * weights.reshape(-1)[order, None]), counts

    def step(self, counts, lr=0.02, max_norm=1.0):
        """Clip, update every parameter, round the weights to 8 bits anew; the
        gradients' norm before clipping (on the device)."""
        self.steps += 1
        grads = [w.weight.grad for w in self.layers] + [self.router.grad]
        norm = mg.muon_grad_clip(grads, max_norm)
        matrices = [m for w in self.layers for m in w.weight.detach()]
        mg.muon_step_ex(matrices, [m for w in self.layers for m in w.weight.grad],
                        [m for mom in self.momentum for m in mom], lr, 0.95, 0.0)
        mg.muon_adamw_step([self.router.detach()], [self.router.grad], [self.adam[0]], [self.adam[1]], lr=1e-3,
                           step=self.steps)
        load = counts.float()
        self.bias += 1e-3 * torch.sign(load.mean() - load)
        for w in self.layers:
            w.update()
            w.weight.grad = None
        self.router.grad = None
        for gate_up, down in self.kept.values():
            gate_up.update(self.gate_and_up())
            down.update(self.down.weight)
        return norm

    def gate_and_up(self):
        return torch.cat([self.gate.weight, self.up.weight], 1)          # one product makes gate and up

    @torch.no_grad()
    def serve(self, h, block=64):
        """The layer's output for a few tokens, on weights of 4 bits with scales of ``block`` columns, made by the
        first call with it and anew by each step."""
        if block not in self.kept:
            self.kept[block] = (experts.Int4Linear(self.gate_and_up(), block),
                                experts.Int4Linear(self.down.weight, block))
        gate_up, down = self.served = self.kept[block]
        weights, chosen, _ = mg.muon_route(h.float() @ self.router.t(), self.top_k, bias=self.bias, score="sigmoid",
                                           groups=self.groups, top_groups=self.top_groups)
        plan = experts.plan_tokens(chosen, self.bias.numel())
        x = experts.dispatch(h, plan)
        y = down(experts.swiglu(gate_up(x, plan.offsets)), plan.offsets)
        return experts.combine(y, plan, weights, out_dtype=torch.float32)


def train(steps=20, tokens=1024, hidden=512, seed=0, fused=False, layer=None):
    """Losses of fitting the layer to a fixed random target, and the gradients' norms."""
    layer = MoeLayer(hidden=hidden, seed=seed, fused=fused) if layer is None else layer
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    h = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn(tokens, hidden, generator=g, device="cuda") * 0.5
    losses, norms = [], []
    for _ in range(steps):
        out, counts = layer(h)
        loss = (out - target).square().mean()
        loss.backward()
        norms.append(layer.step(counts))
        losses.append(loss.detach())
    return [float(v) for v in losses], [float(v) for v in norms]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--fused", action="store_true", help="rows and activation by the library's kernels too")
    ap.add_argument("--serve", action="store_true", help="then single tokens on weights of 4 bits")
    args = ap.parse_args()
    layer = MoeLayer(fused=args.fused)
    losses, norms = train(args.steps, layer=layer)
    for i, (a, b) in enumerate(zip(losses, norms)):
        print(f"step {i:3d}  loss {a:.4f}  gradient norm {b:.4f}")
    if args.serve:
        h = torch.randn(4, 512, device="cuda").to(torch.bfloat16)
        with torch.no_grad():
            off = layer.serve(h) - layer(h)[0]
        print(f"4 bits: off by {float(off.norm() / layer(h)[0].norm()):.3f} of the 8-bit layer's output")
