"""A layer that serves runs on the weights that it has, in the block that is asked for, in captured graphs too."""
import os
import sys

import pytest
import torch

from muon_newton_schulz_step_gb300 import experts

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def fresh(layer, h, block):
    """What another layer serves that has the same weights and has served nothing before."""
    import moe_layer_step

    other = moe_layer_step.MoeLayer(seed=0, fused=True)
    with torch.no_grad():
        for a, b in zip(other.layers, layer.layers):
            a.weight.copy_(b.weight)
        other.router.copy_(layer.router)
        other.bias.copy_(layer.bias)
    return other.serve(h, block)


def test_serving_follows_steps_and_blocks():
    import moe_layer_step

    layer = moe_layer_step.MoeLayer(seed=8, fused=True)
    h = torch.randn(5, 512, device="cuda").to(torch.bfloat16)
    seen = []
    for block in (64, 32, 128, 64):
        seen.append(layer.serve(h, block))
        assert torch.equal(seen[-1], fresh(layer, h, block)), block
    assert not torch.equal(seen[0], seen[1]) and torch.equal(seen[0], seen[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer.serve(h)
    for _ in range(2):
        before = layer.serve(h)
        out, counts = layer(h)
        out.square().sum().backward()
        layer.step(counts, lr=0.5)
        after = layer.serve(h)
        assert not torch.equal(after, before)
        for block in (32, 64, 128):
            assert torch.equal(layer.serve(h, block), fresh(layer, h, block)), block
        graph.replay()
        assert torch.equal(held, after)


def test_update_keeps_its_memory_and_refuses_other_shapes():
    w = torch.randn(3, 40, 200, device="cuda")
    x = torch.randn(6, 200, device="cuda")
    offsets = torch.tensor([0, 2, 3, 6], dtype=torch.int32, device="cuda")
    layer = experts.Int4Linear(torch.randn_like(w), 32)
    at = layer.codes.codes.data_ptr(), layer.codes.scale.data_ptr()
    layer.update(w)
    assert at == (layer.codes.codes.data_ptr(), layer.codes.scale.data_ptr())
    assert torch.equal(layer(x, offsets), experts.Int4Linear(w, 32)(x, offsets))
    for bad in (w[:1], w[:, :1], w[:, :, :130], w[0], w[:, :, :1]):
        with pytest.raises(ValueError, match="shape"):
            layer.update(bad.contiguous())
    assert torch.equal(layer(x, offsets), experts.Int4Linear(w, 32)(x, offsets))
