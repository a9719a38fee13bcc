"""Products with weights of 4 bits where each block of the kernel works off several items (a tile
of the weight's rows by a tile of one group's tokens) in a row: copies that run on over an
item's end, tokens looked up ahead, and the sums of consecutive items."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_step_gb300 as mg
from tests.test_int4_gpu import check, expected, rows, weight

pytestmark = pytest.mark.gpu

TILES = {"1x1": (16, 8), "2x1": (32, 8), "2x2": (32, 16)}        # rows and tokens of an item


def blocks(dtype):
    """The most blocks of a launch, whatever the shape: three on an SM, two with fp32 x."""
    return (3 if dtype == torch.bfloat16 else 2) * torch.cuda.get_device_properties(0).multi_processor_count


def counted(seed, groups, most):
    """Rows of each group, 0 to `most`, some groups empty at both ends and in between."""
    counts = np.random.RandomState(seed).randint(0, most + 1, groups)
    counts[[0, groups // 2, groups - 1]] = 0
    return counts.tolist()


# name: (tile, rows of each group or of the one weight, n; None: as many as 16-row tiles are taken for)
CASES = {
    "two tiles of tokens for most experts": ("1x1", [9, 9, 9, 5], None),
    "a few rows for each of 96 experts": ("2x1", counted(1, 96, 6), 501),
    "eight tokens, many rows": ("2x1", 8, 40003),
    "one token, many rows": ("2x1", 1, 40000),
    "many tokens of one weight": ("2x2", 300, 2001),
    "many rows for each of 40 experts": ("2x2", counted(2, 40, 41), 610),
}


def setting(name, k, block, dtype, how, whole):
    tile, counts, n = CASES[name]
    if n is None:
        n = 16 * (blocks(dtype) // len(counts)) - 3
    gen = torch.Generator(device="cuda").manual_seed(k + n)
    stacked = isinstance(counts, list)
    lead, tail = (3, 2) if stacked and tile != "1x1" else (0, 0)
    tokens = lead + (sum(counts) if stacked else counts) + tail
    offsets = None
    if stacked:
        offsets = torch.tensor(lead + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    high, wide = TILES[tile]
    items = -(-n // high) * sum(-(-c // wide) for c in (counts if stacked else [counts]))
    groups = min(len(counts), tokens) if stacked else 1
    # the tile that these sizes are given, and more items than blocks
    assert tile == ("2x2" if tokens // groups > 8 else "2x1" if groups * -(-n // 16) > blocks(dtype) else "1x1")
    assert items > blocks(dtype)
    m = weight((len(counts), n, k) if stacked else (n, k), block, gen, whole=whole)
    x = rows(tokens, k, dtype, how, gen)
    if whole:
        x.copy_(torch.randint(-20, 21, (tokens, k), generator=gen, device="cuda"))
    return m, x, offsets, lead, tail


def product(m, x, offsets, lead, tail, out_dtype):
    bad = x.clone() if x.is_contiguous() else x
    if lead + tail:
        bad[:lead] = float("nan")                    # rows of no expert: zero, whatever they hold
        bad[len(bad) - tail:] = float("inf")
    out = mg.muon_int4_linear(bad, m, offsets=offsets, out_dtype=out_dtype)
    assert (out[:lead] == 0).all() and (out[len(out) - tail:] == 0).all()
    return out


# k: fewer blocks of 128 columns than warps, so that some have none; more, the last one ragged; two for each warp
@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("k", [700, 1300, 2048])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", ["plain", "odd"])
def test_several_items_a_block(name, k, block, dtype, how):
    m, x, offsets, lead, tail = setting(name, k, block, dtype, how, whole=False)
    want, off = expected(x, m, offsets)              # before rows of no expert are filled
    for out_dtype in (torch.float32, torch.bfloat16):
        check(product(m, x, offsets, lead, tail, out_dtype), want, off)


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("k", [700, 1300])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_several_items_of_whole_numbers(name, k, block, dtype):
    """Sums of whole halves below 2^22 (20 * 8 * 2 * 1300) have one value in fp32, in any order."""
    m, x, offsets, lead, tail = setting(name, k, block, dtype, "plain", whole=True)
    want, _ = expected(x, m, offsets)
    assert torch.equal(product(m, x, offsets, lead, tail, torch.float32).double(), want)
