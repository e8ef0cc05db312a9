"""The 8-bit operators where their arithmetic is at its ends: quotients beside a
midpoint at the smallest scales."""
import numpy as np
import pytest
import torch

import fp8_cases as fc
import routed_cases as rc
from test_gpu_fp8 import check_encode, report

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- encoder
def e4m3_midpoints():
    """The 126 borders of two non-negative finite codes."""
    codes = torch.arange(127, dtype=torch.uint8).view(fc.F8).double()
    return (codes[1:] + codes[:-1]) / 2


def beside_midpoints(scale, seed):
    """127 numbers whose quotients by `scale` are a midpoint of two codes, or one
    or two steps of fp32 beside one, of either sign."""
    g = np.random.default_rng(seed)
    x = (e4m3_midpoints().numpy() * float(scale)).astype(np.float32)
    x = (x.view(np.int32) + g.integers(-2, 3, x.shape, dtype=np.int32)).clip(0).view(np.float32)
    x = np.concatenate([x, np.float32([0.0])])
    return x * g.choice(np.float32([-1, 1]), x.shape)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_encode_smallest_scales(ty, block_rows):
    """Blocks whose scale lies from 2^-126, the least one, to 2^-94: products of
    a code and the scale that end below fp32's smallest number.  And a block
    of each kind beside ordinary ones, and beside one with an infinity."""
    report(f"encode smallest scales {ty} {block_rows}")
    g = np.random.default_rng(17)
    rows = []
    for e in [*range(-126, -93), -60]:
        for _ in range(4):
            s = np.float32(np.ldexp(1.0 + int(g.integers(0, 64)) * 2.0 ** -23, e))
            rows.append(np.concatenate([[np.float32(448.0) * s], beside_midpoints(s, len(rows))]))
    # a quotient just above 8.5, and one just above 0.09765625
    s = np.ldexp(np.float64(2 ** 23 + 15), -149)
    rows.append(np.resize(np.float64([448 * s, (17 * (2 ** 23 + 15) + 1) // 2 * 2.0 ** -149]), 128))
    rows.append(np.resize(np.float64([448 * 1.8072718654108278e-38, 1.7649143963401422e-39]), 128))
    x = torch.tensor(np.stack([np.float32(r[:128]) for r in rows]))
    if block_rows == 128:
        x = x.repeat_interleave(3, 0)[:, torch.randperm(128, generator=torch.Generator().manual_seed(1))]
        x = torch.cat([r.expand(128, 128) for r in x[::3]])
    x = torch.cat([x, x.roll(block_rows, 0), torch.ones_like(x)], dim=1)
    x[-block_rows:, 300] = float("inf")
    check_encode(x.to(rc.TYPES[ty]).cuda(), block_rows)
