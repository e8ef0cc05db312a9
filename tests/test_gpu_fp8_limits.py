"""The 8-bit operators where their arithmetic is at its ends: quotients beside a
midpoint at the smallest scales, gates whose exponential is almost infinite,
infinite scales."""
import numpy as np
import pytest
import torch

import bitplane_quantized_expert_amd as pm
import fp8_cases as fc
import routed_cases as rc
from test_gpu_fp8 import SWIGLU, check_encode, report

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


# ---------------------------------------------------------------- gates
@pytest.mark.parametrize("R", [256, 80])
@pytest.mark.parametrize("counts", [[2], [40, 9], [300]])
@pytest.mark.parametrize("y_ty", ["f32", "bf16"])
def test_grouped8_gates_at_the_ends(y_ty, counts, R):
    """SiLU of gates from -88.7, whose exponential is about fp32's largest, to 88,
    times up values that make the smallest results count.  One product per
    output, so sums are exact, and only the roundings of SiLU are allowed:
    16 steps of fp32, and that to the type of y."""
    report(f"fp8 gates {counts} {R} {y_ty}")
    E, C, h = len(counts), 128, R // 2
    off, _ = rc.groups(counts, 0)
    n = sum(counts)
    g = rc.gen(n + R)
    W = torch.zeros(E, R, C, device="cuda")
    W[:, :h, 5] = torch.tensor([-88.0, -72.0, -8.0, -0.5, 0.0, 0.5, 9.0, 88.0],
                               device="cuda")[torch.arange(h, device="cuda") % 8]
    W[:, h:, 5] = torch.randint(1, 9, (h,), generator=g, device="cuda").float() * 2.0 ** -3
    W = W.to(fc.F8)
    ws = torch.ones(E, -(-R // 128), 1, device="cuda")
    up = 1.0
    if R == 256:                                   # (else gate and up share a block)
        up = 2.0 ** 100
        ws[:, 1] = up
    x = torch.zeros(n, C, device="cuda")
    x[:, 5] = 1.0
    x = x.to(fc.F8)
    xs = 0.985 + 0.023 * torch.rand(n, 1, generator=g, device="cuda")
    y = torch.full((n, h), -7.0, dtype=rc.TYPES[y_ty], device="cuda")
    pm.pm_grouped_gemm_fp8(W, ws, x, xs, y, off, None, 1, SWIGLU)
    gate = (xs * W[0, :h, 5].float()).double()     # as fp32 rounds it
    s = torch.where(gate < 0, gate * torch.exp(gate) / (1 + torch.exp(gate)),
                    gate / (1 + torch.exp(-gate)))
    p = s * (xs * up * W[0, h:, 5].float()).double()
    # (an exponential beyond fp32's range may make the result 0)
    free = gate < -88.72
    lim = 16 * 2.0 ** -24 * p.abs() + rc.HALF_STEP[y.dtype] * p.abs() * (1 + 2.0 ** -19) + 2.0 ** -126
    bad = ~((y.double() - p).abs() <= lim) & ~free
    assert not bad.any(), (bad.nonzero()[0].tolist(), int(bad.sum()),
                           sorted(set(gate[bad].tolist()))[:4])


# ---------------------------------------------------------------- scales
@pytest.mark.parametrize("y_ty", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("counts", [[3, 1], [40, 40], [300, 20]])
@pytest.mark.parametrize("C", [16, 128, 144, 256, 272])
def test_grouped8_infinite_scale(y_ty, counts, C):
    """An infinite scale of weights, or of a row of x, makes its outputs infinite,
    with the sign of the block's sum, however few blocks of inputs there are;
    outputs of other rows and experts are as without it."""
    report(f"fp8 infinite scale {counts} {C} {y_ty}")
    R = 144
    off, _ = rc.groups(counts, 0)
    n = sum(counts)
    W, ws = fc.make_weights(2, R, C, 3)
    x, xs = fc.make_x(n, C, 4)
    # one sign throughout: no sum is 0
    W = W.view(torch.uint8).bitwise_and(0x77).bitwise_or(1).view(fc.F8)
    x = x.contiguous().view(torch.uint8).bitwise_and(0x77).bitwise_or(1)
    x[1] |= 0x80
    x = x.view(fc.F8)
    for last in (False, True):
        b = -1 if last else 0
        w2, x2 = ws.clone(), xs.clone()
        w2[0, 0, b] = float("inf")
        x2[2, b] = float("inf")
        y = torch.full((n, R), -7.0, dtype=rc.TYPES[y_ty], device="cuda")
        z = torch.full_like(y, -7.0)
        pm.pm_grouped_gemm_fp8(W, w2, x, x2, y, off, None, 1, 0)
        pm.pm_grouped_gemm_fp8(W, ws, x, xs, z, off, None, 1, 0)
        inf = torch.zeros(n, R, dtype=torch.bool, device="cuda")
        inf[:counts[0], :128] = True
        inf[2] = True
        sign = torch.ones(n, 1, device="cuda")
        sign[1] = -1.0
        want = torch.where(inf, float("inf") * sign, z.float())
        assert torch.equal(y.float(), want), (last, (y.float() != want).nonzero()[0].tolist())
