"""Grouped products on inputs whose every partial sum is a whole number below
2^24 (or a multiple of a power of two with as few bits): the result has to be
equal, so that one input left out, taken twice or rounded shows at any length.
Random products cannot show that where a sum is long: their bound grows with it."""
import pytest
import torch

import bitplane_quantized_expert_amd as pm
import routed_cases as rc

pytestmark = pytest.mark.gpu
GATHER, SCATTER, SWIGLU = pm.PM_GROUPED_GATHER, pm.PM_GROUPED_SCATTER, pm.PM_GROUPED_SWIGLU


def report(name):
    print(f"[gpu case] {name}", flush=True)


def nonzero(shape, top, g):
    """Whole numbers of 1 to top in magnitude, both signs."""
    v = torch.randint(1, top + 1, shape, generator=g, device="cuda")
    return v * (2 * torch.randint(0, 2, shape, generator=g, device="cuda") - 1)


def check_exact(y, w64, x, off, order, n, top_k, flags, what):
    """y equals the plain form, whose sums are exact in fp64."""
    want = rc.grouped_plain(w64, x, off, order, n, top_k, bool(flags & GATHER),
                            bool(flags & SCATTER), bool(flags & SWIGLU))
    for rows, p, _ in want:
        assert torch.equal(y[rows].double(), p), what


# (counts, outputs): the streamed kernel, tiles of 128 rows, tiles of 256
W16 = [([3, 0, 5], 40), ([60, 0, 90], 258), ([300, 1800], 16640)]


@pytest.mark.parametrize("C", [8, 264, 1032, 2056, 4096, 4104, 8320, 12288])
@pytest.mark.parametrize("counts,R", W16)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_grouped16_exact(counts, R, C, ty):
    if sum(counts) > 2000 and C > 2056:
        C = 8 * (C // 64)              # (many outputs: fewer inputs, as many steps)
    report(f"grouped exact {ty} {counts} {R} x {C}")
    g = rc.gen(C + R)
    E, n = len(counts), sum(counts)
    # sums of C products of up to 49 each: below 2^20
    w = nonzero((E, R, C), 7, g).to(rc.TYPES[ty])
    x = nonzero((n, C), 7, g).to(rc.TYPES[ty])
    off, order = rc.groups(counts, C)
    y = torch.full((n, R), 0.5, device="cuda")
    pm.pm_grouped_gemm(w, x, y, off, order, 1, SCATTER)
    check_exact(y, lambda e: w[e].double(), x, off, order, n, 1, SCATTER, (counts, R, C))


# the streamed kernel, tiles
COUNTS = [[3, 0, 4], [65, 0, 130]]


def codes(E, R, C, group, zeros, g, lo=-1, hi=1):
    """4-bit weights whose scales are powers of two."""
    q = torch.randint(0, 256, (E, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.exp2(torch.randint(lo, hi, (E, R, C // group), generator=g, device="cuda").float()).half()
    z = None
    if zeros:
        z = torch.randint(0, 16, (E, R, C // group), generator=g, device="cuda", dtype=torch.uint8)
    return q, s, z


@pytest.mark.parametrize("group,C", [(32, 32), (64, 448), (128, 1280), (128, 2176), (64, 2048),
                                     (32, 4096), (96, 4128), (128, 4224), (64, 8320), (256, 8192),
                                     (128, 12288)])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
def test_w4_exact(counts, group, C, zeros, ty):
    """fp32 rows hold three values of 17 bits among small ones: what a single
    half would round away."""
    report(f"w4 exact {ty} {counts} group {group} cols {C} zeros {zeros}")
    g = rc.gen(C + group)
    E, R, n = len(counts), 50, sum(counts)
    q, s, z = codes(E, R, C, group, zeros, g)
    x = nonzero((n, C), 3, g)
    if ty == "f32":
        at = torch.stack([torch.randperm(C, generator=g, device="cuda")[:3] for _ in range(n)])
        # (odd, and the first in turn in each block of 128 inputs)
        at[:, 0] = (torch.arange(n, device="cuda") * 128 + at[:, 0] % 128) % C
        x.scatter_(1, at, (65536 + 2 * torch.randint(0, 32768, (n, 3), generator=g, device="cuda") + 1))
    # in units of the smallest scale, 1/2: 2 * 15 * (3 * 2^17 + 3 C) < 2^24
    assert 2 * 15 * (3 * 2 ** 17 * (ty == "f32") + 3 * C) < 2 ** 24
    x = x.to(rc.TYPES[ty])
    off, order = rc.groups(counts, C)
    y = torch.full((n, R), 0.25, device="cuda")
    pm.pm_grouped_gemm_w4(q, s, z, group, x, y, off, order, 1, SCATTER)
    check_exact(y, lambda e: rc.decode_w4(q[e], s[e], None if z is None else z[e], group), x, off,
                order, n, 1, SCATTER, (counts, group, C, zeros, ty))


@pytest.mark.parametrize("group,C", [(32, 96), (64, 448), (128, 2176), (32, 4096), (96, 4128),
                                     (64, 8320), (128, 12288)])
@pytest.mark.parametrize("counts", COUNTS)
def test_w4_fp32_one_hot_in_every_block(counts, group, C):
    """1 + 2^-20 in one input of every 32 (in turn over rows and calls): the
    weight times it, 24 bits, of which a half has 11."""
    report(f"w4 one-hot of 21 bits {counts} group {group} cols {C}")
    g = rc.gen(C)
    E, R, n = len(counts), 50, sum(counts)
    q, s, z = codes(E, R, C, group, True, g, -3, 4)
    off, order = rc.groups(counts, C)
    blocks = (C + 31) // 32
    for first in range(0, blocks, n):
        at = ((first + torch.arange(n)) % blocks * 32 + torch.randint(0, 32, (n,))) % C
        x = torch.zeros(n, C)
        x[torch.arange(n), at] = 1.0 + 2.0 ** -20
        x = x.cuda()
        y = torch.full((n, R), 0.25, device="cuda")
        pm.pm_grouped_gemm_w4(q, s, z, group, x, y, off, order, 1, SCATTER)
        check_exact(y, lambda e: rc.decode_w4(q[e], s[e], z[e], group), x, off, order, n, 1,
                    SCATTER, (counts, group, C, first))


@pytest.mark.parametrize("C", [2176, 4224])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
def test_w4_gate_and_up_exact(counts, C, ty):
    """Gates of 128 and more, where SiLU(g) is max(g, 0) in fp32: gate and up
    come from the same input of the two halves of the matrix."""
    report(f"w4 gate and up exact {ty} {counts} cols {C}")
    g = rc.gen(C + 1)
    E, R, n, K = len(counts), 100, sum(counts), 2
    q, s, z = codes(E, R, C, 128, True, g, 7, 9)
    off, order = rc.groups(counts, C)
    nx = (n + K - 1) // K
    x = torch.zeros(nx, C)
    x[torch.arange(nx), (torch.arange(nx) * 128 + torch.randint(0, 128, (nx,))) % C] = 1.0
    x = x.to(rc.TYPES[ty]).cuda()
    y = torch.full((n, R // 2), 0.25, device="cuda")
    pm.pm_grouped_gemm_w4(q, s, z, 128, x, y, off, order, K, GATHER | SWIGLU)
    offs, ordl = off.tolist(), order.long()
    for e in range(E):
        a, b = offs[e], offs[e + 1]
        p = x[ordl[a:b] // K].double() @ rc.decode_w4(q[e], s[e], z[e], 128).T
        assert torch.equal(y[a:b].double(), p[:, :R // 2].clamp(min=0) * p[:, R // 2:]), e
