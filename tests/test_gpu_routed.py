"""Routed experts on the device against plain fp64 forms, through the C ABI:
the router, the products grouped by expert with 16-bit and 4-bit weights, the
4-bit encoder, the combine, and whole layers of them, eager and captured."""
import numpy as np
import pytest
import torch

import bitplane_quantized_expert_amd as pm
import routed_cases as rc
import synth

pytestmark = pytest.mark.gpu
F = pm.PM_GROUPED_GATHER, pm.PM_GROUPED_SCATTER, pm.PM_GROUPED_SWIGLU
GATHER, SCATTER, SWIGLU = F


def report(name):
    print(f"[gpu case] {name}", flush=True)


# ---------------------------------------------------------------- router
def run_route(logits, top_k, stream=None):
    T, E = logits.shape
    ids = torch.full((T, top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, top_k), -7.0, device="cuda")
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((T * top_k,), -7, dtype=torch.int32, device="cuda")
    ws = torch.randint(0, 256, (max(1, pm.pm_route_workspace_bytes(T, E, top_k)),),
                       dtype=torch.uint8, device="cuda")
    pm.pm_route_topk_device(logits, top_k, ids, w, off, order, ws, stream)
    return ids, w, off, order


def check_route(logits, top_k, got=None, what=""):
    ids, w, off, order = (t.cpu().numpy() for t in (got or run_route(logits, top_k)))
    wi, ww, woff, word = rc.route_plain(logits, top_k)
    assert np.array_equal(ids, wi), what
    # fp64 softmax rounded to fp32: half a step, and a little for the exponential
    assert np.all(np.abs(w - ww) <= 1.01 * 2.0 ** -24 * ww + 2.0 ** -149), what
    assert np.array_equal(off, woff), what
    n = woff[-1]
    assert np.array_equal(order[:n], word), what
    assert np.all(order[n:] == -7), what


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 512, 10), (2, 4, 4), (5, 64, 8), (15, 65, 3),
                                   (16, 128, 2), (17, 200, 64), (33, 512, 10), (64, 256, 8),
                                   (65, 60, 4), (300, 1000, 10), (1003, 60, 4), (257, 4096, 64),
                                   (4100, 512, 10), (9000, 33, 1), (24, 512, 10), (25, 512, 10),
                                   (26, 512, 10), (32, 60, 8), (33, 60, 8), (48, 300, 5),
                                   (49, 300, 5), (47, 4096, 2), (48, 8, 1), (16, 4096, 64),
                                   (4, 4096, 8), (13, 2049, 8), (8, 2048, 16), (23, 1500, 4),
                                   (9, 1025, 64), (700, 2048, 10), (1, 1024, 1)])
def test_route_sizes(T, E, K):
    report(f"route {T} x {E} top-{K}")
    g = rc.gen(T * 7 + E)
    check_route(torch.randn(T, E, generator=g, device="cuda"), K)


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
def test_route_types_strides_ties_and_masks(ty):
    """Rows of a wider buffer; many equal logits; experts masked with -inf or
    the type's lowest value; NaN; +inf; signed zeros; tokens with nothing."""
    report(f"route masks and ties {ty}")
    dt = rc.TYPES[ty]
    T, E, K = 211, 96, 6
    g = rc.gen(5)
    buf = torch.randn(T, E + 13, generator=g, device="cuda").mul_(2).round_().div_(2).to(dt)
    l = buf[:, 7:7 + E]
    l[3] = -float("inf")                           # padding
    l[4, :] = float("nan")
    l[5, 4:] = -float("inf")                       # fewer than K left
    l[6, 10:] = torch.finfo(dt).min
    l[7, :] = torch.finfo(dt).min                  # all at the lowest value
    l[8, 20] = float("nan")
    l[9, 11] = l[9, 50] = float("inf")
    l[10, 0::2] = 0.0
    l[10, 1::2] = -0.0
    l[11, :] = torch.finfo(dt).max
    l[12, 95] = torch.finfo(dt).max
    l[13, :] = 0.0
    l[200:, :] = -float("inf")                     # a padded tail
    check_route(l, K)
    check_route(l[:1], K)
    check_route(l[3:5], K)


def test_route_agrees_with_the_host_router():
    report("route vs pm_route_topk")
    lg = np.stack([synth.router_logits(3, 1, 0, 0, 512, step=t) for t in range(70)])
    hi, hw = pm.pm_route_topk(lg, 10)
    ids, w, _, _ = run_route(torch.from_numpy(lg).cuda(), 10)
    assert np.array_equal(ids.cpu().numpy(), hi)
    assert np.all(np.abs(w.cpu().numpy().view(np.int32) - hw.view(np.int32)) <= 1)


def test_route_without_sorting_and_without_tokens():
    report("route: no order, no tokens")
    l = torch.randn(9, 40, generator=rc.gen(1), device="cuda")
    ids = torch.empty(9, 5, dtype=torch.int32, device="cuda")
    w = torch.empty(9, 5, device="cuda")
    pm.pm_route_topk_device(l, 5, ids, w)
    assert np.array_equal(ids.cpu().numpy(), rc.route_plain(l, 5)[0])
    off = torch.full((41,), 9, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 40, device="cuda")
    pm.pm_route_topk_device(e, 5, ids, w, off, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert not off.any()


def test_route_many_tokens():
    """More tokens than 256 blocks of the sorting hold."""
    report("route 17 000 000 tokens")
    T = 17_000_000
    l = torch.randn(T, 2, generator=rc.gen(2), device="cuda")
    l[12345:23456] = -float("inf")
    ids, w, off, order = run_route(l, 1)
    want = torch.where(l[:, 0] >= l[:, 1], 0, 1)
    want[12345:23456] = -1
    assert torch.equal(ids[:, 0].long(), want)
    assert torch.equal(w[:, 0], (want >= 0).float())
    n0, n1 = int((want == 0).sum()), int((want == 1).sum())
    assert off.tolist() == [0, n0, n0 + n1]
    assert torch.equal(order[:n0].long(), (want == 0).nonzero()[:, 0])
    assert torch.equal(order[n0:n0 + n1].long(), (want == 1).nonzero()[:, 0])


# ---------------------------------------------------------------- grouped products
def make_w16(E, R, C, dt, seed):
    w = torch.empty(E, R, C, dtype=dt, device="cuda")
    return w.normal_(0.0, 0.05, generator=rc.gen(seed))


def run_grouped16(counts, R, C, ty, y_ty, top_k, flags, seed=0, n_rows=None, order=True, pad=0,
                  wide=0):
    """One call against the plain form.  pad: extra elements per row of x and
    y; wide: columns of y kept from the right of the output."""
    dt = rc.TYPES[ty]
    E = len(counts)
    off, ordr = rc.groups(counts, seed, n_rows)
    n = ordr.numel()
    if not order:
        ordr = None
    w = make_w16(E, R, C, dt, seed + 1)
    nx = (n + top_k - 1) // top_k if flags & GATHER else n
    x = torch.randn(nx, C + 8 * pad, generator=rc.gen(seed + 2), device="cuda").to(dt)[:, :C]
    out = R // 2 if flags & SWIGLU else R
    ybuf = torch.full((n, out + pad + wide), 3.0, dtype=rc.TYPES[y_ty], device="cuda")
    y = ybuf[:, :out]
    pm.pm_grouped_gemm(w, x, y, off, ordr, top_k, flags)
    torch.cuda.synchronize()
    want = rc.grouped_plain(lambda e: w[e].double(), x, off, ordr, n, top_k, bool(flags & GATHER),
                            bool(flags & SCATTER), bool(flags & SWIGLU))
    rc.check_grouped(y, 3.0, want, f"{counts} {R}x{C} {ty}->{y_ty} flags {flags}")
    assert torch.all(ybuf[:, out:] == 3.0)


LAYOUTS = [(GATHER | SWIGLU, 2), (SCATTER, 3), (0, 1), (GATHER | SCATTER | SWIGLU, 4), (SWIGLU, 1)]


@pytest.mark.parametrize("ty,y_ty", [("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16"),
                                     ("f16", "f32")])
@pytest.mark.parametrize("flags,top_k", LAYOUTS)
def test_grouped16_layouts(ty, y_ty, flags, top_k):
    report(f"grouped {ty}->{y_ty} flags {flags}")
    run_grouped16([3, 0, 1, 17, 0, 40, 2], 96, 136, ty, y_ty, top_k, flags, seed=flags)


@pytest.mark.parametrize("counts", [[1], [0, 0, 1, 0], [16], [15, 16, 17], [31, 32, 33, 0, 1],
                                    [63, 64, 65], [127, 0, 128, 129], [255, 256, 257],
                                    [300, 1, 0, 77], [0, 0, 0]])
def test_grouped16_group_sizes(counts):
    report(f"grouped counts {counts}")
    n = max(1, sum(counts))
    run_grouped16(counts, 72, 256, "bf16", "f32", 1, SCATTER, seed=1, n_rows=n)
    run_grouped16(counts, 144, 256, "f16", "f16", 2, GATHER | SWIGLU, seed=2, n_rows=n)


@pytest.mark.parametrize("R,C", [(1, 8), (2, 16), (3, 24), (15, 40), (16, 64), (17, 72), (33, 128),
                                 (64, 200), (126, 512), (255, 1000), (258, 1032), (512, 264),
                                 (1000, 712), (40, 4104)])
def test_grouped16_odd_sizes(R, C):
    """Outputs and inputs off every tile, few rows and many."""
    report(f"grouped {R} x {C}")
    run_grouped16([2, 0, 21, 1], R, C, "bf16", "f32", 1, 0, seed=3)
    run_grouped16([130, 5, 290], R, C, "f16", "f16", 1, SCATTER, seed=4)
    if R % 2 == 0:
        run_grouped16([2, 140, 9], R, C, "bf16", "bf16", 3, GATHER | SWIGLU, seed=5)


def test_grouped16_strides_and_rows_outside():
    """Rows of wider buffers, unaligned output rows, fewer rows in the groups
    than entries of the order: the rest of y stays."""
    report("grouped strides, untouched rows")
    for counts in ([2, 5, 0, 9], [300, 70]):
        for flags in (0, SCATTER, GATHER | SWIGLU):
            run_grouped16(counts, 50, 88, "bf16", "bf16", 2, flags, seed=6, pad=3,
                          n_rows=sum(counts) + 37)
            run_grouped16(counts, 50, 88, "f16", "f32", 1, flags, seed=7, order=False, wide=1)


def test_grouped16_order_entries_out_of_range_are_left_out():
    report("grouped: order entries out of range")
    for counts in ([4, 9, 3], [200, 150]):
        n, R, C = sum(counts), 40, 64
        off, order = rc.groups(counts, 1)
        order[2] = -1
        order[7] = n
        order[11] = 2 ** 31 - 1
        w = make_w16(len(counts), R, C, torch.float16, 1)
        x = torch.randn(n, C, generator=rc.gen(2), device="cuda").half()
        for flags in (SCATTER, 0, GATHER):
            y = torch.full((n, R), 3.0, device="cuda")
            pm.pm_grouped_gemm(w, x, y, off, order, 1, flags)
            want = rc.grouped_plain(lambda e: w[e].double(), x, off, order, n, 1,
                                    bool(flags & GATHER), bool(flags & SCATTER), False)
            rc.check_grouped(y, 3.0, want, f"flags {flags}")


def test_grouped16_values_that_do_not_mix():
    """Infinities and NaN in one row of x or one row of W stay in that row's
    or column's outputs; rows no use maps to reach nothing; tiny values are
    not flushed."""
    report("grouped: inf, NaN, subnormals")
    for counts in ([3, 6, 2], [150, 40, 140]):
        n, R, C = sum(counts), 70, 136
        off, _ = rc.groups(counts, 1)
        for ty in (torch.float16, torch.bfloat16):
            w = make_w16(3, R, C, ty, 1)
            x = torch.randn(n, C, generator=rc.gen(2), device="cuda").to(ty)
            clean = torch.empty(n, R, device="cuda")
            pm.pm_grouped_gemm(w, x, clean, off)
            x2, w2 = x.clone(), w.clone()
            x2[1, 5] = float("nan")
            x2[counts[0], 135] = float("inf")
            w2[2, 69, 0] = float("nan")
            y = torch.empty(n, R, device="cuda")
            pm.pm_grouped_gemm(w2, x2, y, off)
            hit = torch.zeros(n, R, dtype=torch.bool, device="cuda")
            hit[1] = hit[counts[0]] = True
            hit[counts[0] + counts[1]:, 69] = True
            assert torch.equal(y[~hit], clean[~hit])
            assert y[1].isnan().all() and not y[counts[0]].isfinite().any()
            assert y[counts[0] + counts[1]:, 69].isnan().all()
        # fp16 subnormals times large values
        w = torch.full((3, R, C), 2.0 ** -24, dtype=torch.float16, device="cuda")
        x = torch.full((n, C), 1024.0, dtype=torch.float16, device="cuda")
        y = torch.empty(n, R, device="cuda")
        pm.pm_grouped_gemm(w, x, y, off)
        assert torch.all(y == C * 2.0 ** -14)


def test_grouped16_without_inputs_gives_zeros():
    report("grouped: cols 0")
    off, order = rc.groups([2, 3], 0)
    w = torch.empty(2, 10, 0, dtype=torch.float16, device="cuda")
    x = torch.empty(5, 0, dtype=torch.float16, device="cuda")
    y = torch.full((5, 10), 3.0, device="cuda")
    pm.pm_grouped_gemm(w, x, y, off, order, 1, SCATTER)
    assert not y.any()
    y = torch.full((5, 5), 3.0, device="cuda")
    pm.pm_grouped_gemm(w, x, y, off, order, 1, SWIGLU)
    assert not y.any()


def test_grouped16_many_rows_and_experts():
    """Hundreds of experts, most of them small or empty, some large."""
    report("grouped: 512 experts, ragged")
    rng = np.random.default_rng(0)
    counts = rng.integers(0, 6, 512)
    counts[[3, 100, 511]] = [400, 129, 260]
    run_grouped16(counts.tolist(), 128, 192, "bf16", "f32", 1, SCATTER, seed=9)
    run_grouped16((counts * 12).tolist(), 130, 192, "bf16", "bf16", 4, GATHER | SWIGLU, seed=9)
    run_grouped16([1] * 300, 64, 64, "f16", "f32", 10, GATHER, seed=9)


def test_grouped16_repeats_bit_for_bit_and_on_two_streams():
    report("grouped: repeats, two streams")
    counts = [5, 300, 0, 64]
    off, order = rc.groups(counts, 1)
    n = sum(counts)
    w = make_w16(4, 256, 512, torch.bfloat16, 1)
    x = torch.randn(n, 512, generator=rc.gen(2), device="cuda").bfloat16()
    ys = [torch.empty(n, 256, device="cuda") for _ in range(5)]
    pm.pm_grouped_gemm(w, x, ys[0], off, order, 1, SCATTER)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, y in enumerate(ys[1:]):
        pm.pm_grouped_gemm(w, x, y, off, order, 1, SCATTER, streams[i % 2])
    torch.cuda.synchronize()
    for y in ys[1:]:
        assert torch.equal(y, ys[0])


@pytest.mark.parametrize("counts,R", [([2100, 2000], 8192),      # 544 tiles: a short last round
                                      ([1800, 0, 2900, 3], 8190),  # outputs off the tile
                                      ([256, 4000], 8448)])
def test_grouped16_large_tiles(counts, R):
    """Enough 256-row tiles for several rounds of the device, the last of them
    short or long."""
    report(f"grouped large tiles {counts} {R}")
    run_grouped16(counts, R, 136, "bf16", "f32", 1, SCATTER, seed=11)
    run_grouped16(counts, R, 64, "f16", "f16", 2, GATHER | SWIGLU, seed=12)


@pytest.mark.parametrize("n", [63, 64, 65, 128, 129])
def test_grouped16_short_calls(n):
    """Around the number of rows up to which the uses are loaded at the start."""
    report(f"grouped {n} rows")
    counts = [1] * (n - 20) + [0, 13, 7]
    run_grouped16(counts, 40, 2048, "bf16", "f32", 3, GATHER, seed=13)
    run_grouped16(counts, 40, 4096, "f16", "f32", 1, SCATTER, seed=13)


def test_grouped16_offsets_beyond_32_bits():
    """Rows of x and y so far apart that their byte offsets pass 2^32, through
    the kernels of few and of many rows."""
    report("grouped: offsets beyond 32 bits")
    C, R, ld = 64, 48, 1 << 30
    xbuf = torch.empty(2 * ld + C, dtype=torch.bfloat16, device="cuda")
    x = xbuf.as_strided((3, C), (ld, 1))
    x.copy_(torch.randn(3, C, generator=rc.gen(1), device="cuda"))
    w = make_w16(2, R, C, torch.bfloat16, 2)
    for counts, top_k in (([3, 3], 2), ([400, 300], 234)):
        off, order = rc.groups(counts, 3)
        n = sum(counts)
        y = torch.full((n, R), 3.0, device="cuda")
        pm.pm_grouped_gemm(w, x, y, off, order, top_k, GATHER | SCATTER)
        want = rc.grouped_plain(lambda e: w[e].double(), x, off, order, n, top_k, True, True, False)
        rc.check_grouped(y, 3.0, want, f"x, {n} rows")
    del xbuf, x
    ybuf = torch.empty(2 * ld + R, dtype=torch.bfloat16, device="cuda")
    y = ybuf.as_strided((3, R), (ld, 1))
    y.fill_(3.0)
    x = torch.randn(3, C, generator=rc.gen(1), device="cuda").bfloat16()
    off, order = rc.groups([2, 1], 4)
    pm.pm_grouped_gemm(w, x, y, off, order, 1, SCATTER)
    want = rc.grouped_plain(lambda e: w[e].double(), x, off, order, 3, 1, False, True, False)
    rc.check_grouped(y, 3.0, want, "y")
    del ybuf, y
    # tiles whose rows lie beyond 2^32 bytes of x and y
    ld, counts = 1 << 22, [400, 300]
    x = torch.empty(700 * ld, dtype=torch.bfloat16, device="cuda").as_strided((700, C), (ld, 1))
    x.copy_(torch.randn(700, C, generator=rc.gen(5), device="cuda"))
    y = torch.empty(700 * ld, dtype=torch.bfloat16, device="cuda").as_strided((700, R), (ld, 1))
    off, order = rc.groups(counts, 6)
    for flags in (0, SCATTER):
        y.fill_(3.0)
        pm.pm_grouped_gemm(w, x, y, off, order, 1, flags)
        want = rc.grouped_plain(lambda e: w[e].double(), x, off, order, 700, 1, False, bool(flags),
                                False)
        rc.check_grouped(y, 3.0, want, f"tiles, flags {flags}")


def test_grouped16_most_experts():
    report("grouped: 4096 experts")
    counts = np.zeros(4096, np.int64)
    counts[[0, 1, 63, 64, 2047, 4094, 4095]] = [1, 2, 3, 20, 1, 5, 1]
    run_grouped16(counts.tolist(), 16, 64, "bf16", "f32", 1, 0, seed=14)
    counts[[5, 4000]] = [90000, 120000]
    run_grouped16(counts.tolist(), 16, 64, "bf16", "f32", 1, 0, seed=14)


# ---------------------------------------------------------------- 4-bit weights
def make_w4(E, R, C, group, zeros, seed):
    g = rc.gen(seed)
    q = torch.randint(0, 256, (E, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(E, R, C // group, generator=g, device="cuda") * 0.02 + 0.001).half()
    z = None
    if zeros:
        z = torch.randint(0, 16, (E, R, C // group), generator=g, device="cuda",
                          dtype=torch.uint8)
    return q, s, z


def run_w4(counts, R, C, group, zeros, ty, y_ty, top_k, flags, seed=0, n_rows=None, pad=0,
           order=True, spread=False):
    dt = rc.TYPES[ty]
    off, ordr = rc.groups(counts, seed, n_rows)
    n = ordr.numel()
    if not order:
        ordr = None
    q, s, z = make_w4(len(counts), R, C, group, zeros, seed + 1)
    nx = (n + top_k - 1) // top_k if flags & GATHER else n
    x = torch.randn(nx, C + 8 * pad, generator=rc.gen(seed + 2), device="cuda")
    if spread:
        # magnitudes over many powers of two within a row
        x *= torch.exp2(torch.randint(-20, 14, x.shape, generator=rc.gen(seed + 3),
                                      device="cuda").float())
    x = x.to(dt)[:, :C]
    out = R // 2 if flags & SWIGLU else R
    ybuf = torch.full((n, out + pad), 3.0, dtype=rc.TYPES[y_ty], device="cuda")
    y = ybuf[:, :out]
    pm.pm_grouped_gemm_w4(q, s, z, group, x, y, off, ordr, top_k, flags)
    torch.cuda.synchronize()
    want = rc.grouped_plain(
        lambda e: rc.decode_w4(q[e], s[e], None if z is None else z[e], group), x, off, ordr, n,
        top_k, bool(flags & GATHER), bool(flags & SCATTER), bool(flags & SWIGLU))
    rc.check_grouped(y, 3.0, want, f"{counts} {R}x{C}/{group} {ty}->{y_ty} flags {flags}")
    assert torch.all(ybuf[:, out:] == 3.0)


@pytest.mark.parametrize("ty,y_ty", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32"),
                                     ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("flags,top_k", LAYOUTS)
def test_w4_layouts(ty, y_ty, flags, top_k):
    report(f"w4 {ty}->{y_ty} flags {flags}")
    run_w4([3, 0, 1, 17, 0, 40, 2], 96, 256, 64, bool(flags & SCATTER), ty, y_ty, top_k, flags,
           seed=flags)


@pytest.mark.parametrize("group,C", [(32, 32), (32, 96), (32, 1056), (64, 64), (64, 448),
                                     (96, 288), (128, 128), (128, 1408), (256, 512), (1024, 1024),
                                     (128, 4096)])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_groups(group, C, zeros):
    report(f"w4 group {group} cols {C} zeros {zeros}")
    for ty in ("f32", "bf16"):
        run_w4([1, 2, 0, 5, 19], 50, C, group, zeros, ty, "f32", 1, SCATTER, seed=1)
    run_w4([1, 2, 0, 5, 19], 34, C, group, zeros, "f16", "f16", 2, GATHER | SWIGLU, seed=2)


@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [4, 5, 6], [7, 8, 9], [15, 16, 17],
                                    [31, 32, 33], [63, 64, 65], [130, 1, 0, 257], [0, 0]])
def test_w4_group_sizes(counts):
    report(f"w4 counts {counts}")
    n = max(1, sum(counts))
    for ty in ("f32", "f16", "bf16"):
        run_w4(counts, 72, 256, 128, False, ty, "f32", 1, SCATTER, seed=1, n_rows=n)
    run_w4(counts, 144, 256, 64, True, "bf16", "bf16", 2, GATHER | SWIGLU, seed=2, n_rows=n)


@pytest.mark.parametrize("R", [1, 2, 15, 16, 17, 31, 33, 64, 100, 257])
def test_w4_odd_rows(R):
    report(f"w4 rows {R}")
    run_w4([2, 0, 9, 1], R, 384, 128, True, "f32", "f32", 1, 0, seed=3, pad=1, n_rows=17)
    if R % 2 == 0:
        run_w4([2, 0, 9, 1], R, 384, 128, False, "bf16", "f32", 3, GATHER | SWIGLU, seed=4,
               order=False)


@pytest.mark.parametrize("group,C", [(128, 4224), (64, 8320), (32, 4128), (96, 4896), (256, 8192),
                                     (128, 12288), (2176, 4352)])
def test_w4_many_inputs(group, C):
    """More inputs than the waves hold at once."""
    report(f"w4 group {group} cols {C}")
    for ty in ("f32", "bf16"):
        run_w4([1, 0, 3, 17], 34, C, group, True, ty, "f32", 1, SCATTER, seed=6)
    run_w4([9, 2], 40, C, group, False, "f16", "f16", 2, GATHER | SWIGLU, seed=7)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("E,group,C", [(65, 32, 128), (65, 64, 128), (65, 128, 128), (65, 96, 96),
                                       (33, 32, 256), (33, 64, 256), (33, 128, 256), (33, 96, 192),
                                       (33, 128, 384), (33, 32, 512), (33, 64, 512), (33, 96, 480),
                                       (4, 32, 1024), (4, 128, 1280), (4, 96, 1152)])
def test_w4_few_rows(E, group, C, zeros):
    """Few rows, with many experts where the inputs are few."""
    report(f"w4 few rows {E} experts group {group} cols {C} zeros {zeros}")
    counts = np.random.default_rng(E + C).integers(0, 4, E)
    counts[[0, E // 2, E - 1]] = [17, 5, 1]
    run_w4(counts.tolist(), 4096, C, group, zeros, "f16", "f32", 1, SCATTER, seed=8)
    run_w4(counts.tolist(), 4094, C, group, zeros, "bf16", "bf16", 2, GATHER | SWIGLU, seed=9)
    run_w4(counts.tolist(), 4096, C, group, zeros, "f32", "f32", 1, 0, seed=10)


@pytest.mark.parametrize("ty,y_ty", [("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16"),
                                     ("f32", "f32")])
@pytest.mark.parametrize("flags,top_k", LAYOUTS)
def test_w4_many_rows_layouts(ty, y_ty, flags, top_k):
    report(f"w4 tiles {ty}->{y_ty} flags {flags}")
    counts = [130, 0, 70, 257, 1, 128]
    run_w4(counts, 96, 256, 64, bool(flags & SCATTER), ty, y_ty, top_k, flags, seed=1)
    run_w4(counts, 562, 640, 128, not flags & SCATTER, ty, y_ty, top_k, flags, seed=2, n_rows=600)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,C", [(128, 128), (128, 4224), (64, 384), (32, 256), (32, 32),
                                     (96, 288), (64, 192), (256, 1024), (160, 800)])
def test_w4_many_rows_groups(group, C, zeros):
    report(f"w4 tiles group {group} cols {C} zeros {zeros}")
    run_w4([60, 48, 100], 258, C, group, zeros, "f16", "f32", 2, GATHER, seed=3)
    run_w4([200, 16, 129], 130, C, group, zeros, "bf16", "bf16", 1, SCATTER | SWIGLU, seed=4)
    run_w4([64, 16, 129], 258, C, group, zeros, "f32", "f32", 1, SCATTER, seed=5)


@pytest.mark.parametrize("ty", ["f16", "bf16", "f32"])
def test_w4_many_rows_rounds_and_bad_entries(ty):
    """Several rounds of tiles; rows and order entries left out; a wide x; no
    order; infinities beside other rows."""
    report(f"w4 tiles {ty}: rounds, entries out of range, strides")
    run_w4([1500, 3, 0, 900, 128, 64], 4100, 256, 128, True, ty, ty, 3, GATHER, seed=5)
    run_w4([1500, 3, 0, 900, 128, 64], 4096, 128, 32, False, ty, ty, 1, SWIGLU, seed=6,
           pad=2, order=False)
    off, order = rc.groups([300, 200, 100], 1)
    order[2], order[7], order[411] = -1, 600, 2 ** 31 - 1
    q, sc, z = make_w4(3, 72, 320, 64, True, 1)
    x = torch.randn(600, 320, generator=rc.gen(2), device="cuda").to(rc.TYPES[ty])
    for flags in (SCATTER, 0, GATHER):
        y = torch.full((600, 72), 3.0, device="cuda")
        pm.pm_grouped_gemm_w4(q, sc, z, 64, x, y, off, order, 1, flags)
        want = rc.grouped_plain(lambda e: rc.decode_w4(q[e], sc[e], z[e], 64), x, off, order, 600,
                                1, bool(flags & GATHER), bool(flags & SCATTER), False)
        rc.check_grouped(y, 3.0, want, f"flags {flags}")
    off, _ = rc.groups([300, 200, 100], 1)
    clean = torch.empty(600, 72, device="cuda")
    pm.pm_grouped_gemm_w4(q, sc, z, 64, x, clean, off, None, 1, 0)
    bad = x.clone()
    bad[5], bad[299, 3], bad[450, 319] = float("nan"), float("inf"), -float("inf")
    y = torch.empty(600, 72, device="cuda")
    pm.pm_grouped_gemm_w4(q, sc, z, 64, bad, y, off, None, 1, 0)
    keep = torch.ones(600, dtype=torch.bool, device="cuda")
    keep[[5, 299, 450]] = False
    assert torch.equal(y[keep], clean[keep])
    assert not torch.isfinite(y[5]).any()
    # offsets that decrease or pass the rows: every access stays in bounds
    for o in ([0, 400, 100, 600], [-5, 300, 9999, 600], [600, 0, 0, 0]):
        pm.pm_grouped_gemm_w4(q, sc, z, 64, x, y, torch.tensor(o, dtype=torch.int32, device="cuda"),
                              order, 1, SCATTER)
    torch.cuda.synchronize()
    y.zero_()
    pm.pm_grouped_gemm_w4(q, sc, z, 64, x, y, off, None, 1, 0)
    assert torch.equal(y, clean)


def test_w4_many_rows_and_experts():
    report("w4: 512 experts, ragged")
    counts = np.random.default_rng(1).integers(0, 4, 512)
    counts[[0, 200, 511]] = [70, 33, 129]
    run_w4(counts.tolist(), 48, 256, 128, True, "bf16", "bf16", 4, GATHER | SWIGLU, seed=8)
    run_w4(counts.tolist(), 33, 384, 64, False, "f32", "f32", 1, SCATTER, seed=9)


def test_w4_strides_and_rows_outside():
    report("w4 strides, untouched rows, order entries out of range")
    run_w4([2, 5, 0, 9], 50, 96, 32, True, "f16", "f32", 2, GATHER, seed=6, pad=3, n_rows=70)
    run_w4([2, 5, 0, 9], 50, 96, 32, False, "f32", "f32", 1, 0, seed=6, pad=1, order=False)
    off, order = rc.groups([4, 9, 3], 1)
    order[2], order[7], order[11] = -1, 16, 2 ** 31 - 1
    q, sc, z = make_w4(3, 40, 64, 32, True, 1)
    x = torch.randn(16, 64, generator=rc.gen(2), device="cuda")
    for flags in (SCATTER, 0, GATHER):
        y = torch.full((16, 40), 3.0, device="cuda")
        pm.pm_grouped_gemm_w4(q, sc, z, 32, x, y, off, order, 1, flags)
        want = rc.grouped_plain(lambda e: rc.decode_w4(q[e], sc[e], z[e], 32), x, off, order, 16,
                                1, bool(flags & GATHER), bool(flags & SCATTER), False)
        rc.check_grouped(y, 3.0, want, f"flags {flags}")


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_w4_wide_ranges_many_inputs(ty):
    """The same through the streamed kernel (few rows) and through tiles, with
    infinities and NaN in single rows."""
    report(f"w4 wide ranges {ty}, many inputs")
    run_w4([1, 3, 12], 48, 1280, 128, True, ty, "f32", 1, 0, seed=5, spread=True)
    run_w4([65, 3, 130], 48, 1280, 64, False, ty, "f32", 1, 0, seed=6, spread=True)
    q, s, z = make_w4(2, 32, 1280, 64, True, 1)
    for counts in ([4, 3], [70, 60]):
        off, _ = rc.groups(counts, 0)
        n = sum(counts)
        x = torch.randn(n, 1280, generator=rc.gen(2), device="cuda")
        x[:5] *= torch.tensor([1e30, 1e-30, 0.0, 1e5, 1e-7], device="cuda")[:, None]
        x = x.to(rc.TYPES[ty])
        y = torch.full((n, 32), 3.0, device="cuda")
        pm.pm_grouped_gemm_w4(q, s, z, 64, x, y, off)
        want = rc.grouped_plain(lambda e: rc.decode_w4(q[e], s[e], z[e], 64), x, off, None, n, 1,
                                False, False, False)
        rc.check_grouped(y, 3.0, want, "row ranges")
        assert not y[2].any()
        bad = x.clone()
        bad[3, 700], bad[6, 1279] = float("nan"), float("inf")
        got = torch.empty_like(y)
        pm.pm_grouped_gemm_w4(q, s, z, 64, bad, got, off)
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[[3, 6]] = False
        assert torch.equal(got[keep], y[keep])
        assert torch.isnan(got[3]).all() and not torch.isfinite(got[6]).all()


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
def test_w4_wide_ranges(ty):
    """Activations over 34 powers of two in one row: every output within the
    bound of its own products."""
    report(f"w4 wide ranges {ty}")
    run_w4([1, 3, 20], 48, 512, 128, True, ty, "f32", 1, 0, seed=5, spread=ty != "f16")
    # large and small rows of fp32 and bf16 activations, beyond fp16's range
    if ty == "f16":
        return
    counts = [2, 3]
    off, _ = rc.groups(counts, 0)
    q, s, z = make_w4(2, 32, 256, 64, True, 1)
    x = torch.randn(5, 256, generator=rc.gen(2), device="cuda")
    x *= torch.tensor([1e30, 1e-30, 1.0, 1e5, 1e-7], device="cuda")[:, None]
    x = x.to(rc.TYPES[ty])
    x[2] = 0.0
    y = torch.full((5, 32), 3.0, device="cuda")
    pm.pm_grouped_gemm_w4(q, s, z, 64, x, y, off)
    want = rc.grouped_plain(lambda e: rc.decode_w4(q[e], s[e], z[e], 64), x, off, None, 5, 1,
                            False, False, False)
    rc.check_grouped(y, 3.0, want, "row ranges")
    assert not y[2].any()


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
def test_w4_one_hot_and_non_finite(ty):
    """A one-hot x gives the weight itself; an infinity or NaN stays in its row."""
    report(f"w4 one-hot, inf, NaN {ty}")
    dt = rc.TYPES[ty]
    q, s, z = make_w4(1, 40, 256, 64, True, 1)
    w = rc.decode_w4(q[0], s[0], z[0], 64)
    cols = [0, 1, 7, 8, 31, 32, 63, 100, 127, 128, 200, 254, 255]
    x = torch.zeros(len(cols), 256, dtype=dt, device="cuda")
    for i, c in enumerate(cols):
        x[i, c] = 1.0
    off = torch.tensor([0, len(cols)], dtype=torch.int32, device="cuda")
    y = torch.empty(len(cols), 40, device="cuda")
    pm.pm_grouped_gemm_w4(q, s, z, 64, x, y, off)
    assert torch.equal(y.double(), w[:, cols].T)
    base = torch.randn(6, 256, generator=rc.gen(3), device="cuda").to(dt)
    off = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    y0, y1 = torch.empty(6, 40, device="cuda"), torch.empty(6, 40, device="cuda")
    pm.pm_grouped_gemm_w4(q, s, z, 64, base, y0, off)
    bad = base.clone()
    bad[1, 70] = float("nan")
    bad[4, 3] = float("inf")
    pm.pm_grouped_gemm_w4(q, s, z, 64, bad, y1, off)
    keep = [0, 2, 3, 5]
    assert torch.equal(y1[keep], y0[keep])
    assert y1[1].isnan().all()
    # inf * (q - z) * s: an infinity of the weight's sign, NaN where it is 0
    want = torch.full((40,), float("inf"), device="cuda") * w[:, 3].float()
    assert torch.equal(y1[4].nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_encoder(ty, zeros):
    """Codes, scales and zero points as documented, and the decoded weights
    within half a step of the weights."""
    report(f"encode w4 {ty} zeros {zeros}")
    R, C, group = 37, 384, 64
    w = torch.randn(R, C, generator=rc.gen(1), device="cuda").to(rc.TYPES[ty])
    w[3, :64] = 0.0
    w[4, :64] = 0.5
    w[5, 64:128] = -0.25
    q = torch.empty(R, C // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(R, C // group, dtype=torch.float16, device="cuda")
    z = torch.empty(R, C // group, dtype=torch.uint8, device="cuda") if zeros else None
    pm.pm_encode_w4_device(w, group, q, s, z)
    wf = w.float().cpu().numpy().reshape(R, -1, group)
    if zeros:
        lo, hi = np.minimum(wf.min(2), 0), np.maximum(wf.max(2), 0)
        ws = ((hi - lo) / np.float32(15)).astype(np.float16)
    else:
        ws = (np.abs(wf).max(2) / np.float32(7)).astype(np.float16)
    assert np.array_equal(s.cpu().numpy().view(np.uint16), ws.view(np.uint16))
    sf = ws.astype(np.float32)
    nz = sf > 0
    safe = np.where(nz, sf, 1)
    wz = np.full(sf.shape, 8.0, np.float32)
    if zeros:
        wz = np.where(nz, np.clip(np.rint(-lo / safe), 0, 15), 0).astype(np.float32)
        assert np.array_equal(z.cpu().numpy(), wz.astype(np.uint8))
    code = np.where(nz[:, :, None], np.clip(np.rint(wf / safe[:, :, None]) + wz[:, :, None], 0, 15),
                    wz[:, :, None])
    got = q.cpu().numpy()
    got = np.stack((got & 15, got >> 4), -1).reshape(R, -1, group)
    assert np.array_equal(got, code.astype(np.uint8))
    # the scale's own rounding (2^-11 of it) moves the ends of the range by
    # up to 15 * 2^-11 of a step, and the zero point by another half
    dec = (got - wz[:, :, None]) * sf[:, :, None]
    lim = (0.5 + 0.5 * zeros + 15 * 2.0 ** -11) * sf[:, :, None] + 1e-9
    assert np.all(np.abs(dec - wf) <= lim)


# ---------------------------------------------------------------- combine
@pytest.mark.parametrize("T,K,H", [(1, 1, 1), (1, 10, 4096), (7, 3, 33), (8, 10, 256), (130, 10, 1001),
                                   (65, 1, 8), (3, 64, 100), (1025, 2, 516)])
@pytest.mark.parametrize("z_ty,y_ty", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"),
                                       ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_combine(T, K, H, z_ty, y_ty, pad):
    report(f"combine {T} x {K} x {H} {z_ty}->{y_ty} pad {pad}")
    g = rc.gen(T + K + H)
    zb = torch.randn(T * K, H + pad, generator=g, device="cuda").to(rc.TYPES[z_ty])
    z = zb[:, pad:] if pad == 1 else zb[:, :H]
    w = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
    if K > 1:
        w[0, 1] = 0.0
        z[1] = float("nan")                       # a slot the router left empty
    yb = torch.full((T, H + pad), 3.0, dtype=rc.TYPES[y_ty], device="cuda")
    y = yb[:, :H]
    pm.pm_combine_uses(z, w, y)
    z64 = z.double().nan_to_num().reshape(T, K, H)
    terms = w.double()[:, :, None] * z64
    want, S = terms.sum(1), terms.abs().sum(1)
    half = rc.HALF_STEP[y.dtype]
    # K products and sums in fp32, one rounding to y
    tol = (K + 1) * 2.0 ** -24 * S + 2.0 ** -126
    tol = tol + half * (want.abs() + tol) + torch.finfo(y.dtype).smallest_normal * half
    assert torch.all((y.double() - want).abs() <= tol)
    assert torch.all(yb[:, H:] == 3.0)


@pytest.mark.parametrize("H", [4, 8])
def test_combine_many_tokens(H):
    """More tokens than one grid's waves."""
    report(f"combine 5 000 000 x {H}")
    T = 5_000_000
    z = torch.randn(T, H, generator=rc.gen(H), device="cuda").bfloat16()
    w = torch.full((T, 1), 0.5, device="cuda")
    y = torch.full((T, H), 3.0, dtype=torch.bfloat16, device="cuda")
    pm.pm_combine_uses(z, w, y)
    assert torch.equal(y, z * 0.5)


# ---------------------------------------------------------------- whole layers
class Layer:
    """A routed layer's operators in a row, on fixed buffers."""

    def __init__(self, T, E, K, hidden, inter, bits, dt, seed=0):
        self.T, self.E, self.K, self.bits = T, E, K, bits
        g = rc.gen(seed)
        self.logits = torch.empty(T, E, device="cuda")
        self.x = torch.empty(T, hidden, dtype=dt, device="cuda")
        gu = torch.empty(E, 2 * inter, hidden, dtype=dt, device="cuda").normal_(0, 0.05, generator=g)
        dn = torch.empty(E, hidden, inter, dtype=dt, device="cuda").normal_(0, 0.05, generator=g)
        self.group = 64
        if bits == 4:
            self.gu, self.dn = self.encode(gu), self.encode(dn)
        else:
            self.gu, self.dn = gu, dn
        n = T * K
        i32 = torch.int32
        self.ids = torch.empty(T, K, dtype=i32, device="cuda")
        self.w = torch.empty(T, K, device="cuda")
        self.off = torch.empty(E + 1, dtype=i32, device="cuda")
        self.order = torch.empty(n, dtype=i32, device="cuda")
        self.ws = torch.empty(pm.pm_route_workspace_bytes(T, E, K), dtype=torch.uint8,
                              device="cuda")
        self.h = torch.empty(n, inter, dtype=dt, device="cuda")
        self.z = torch.empty(n, hidden, dtype=torch.float32, device="cuda")
        self.y = torch.empty(T, hidden, device="cuda")

    def encode(self, w):
        E, R, C = w.shape
        q = torch.empty(E, R, C // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(E, R, C // self.group, dtype=torch.float16, device="cuda")
        z = torch.empty(E, R, C // self.group, dtype=torch.uint8, device="cuda")
        for e in range(E):
            pm.pm_encode_w4_device(w[e], self.group, q[e], s[e], z[e])
        return q, s, z

    def new_tokens(self, seed, padding=0):
        g = rc.gen(seed)
        self.logits.copy_(torch.randn(self.logits.shape, generator=g, device="cuda"))
        if padding:
            self.logits[-padding:] = -float("inf")
        self.x.copy_(torch.randn(self.x.shape, generator=g, device="cuda"))

    def product(self, w, x, y, flags, stream):
        if self.bits == 4:
            pm.pm_grouped_gemm_w4(*w, self.group, x, y, self.off, self.order, self.K, flags, stream)
        else:
            pm.pm_grouped_gemm(w, x, y, self.off, self.order, self.K, flags, stream)

    def run(self, stream=None):
        pm.pm_route_topk_device(self.logits, self.K, self.ids, self.w, self.off, self.order,
                                self.ws, stream)
        self.product(self.gu, self.x, self.h, GATHER | SWIGLU, stream)
        self.product(self.dn, self.h, self.z, SCATTER, stream)
        pm.pm_combine_uses(self.z, self.w, self.y, stream)

    def weights64(self, w, e):
        if self.bits == 4:
            return rc.decode_w4(w[0][e], w[1][e], w[2][e], self.group)
        return w[e].double()

    def check(self):
        """y against the dense fp64 layer; the rounding of h to its type moves
        an output by up to half a step of every term."""
        ids, w, _, _ = rc.route_plain(self.logits, self.K)
        half = rc.HALF_STEP[self.h.dtype]
        for t in range(self.T):
            want = torch.zeros(self.x.shape[1], dtype=torch.float64, device="cuda")
            tol = torch.full_like(want, 2.0 ** -100)
            for j in range(self.K):
                e = int(ids[t, j])
                if e < 0:
                    continue
                gu, dn = self.weights64(self.gu, e), self.weights64(self.dn, e)
                x = self.x[t].double()
                p, S = gu @ x, (gu.abs() @ x.abs()) * (gu.shape[1] + 16) * 2.0 ** -23
                n = p.shape[0] // 2
                gate, up = p[:n], p[n:]
                s = gate * torch.sigmoid(gate)
                h = s * up
                dh = 1.1 * S[:n] * (up.abs() + S[n:]) + s.abs() * S[n:] + h.abs() * (half + 2.0 ** -20)
                want += w[t, j] * (dn @ h)
                tol += w[t, j] * (dn.abs() @ (dh + h.abs() * (dn.shape[1] + 32) * 2.0 ** -23))
            got = self.y[t].double()
            assert torch.all((got - want).abs() <= tol), (t, float(((got - want).abs() / tol).max()))


@pytest.mark.parametrize("bits,dt", [(16, torch.bfloat16), (16, torch.float16),
                                     (4, torch.float32), (4, torch.bfloat16)])
@pytest.mark.parametrize("T,E,K,padding", [(1, 16, 2, 0), (9, 32, 4, 2), (70, 8, 3, 0)])
def test_layer_of_device_operators(bits, dt, T, E, K, padding):
    report(f"layer {bits}-bit {dt} {T} tokens x {E} experts top-{K}")
    L = Layer(T, E, K, 256, 128, bits, dt)
    L.h.fill_(float("nan"))                       # nothing may be read before it is written
    L.z.fill_(float("nan"))
    L.new_tokens(1, padding)
    L.run()
    L.check()


@pytest.mark.parametrize("bits,dt", [(16, torch.bfloat16), (4, torch.float32)])
def test_captured_layer_serves_new_tokens(bits, dt):
    """One graph of two layers (one with 150 tokens, its own workspace each):
    every replay on new tokens, with eager work and synchronisations between,
    against the eager result bit for bit and the fp64 layer."""
    report(f"captured layer {bits}-bit")
    Ls = [Layer(5, 16, 3, 256, 128, bits, dt), Layer(150, 8, 2, 128, 64, bits, dt, seed=3)]
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for L in Ls:
            L.new_tokens(1)
            L.run(st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        for L in Ls:
            L.run(st)
    for rep in range(3):
        for i, L in enumerate(Ls):
            L.new_tokens(10 + rep, padding=rep * i)
            L.y.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for L in Ls:
            got = L.y.clone()
            L.check()
            L.y.zero_()
            L.run()
            torch.cuda.synchronize()
            assert torch.equal(L.y, got), rep


def test_layers_on_two_streams_at_once():
    """Two layers, each with its own buffers, issued in turn on two streams
    give what each gives alone."""
    report("two layers on two streams")
    Ls = [Layer(40, 32, 4, 512, 256, 16, torch.bfloat16), Layer(6, 32, 4, 512, 256, 4, torch.float32)]
    for i, L in enumerate(Ls):
        L.new_tokens(20 + i)
        L.run()
    torch.cuda.synchronize()
    alone = [L.y.clone() for L in Ls]
    streams = [torch.cuda.Stream() for _ in Ls]
    for rep in range(5):
        for L in Ls:
            L.y.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for L, st in zip(Ls, streams):
                L.run(st)
        torch.cuda.synchronize()
        for L, want in zip(Ls, alone):
            assert torch.equal(L.y, want), rep


def test_grouped_on_materialized_prefixes():
    """Experts read at a prefix and materialised as fp16 go through the grouped
    product: the same values as the single-matrix comparator."""
    report("grouped over pm_materialize_fp16")
    R, C, group, E = 128, 256, 64, 3
    sh = pm.mshape(R, C, group)
    w = torch.empty(E, R, C, dtype=torch.float16, device="cuda")
    pw = R * C // 32
    for e in range(E):
        planes = np.zeros((8, pw), np.uint32)
        levels = np.zeros(pm.pm_levels_floats(sh), np.float32)
        pm.pm_encode_matrix(sh, synth.codes(5, 0, 0, e, 0, R, C),
                            synth.leaves(5, 0, 0, e, 0, R, C // group), None, planes, pw, levels)
        dp, dl = torch.from_numpy(planes.view(np.int32)).cuda(), torch.from_numpy(levels).cuda()
        pm.pm_materialize_fp16(sh, 3 + e, dp, pw, dl, w[e])
        torch.cuda.synchronize()
    x = torch.randn(E, C, generator=rc.gen(1), device="cuda").half()
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    y = torch.empty(E, R, device="cuda")
    pm.pm_grouped_gemm(w, x, y, off)
    for e in range(E):
        ref = torch.empty(R, device="cuda")
        pm.pm_gemv_fp16(sh, w[e], x[e].float(), ref)
        S = w[e].double().abs() @ x[e].double().abs()
        assert torch.all((ref.double() - y[e].double()).abs() <= 2 * (C + 16) * 2.0 ** -23 * S)
