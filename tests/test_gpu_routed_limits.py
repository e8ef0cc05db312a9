"""Routed experts' device operators at the ends of their ranges: values, sizes
and offsets where a mistake would not show in random products."""
import numpy as np
import pytest
import torch

import bitplane_quantized_expert_amd as pm
import routed_cases as rc

pytestmark = pytest.mark.gpu
GATHER, SCATTER, SWIGLU = pm.PM_GROUPED_GATHER, pm.PM_GROUPED_SCATTER, pm.PM_GROUPED_SWIGLU


def report(name):
    print(f"[gpu case] {name}", flush=True)


# ---------------------------------------------------------------- 4-bit encoder
@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_encoder_of_large_weights(ty, zeros):
    """Finite weights beyond 7 (15) of fp16's largest scale saturate: the scale
    is finite, zeros stay zeros and every code is the nearest there is."""
    report(f"encode w4 large weights {ty} zeros {zeros}")
    top = torch.finfo(rc.TYPES[ty]).max
    w = torch.randn(8, 64, generator=rc.gen(1), device="cuda")
    w[:, 5] = 0.0
    # (lowest, highest) of each row
    for r, (lo, hi) in enumerate([(-1e5, 3e5), (0.0, 4.58e5), (-5e5, 5e5), (-1e6, 1e6),
                                  (-top, top), (0.0, top), (-top, 0.0), (-9.9e5, 0.0)]):
        w[r, 0], w[r, 63] = max(lo, -top), min(hi, top)
    w = w.to(rc.TYPES[ty])
    q = torch.empty(8, 32, dtype=torch.uint8, device="cuda")
    s = torch.empty(8, 2, dtype=torch.float16, device="cuda")
    z = torch.empty(8, 2, dtype=torch.uint8, device="cuda") if zeros else None
    pm.pm_encode_w4_device(w, 32, q, s, z)
    # the documented formula in 64 bits (hi - lo overflows 32); one rounding
    # to fp32 before fp16 moves no scale here: all lie on one side of a tie
    v = w.double().cpu().numpy().reshape(8, 2, 32)
    lo, hi = np.minimum(v.min(2), 0), np.maximum(v.max(2), 0)
    scale = ((hi - lo) / 15 if zeros else np.abs(v).max(2) / 7)
    scale = np.minimum(scale, 65504).astype(np.float16)
    got = s.cpu().numpy()
    assert np.isfinite(got).all()
    assert np.array_equal(got.view(np.uint16), scale.view(np.uint16))
    sf = scale.astype(np.float64)
    zp = np.clip(np.rint(-lo / sf), 0, 15) if zeros else np.full(sf.shape, 8.0)
    if zeros:
        assert np.array_equal(z.cpu().numpy(), zp.astype(np.uint8))
    code = np.clip(np.rint(v / sf[:, :, None]) + zp[:, :, None], 0, 15).astype(np.uint8)
    b = q.cpu().numpy()
    assert np.array_equal(np.stack((b & 15, b >> 4), -1).reshape(8, 2, 32), code)
    dec = rc.decode_w4(q, s, z, 32)
    assert torch.isfinite(dec).all() and not dec[:, 5].any()


# ---------------------------------------------------------------- 4-bit products
FEW, MANY = [4, 0, 3], [70, 0, 60]        # rows per expert: streamed weights, tiles


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [128, 64, 32, 160])
@pytest.mark.parametrize("counts", [FEW, MANY])
def test_w4_bf16_rows_of_any_size(counts, group, zeros):
    """bf16 activations up to the type's largest value under scales that keep
    the result finite: nothing in between overflows, with zero points up to 255."""
    report(f"w4 bf16 up to its largest value {counts} group {group} zeros {zeros}")
    E, R, C = len(counts), 48, 1280
    g = rc.gen(group)
    q = torch.randint(0, 256, (E, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    # |q - z| <= 255 and scales of 2^-24 to 2^-20: sums below 2^128 * 255 * 1280 * 2^-20
    s = (torch.randint(1, 17, (E, R, C // group), generator=g, device="cuda") * 2.0 ** -24).half()
    z = None
    if zeros:
        z = torch.randint(0, 256, (E, R, C // group), generator=g, device="cuda",
                          dtype=torch.uint8)
    off, _ = rc.groups(counts, 0)
    n = sum(counts)
    x = torch.randn(n, C, generator=g, device="cuda")
    x[0] *= 1e37
    x[1] = torch.finfo(torch.bfloat16).max
    x[2] = torch.finfo(torch.bfloat16).max * x[2].sign()
    x[4, ::3] *= 1e37
    x[5] *= 1e37
    x[n - 1] *= 1e30
    x = x.to(torch.bfloat16)
    assert torch.isfinite(x).all()
    want = rc.grouped_plain(lambda e: rc.decode_w4(q[e], s[e], None if z is None else z[e], group),
                            x, off, None, n, 1, False, False, False)
    assert max(float(p.abs().max()) for _, p, _ in want) < 2.0 ** 127
    for ty in (torch.float32, torch.bfloat16):
        y = torch.full((n, R), 3.0, dtype=ty, device="cuda")
        pm.pm_grouped_gemm_w4(q, s, z, group, x, y, off)
        assert torch.isfinite(y).all()
        rc.check_grouped(y, 3.0, want, f"{ty}")


@pytest.mark.parametrize("group", [128, 64, 32, 160])
@pytest.mark.parametrize("counts", [FEW, MANY])
def test_w4_bf16_smallest_values(counts, group):
    """One-hot rows of bf16's subnormal and smallest normal values: exact, for
    (q - z) * scale of them is a multiple of 2^-133 below 2^-100."""
    report(f"w4 bf16 smallest values {counts} group {group}")
    E, R, C = len(counts), 48, 1280
    g = rc.gen(group + 1)
    q = torch.randint(0, 256, (E, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.exp2(torch.randint(0, 11, (E, R, C // group), generator=g, device="cuda").float()).half()
    z = torch.randint(0, 256, (E, R, C // group), generator=g, device="cuda", dtype=torch.uint8)
    off, _ = rc.groups(counts, 0)
    n = sum(counts)
    values = torch.tensor([2.0 ** -133, -3 * 2.0 ** -133, 127 * 2.0 ** -133, 2.0 ** -126,
                           -255 * 2.0 ** -133, 2.0 ** -120, 1.0], dtype=torch.float64)
    x = torch.zeros(n, C, dtype=torch.float64)
    col = torch.arange(n) * 97 % C
    x[torch.arange(n), col] = values[torch.arange(n) % len(values)]
    xb = x.to(torch.bfloat16)
    assert torch.equal(xb.double(), x)
    y = torch.empty(n, R, device="cuda")
    pm.pm_grouped_gemm_w4(q, s, z, group, xb.cuda(), y, off)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        w = rc.decode_w4(q[e], s[e], z[e], group)
        assert torch.equal(y[a:b].double(), x[a:b].cuda() @ w.T), e


@pytest.mark.parametrize("group", [128, 64, 32, 160])
@pytest.mark.parametrize("counts", [FEW, MANY])
def test_w4_fp32_rows_of_any_size(counts, group):
    """fp32 activations up to the type's largest value, and one-hot rows down to
    its smallest (exact: a value of one bit is one half)."""
    report(f"w4 fp32 up to its largest value {counts} group {group}")
    E, R, C = len(counts), 48, 1280
    g = rc.gen(group + 3)
    q = torch.randint(0, 256, (E, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.randint(1, 17, (E, R, C // group), generator=g, device="cuda") * 2.0 ** -24).half()
    z = torch.randint(0, 256, (E, R, C // group), generator=g, device="cuda", dtype=torch.uint8)
    off, _ = rc.groups(counts, 0)
    n = sum(counts)
    x = torch.randn(n, C, generator=g, device="cuda")
    x[0] *= 1e37
    x[1] = torch.finfo(torch.float32).max
    x[2] = torch.finfo(torch.float32).max * x[2].sign()
    x[4, ::3] *= 1e37
    x[n - 1] *= 1e30
    want = rc.grouped_plain(lambda e: rc.decode_w4(q[e], s[e], z[e], group), x, off, None, n, 1,
                            False, False, False)
    y = torch.full((n, R), 3.0, device="cuda")
    pm.pm_grouped_gemm_w4(q, s, z, group, x, y, off)
    rc.check_grouped(y, 3.0, want, "large")
    s = torch.exp2(torch.randint(0, 11, (E, R, C // group), generator=g, device="cuda").float()).half()
    values = torch.tensor([2.0 ** -149, -2.0 ** -140, 2.0 ** -126, -2.0 ** -100, 2.0 ** 100],
                          dtype=torch.float64)
    x = torch.zeros(n, C, dtype=torch.float64)
    x[torch.arange(n), torch.arange(n) * 97 % C] = values[torch.arange(n) % len(values)]
    pm.pm_grouped_gemm_w4(q, s, z, group, x.float().cuda(), y, off)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        w = rc.decode_w4(q[e], s[e], z[e], group)
        assert torch.equal(y[a:b].double(), x[a:b].cuda() @ w.T), e


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [128, 64, 32, 160])
@pytest.mark.parametrize("counts", [FEW, MANY])
def test_w4_zero_points_of_eight_bits(counts, group, ty):
    """Zero points of 0 to 255: q - z is exact, and with whole numbers so are
    the sums (below 255 * 3 * 1280 < 2^24)."""
    report(f"w4 zero points up to 255 {ty} {counts} group {group}")
    E, R, C = len(counts), 48, 1280
    g = rc.gen(group + 2)
    q = torch.randint(0, 256, (E, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.ones(E, R, C // group, dtype=torch.float16, device="cuda")
    z = torch.randint(0, 256, (E, R, C // group), generator=g, device="cuda", dtype=torch.uint8)
    off, _ = rc.groups(counts, 0)
    n = sum(counts)
    x = torch.randint(-3, 4, (n, C), generator=g, device="cuda").to(rc.TYPES[ty])
    y = torch.full((n, R), 0.5, device="cuda")
    pm.pm_grouped_gemm_w4(q, s, z, group, x, y, off)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        w = rc.decode_w4(q[e], s[e], z[e], group)
        assert torch.equal(y[a:b].double(), x[a:b].double() @ w.T), e


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
def test_w4_without_inputs_gives_zeros(ty):
    report(f"w4 cols 0 {ty}")
    for zeros in (False, True):
        for n in (5, 100):
            off = torch.tensor([0, 2, n], dtype=torch.int32, device="cuda")
            q = torch.empty(2, 10, 0, dtype=torch.uint8, device="cuda")
            s = torch.empty(2, 10, 0, dtype=torch.float16, device="cuda")
            z = torch.empty(2, 10, 0, dtype=torch.uint8, device="cuda") if zeros else None
            x = torch.empty(n, 0, dtype=rc.TYPES[ty], device="cuda")
            for flags, out in ((0, 10), (SWIGLU, 5)):
                y = torch.full((n, out), 3.0, device="cuda")
                pm.pm_grouped_gemm_w4(q, s, z, 32, x, y, off, None, 1, flags)
                assert not y.any()


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_w4_offsets_beyond_32_bits(ty):
    """Rows of x whose byte offsets pass 2^32, in calls of few and of many rows
    (which then take the streamed kernel)."""
    report(f"w4 offsets beyond 32 bits {ty}")
    C, R, group, ld = 192, 48, 64, 1 << 30
    x = torch.empty(2 * ld + C, dtype=rc.TYPES[ty], device="cuda").as_strided((3, C), (ld, 1))
    x.copy_(torch.randn(3, C, generator=rc.gen(1), device="cuda"))
    g = rc.gen(2)
    q = torch.randint(0, 256, (2, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(2, R, C // group, generator=g, device="cuda") * 0.02 + 0.001).half()
    for counts, top_k in (([3, 3], 2), ([400, 300], 234)):
        off, order = rc.groups(counts, 3)
        n = sum(counts)
        y = torch.full((n, R), 3.0, device="cuda")
        pm.pm_grouped_gemm_w4(q, s, None, group, x, y, off, order, top_k, GATHER | SCATTER)
        want = rc.grouped_plain(lambda e: rc.decode_w4(q[e], s[e], None, group), x, off, order, n,
                                top_k, True, True, False)
        rc.check_grouped(y, 3.0, want, f"{n} rows")


# ---------------------------------------------------------------- offsets that decrease
def bad_offsets(E, n, seed):
    """Lists of E + 1 offsets that decrease, repeat, are negative or pass n."""
    rng = np.random.default_rng(seed)
    lists = [rng.integers(-2 * n, 3 * n, E + 1) for _ in range(3)]
    lists += [np.where(np.arange(E + 1) % 2, n, 0), np.full(E + 1, n), np.full(E + 1, -1),
              np.arange(E, -1, -1) * n // E, np.full(E + 1, 2 ** 31 - 1),
              np.where(np.arange(E + 1) % 2, 2 ** 31 - 1, -2 ** 31)]
    return [torch.from_numpy(o.astype(np.int32)).cuda() for o in lists]


# name, weights (16 bits, or the group), x, experts, rows, outputs, inputs
KERNELS = [("streamed", 16, "bf16", 3, 7, 40, 2056), ("streamed", 16, "f16", 70, 90, 40, 4104),
           ("128-row tiles", 16, "bf16", 3, 200, 258, 136),
           ("256-row tiles", 16, "f16", 2, 2100, 16640, 64),
           ("streamed", 128, "bf16", 3, 7, 40, 1280), ("streamed", 64, "f16", 70, 90, 40, 4160),
           ("streamed", 128, "f32", 3, 7, 40, 1280), ("streamed", 96, "f32", 70, 90, 40, 4128),
           ("tiles", 128, "bf16", 3, 200, 258, 256), ("tiles", 32, "f32", 3, 200, 258, 256)]


@pytest.mark.parametrize("name,bits,ty,E,n,R,C", KERNELS)
def test_grouped_offsets_that_decrease(name, bits, ty, E, n, R, C):
    """Any offsets: rows of y outside the call's stay, no row of x outside it is
    read (they are NaN here), and the next call is right."""
    report(f"bad offsets: {name} {bits} {ty} {E} experts {n} rows {R} x {C}")
    g = rc.gen(E + n)
    dt = rc.TYPES[ty]
    xbuf = torch.full((n + 600, C), float("nan"), dtype=dt, device="cuda")
    x = xbuf[300:300 + n]
    x.copy_(torch.randn(n, C, generator=g, device="cuda"))
    ybuf = torch.full((n + 600, R), 3.0, device="cuda")
    y = ybuf[300:300 + n]
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    if bits == 16:
        w = torch.empty(E, R, C, dtype=dt, device="cuda").normal_(0, 0.05, generator=g)

        def call(off):
            pm.pm_grouped_gemm(w, x, y, off, order, 1, SCATTER)
    else:
        q = torch.randint(0, 256, (E, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = (torch.rand(E, R, C // bits, generator=g, device="cuda") * 0.02 + 0.001).half()
        z = torch.randint(0, 16, (E, R, C // bits), generator=g, device="cuda", dtype=torch.uint8)

        def call(off):
            pm.pm_grouped_gemm_w4(q, s, z, bits, x, y, off, order, 1, SCATTER)
    good = torch.linspace(0, n, E + 1).int().cuda()
    call(good)
    want = y.clone()
    assert torch.isfinite(want).all()
    for off in bad_offsets(E, n, n):
        call(off)
        assert torch.isfinite(y).all(), off.tolist()[:8]
        assert torch.all(ybuf[:300] == 3.0) and torch.all(ybuf[300 + n:] == 3.0), off.tolist()[:8]
    y.fill_(3.0)
    call(good)
    assert torch.equal(y, want)


# ---------------------------------------------------------------- most experts, far rows
@pytest.mark.parametrize("bits,ty,C", [(16, "bf16", 2056), (16, "bf16", 64), (128, "f32", 1280),
                                       (128, "bf16", 1280), (64, "f16", 128)])
@pytest.mark.parametrize("many", [False, True])
def test_grouped_most_experts(bits, ty, C, many):
    """4096 experts, nearly all of them empty, the first and last not."""
    E, R = 4096, 18
    report(f"grouped 4096 experts {bits} {ty} cols {C} many {many}")
    g = rc.gen(C)
    dt = rc.TYPES[ty]
    counts = np.zeros(E, np.int64)
    counts[[0, 1, 7, 8, 63, 64, 65, 511, 2047, 2048, 4094, 4095]] = [1, 2, 9, 3, 1, 17, 2, 1, 1, 20, 5, 1]
    if many:
        counts[[3, 4093]] = [40000, 30000]
    off, order = rc.groups(counts, 1)
    n = int(counts.sum())
    x = torch.randn(n, C, generator=g, device="cuda").to(dt)
    y = torch.full((n, R), 3.0, device="cuda")
    if bits == 16:
        w = torch.empty(E, R, C, dtype=dt, device="cuda").normal_(0, 0.05, generator=g)
        pm.pm_grouped_gemm(w, x, y, off, order, 1, SCATTER)

        def w64(e):
            return w[e].double()
    else:
        q = torch.randint(0, 256, (E, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = (torch.rand(E, R, C // bits, generator=g, device="cuda") * 0.02 + 0.001).half()
        pm.pm_grouped_gemm_w4(q, s, None, bits, x, y, off, order, 1, SCATTER)

        def w64(e):
            return rc.decode_w4(q[e], s[e], None, bits)
    rc.check_grouped(y, 3.0, rc.grouped_plain(w64, x, off, order, n, 1, False, True, False))


def test_rows_far_apart():
    """Router and combine on rows whose byte offsets pass 2^32."""
    report("router and combine beyond 32 bits")
    ld = 1 << 30
    buf = torch.empty(4 * ld + 64, dtype=torch.bfloat16, device="cuda")
    l = buf.as_strided((5, 64), (ld, 1))
    l.copy_(torch.randn(5, 64, generator=rc.gen(1), device="cuda"))
    ids = torch.empty(5, 3, dtype=torch.int32, device="cuda")
    w = torch.empty(5, 3, device="cuda")
    off = torch.empty(65, dtype=torch.int32, device="cuda")
    order = torch.empty(15, dtype=torch.int32, device="cuda")
    ws = torch.empty(pm.pm_route_workspace_bytes(5, 64, 3), dtype=torch.uint8, device="cuda")
    pm.pm_route_topk_device(l, 3, ids, w, off, order, ws)
    wi, _, woff, word = rc.route_plain(l, 3)
    assert np.array_equal(ids.cpu().numpy(), wi)
    assert np.array_equal(off.cpu().numpy(), woff) and np.array_equal(order.cpu().numpy(), word)
    z = buf.as_strided((4, 40), (ld, 1))
    yb = torch.empty(ld + 40, dtype=torch.bfloat16, device="cuda")
    y = yb.as_strided((2, 40), (ld, 1))
    pm.pm_combine_uses(z, torch.tensor([[1.0, 0.0], [0.0, 0.5]], device="cuda"), y)
    assert torch.equal(y[0], z[0]) and torch.equal(y[1], z[3] * 0.5)


@pytest.mark.parametrize("K", [63, 65, 130])
@pytest.mark.parametrize("H", [3, 40])
def test_combine_of_many_slots(K, H):
    """More slots than a wave has lanes, whole numbers: exact."""
    report(f"combine top-{K} of {H} columns")
    g = rc.gen(K)
    z = torch.randint(-9, 10, (5 * K, H), generator=g, device="cuda").half()
    w = torch.randint(-9, 10, (5, K), generator=g, device="cuda").float()
    y = torch.empty(5, H, device="cuda")
    pm.pm_combine_uses(z, w, y)
    assert torch.equal(y.double(), (w.double()[:, :, None] * z.double().reshape(5, K, H)).sum(1))


@pytest.mark.parametrize("T,E", [(3, 64), (40, 64), (2, 70), (300, 64)])
def test_route_takes_every_expert_of_64(T, E):
    """top-64: the list of the selected fills the wave."""
    report(f"route {T} x {E} top-64")
    l = torch.randn(T, E, generator=rc.gen(T), device="cuda").mul_(3).round_()
    l[0, 5] = -float("inf")
    ids = torch.empty(T, 64, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 64, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order = torch.full((T * 64,), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(pm.pm_route_workspace_bytes(T, E, 64), dtype=torch.uint8, device="cuda")
    pm.pm_route_topk_device(l, 64, ids, w, off, order, ws)
    wi, ww, woff, word = rc.route_plain(l, 64)
    assert np.array_equal(ids.cpu().numpy(), wi)
    # fp64 softmax rounded to fp32: half a step, and a little for the exponential
    assert np.all(np.abs(w.cpu().numpy() - ww) <= 1.01 * 2.0 ** -24 * ww + 2.0 ** -149)
    n = woff[-1]
    assert np.array_equal(off.cpu().numpy(), woff)
    assert np.array_equal(order.cpu().numpy()[:n], word) and np.all(order.cpu().numpy()[n:] == -7)
