"""The scored router and the 8-bit operators against plain fp64 forms, through
the C ABI: routing, encoder, products grouped by expert, and whole layers of
them, eager and captured."""
import numpy as np
import pytest
import torch

import bitplane_quantized_expert_amd as pm
import fp8_cases as fc
import routed_cases as rc

pytestmark = pytest.mark.gpu
GATHER, SCATTER, SWIGLU = pm.PM_GROUPED_GATHER, pm.PM_GROUPED_SCATTER, pm.PM_GROUPED_SWIGLU
SCORES = {"sigmoid": pm.PM_SCORE_SIGMOID, "softmax": pm.PM_SCORE_SOFTMAX}


def report(name):
    print(f"[gpu case] {name}", flush=True)


# ---------------------------------------------------------------- scored router
def run_scored(logits, bias, top_k, score="sigmoid", n_groups=1, top_groups=1, group_best=1,
               renorm=False, scale=1.0, stream=None):
    T, E = logits.shape
    rule = pm.pm_route_rule(SCORES[score], n_groups, top_groups, group_best,
                            pm.PM_ROUTE_RENORM if renorm else 0, scale)
    ids = torch.full((T, top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, top_k), -7.0, device="cuda")
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((T * top_k,), -7, dtype=torch.int32, device="cuda")
    ws = torch.randint(0, 256, (max(1, pm.pm_route_workspace_bytes(T, E, top_k)),),
                       dtype=torch.uint8, device="cuda")
    pm.pm_route_scored_device(rule, logits, bias, top_k, ids, w, off, order, ws, stream)
    return ids, w, off, order


def check_scored(logits, bias, top_k, what="", got=None, **rule):
    got = got or run_scored(logits, bias, top_k, **rule)
    ids, w, off, order = (t.cpu().numpy() for t in got)
    wi, ww, woff, word = fc.scored_plain(logits, bias, top_k, **rule)
    assert np.array_equal(ids, wi), (what, np.argwhere(ids != wi)[:4])
    # fp64 (a few hundred of its steps) rounded to fp32: half a step
    assert np.all(np.abs(w - ww) <= 1.01 * 2.0 ** -24 * np.abs(ww) + 2.0 ** -149), what
    assert np.array_equal(off, woff), what
    n = woff[-1]
    assert np.array_equal(order[:n], word), what
    assert np.all(order[n:] == -7), what


RULES = [dict(score="sigmoid"), dict(score="softmax"),
         dict(score="sigmoid", n_groups=8, top_groups=4, group_best=2, renorm=True, scale=2.5),
         dict(score="softmax", n_groups=4, top_groups=3, group_best=1, scale=16.0)]


@pytest.mark.parametrize("T,E,K", [(1, 8, 1), (1, 512, 10), (2, 8, 3), (5, 64, 8), (17, 200, 7),
                                   (33, 512, 10), (64, 256, 8), (16, 104, 4), (300, 1000, 10),
                                   (257, 4096, 64), (1030, 512, 10), (3000, 40, 2), (24, 512, 10),
                                   (48, 296, 5), (49, 296, 5), (4, 4096, 8), (13, 2056, 8),
                                   (700, 2048, 10), (9, 72, 64), (8, 1544, 3)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_scored_route_sizes(T, E, K, with_bias):
    report(f"scored route {T} x {E} top-{K} bias {with_bias}")
    g = rc.gen(T * 7 + E)
    l = torch.randn(T, E, generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda").mul_(0.1) if with_bias else None
    for rule in RULES:
        if K * rule.get("n_groups", 1) <= rule.get("top_groups", 1) * E:
            check_scored(l, bias, K, str(rule), **rule)


@pytest.mark.parametrize("n_groups,top_groups,best", [(1, 1, 2), (2, 1, 2), (3, 2, 1), (12, 5, 2),
                                                      (32, 9, 2), (48, 20, 1), (16, 16, 2),
                                                      (64, 30, 2), (64, 7, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_scored_route_groups(n_groups, top_groups, best, score):
    """Groups of 192 down to 3 experts, and of one."""
    for E in {192, n_groups}:
        K = min(6, top_groups * E // n_groups)
        report(f"scored route {E} experts, {top_groups} of {n_groups} groups {score}")
        g = rc.gen(n_groups * 31 + E)
        l = torch.randn(77, E, generator=g, device="cuda")
        bias = torch.randn(E, generator=g, device="cuda").mul_(0.05)
        for b in (None, bias):
            check_scored(l, b, K, score=score, n_groups=n_groups, top_groups=top_groups,
                         group_best=best, renorm=True)


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("grouped", [False, True])
def test_scored_route_ties_and_masks(ty, score, grouped):
    """Rows of a wider buffer; many equal logits (whole groups that count the
    same); experts masked with -inf or the type's lowest value; NaN; +inf;
    signed zeros; saturated scores; tokens with nothing."""
    report(f"scored route masks and ties {ty} {score} {grouped}")
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
    l[14, :] = 50.0                                # sigmoid: all 1.0
    l[14, 40:] = 60.0
    l[15, ::3] = -float("inf")
    l[16, 1:] = -float("inf")                      # one expert
    l[17, 12:] = -float("inf")                     # one group
    l[18, :] = -800.0                              # scores of 0 beside one of 1
    l[18, 3] = 0.0
    l[200:, :] = -float("inf")                     # a padded tail
    rule = dict(score=score, n_groups=8, top_groups=3, group_best=2) if grouped else \
        dict(score=score)
    bias = torch.randn(E, generator=g, device="cuda").mul_(4).round_().div_(16)
    masked = bias.clone()
    masked[5] = -float("inf")
    masked[24:36] = float("nan")                   # a group that no token takes
    masked[40] = float("inf")
    for b in (None, bias, masked, torch.zeros_like(bias)):
        for renorm in (False, True):
            check_scored(l, b, K, renorm=renorm, **rule)
    check_scored(l[:1], bias, K, **rule)
    check_scored(l[3:5], bias, K, **rule)


def test_scored_route_near_ties():
    """Ranks that differ by less than fp32 shows: logits and biases that fp32
    sums would round together, in both directions."""
    report("scored route near ties")
    T, E, K = 64, 256, 8
    g = rc.gen(12)
    # neighbouring fp32 numbers around a few values
    base = torch.tensor([0.3, 0.7, 1.1, -0.4], device="cuda")[torch.randint(
        0, 4, (T, E), generator=g, device="cuda")]
    l = (base.view(torch.int32) + torch.randint(-3, 4, (T, E), generator=g, device="cuda",
                                                dtype=torch.int32)).view(torch.float32)
    bias = torch.randint(-4, 5, (E,), generator=g, device="cuda").float().mul_(2.0 ** -26)
    for score in SCORES:
        for b in (None, bias, bias + 4.0):
            for groups in (dict(), dict(n_groups=16, top_groups=5, group_best=2),
                           dict(n_groups=32, top_groups=5, group_best=1)):
                check_scored(l, b, K, score=score, **groups)


def test_scored_route_large_biases():
    """Biases so large that fp32 sums, and the top halves of fp64 ones, hold
    little of the scores; and such of both signs, which cancel in the sums of
    a group's two best experts."""
    report("scored route large biases")
    g = rc.gen(21)
    for E, K in ((96, 6), (512, 10), (1000, 64), (4096, 10)):
        l = torch.randn(9, E, generator=g, device="cuda")
        for big in (2.0 ** 10, 2.0 ** 20, -2.0 ** 20):
            for score in SCORES:
                check_scored(l, torch.full((E,), big, device="cuda"), K, f"{E} {big}", score=score)
    for big in (1000.0, 60000.0):
        bias = torch.full((64, 4), -big, device="cuda")
        bias[:, 1] = big
        l = torch.randn(100, 256, generator=g, device="cuda")
        for top_groups in (3, 30):
            check_scored(l, bias.view(-1), 8, f"{big} {top_groups}", score="sigmoid",
                         n_groups=64, group_best=2, top_groups=top_groups)


def test_scored_route_adjacent_experts():
    """The largest logits side by side, in few lanes, or all in one group."""
    report("scored route adjacent experts")
    g = rc.gen(23)
    for E, K in ((64, 8), (128, 13), (512, 10), (512, 40), (1000, 10), (4096, 64)):
        l = torch.randn(21, E, generator=g, device="cuda")
        l[:7] = l[:7].sort(dim=1, descending=True).values
        l[7:14] = l[7:14].sort(dim=1).values
        l[14] = torch.arange(E, device="cuda").div(64, rounding_mode="floor")
        bias = torch.randn(E, generator=g, device="cuda").mul_(0.01)
        for score in SCORES:
            for b in (None, bias):
                check_scored(l, b, K, f"{E} {score}", score=score, renorm=True)
                if E % 8 == 0 and K <= E // 8:
                    check_scored(l, b, K, f"{E} {score} one group", score=score, n_groups=8,
                                 top_groups=1, group_best=2)


def test_scored_route_equal_rows():
    """Rows whose experts all count the same, as a padded token's do: the lowest
    ids.  And such rows with one better, one worse and one masked."""
    report("scored route equal rows")
    for E, K in ((8, 3), (72, 64), (100, 12), (512, 10), (520, 13), (4096, 64)):
        l = torch.zeros(12, E, device="cuda")
        l[1:5] = torch.tensor([-1.0, 3.5, 40.0, -90.0], device="cuda")[:, None]
        l[5, E // 2] = 1.0
        l[6, 1] = -1.0
        l[7, 0] = -float("inf")
        l[8, E // 3:] = -float("inf")
        l[9, :3] = 2.0 ** -40                      # (a score of just over 1/2)
        l[10, ::2] = 2.0 ** -40
        for score in SCORES:
            for bias in (None, torch.full((E,), 0.125, device="cuda")):
                check_scored(l, bias, K, f"{E} {score}", score=score, renorm=True)
                if E % 8 == 0 and K <= E // 2:
                    check_scored(l, bias, K, f"{E} {score} groups", score=score, n_groups=8,
                                 top_groups=4, group_best=2)


def test_scored_route_smallest_scores():
    """Sigmoids about the smallest normal fp32 number, a few steps of the logits'
    type apart, and softmax scores as small beside one large."""
    report("scored route smallest scores")
    g = rc.gen(22)
    at = torch.full((40, 128), -87.3365447, device="cuda")
    l = (at.view(torch.int32) + torch.randint(-400, 400, at.shape, generator=g, device="cuda",
                                              dtype=torch.int32)).view(torch.float32)
    check_scored(l, None, 8, score="sigmoid")
    check_scored(l * (1.0 + torch.rand(40, 1, generator=g, device="cuda") / 8), None, 12,
                 score="sigmoid")
    l = torch.cat([torch.zeros(40, 2, device="cuda"), l - 5 * torch.rand(
        40, 128, generator=g, device="cuda")], dim=1)
    check_scored(l, None, 8, "softmax", score="softmax", renorm=True)


def test_scored_route_no_experts_but_the_biased():
    """A bias alone decides between scores of 0; their weights are 0, renormalised
    or not."""
    report("scored route zero scores")
    l = torch.full((5, 40), -3000.0, device="cuda")
    bias = torch.arange(40, device="cuda").float()
    for renorm in (False, True):
        check_scored(l, bias, 4, score="sigmoid", renorm=renorm)


def test_scored_route_many_tokens():
    """More tokens than the blocks of the sorting hold, against the same rule in
    torch's fp64."""
    report("scored route 300 000 tokens")
    T, E = 300_000, 16
    l = torch.randn(T, E, generator=rc.gen(2), device="cuda")
    l[1234:2345] = -float("inf")
    ids, w, off, order = run_scored(l, None, 2, n_groups=4, top_groups=2, group_best=2,
                                    renorm=True)
    s = torch.sigmoid(l.double())
    best = s.reshape(T, 4, 4).topk(2, dim=2).values.sum(2).topk(2, dim=1).indices
    keep = (best[:, :, None] == torch.arange(4, device="cuda")).any(1).repeat_interleave(4, 1)
    top = torch.where(keep, s, -1.0).topk(2, dim=1)
    some = torch.ones(T, dtype=torch.bool, device="cuda")
    some[1234:2345] = False
    assert torch.equal(ids[some].long(), top.indices[some])
    assert bool((ids[~some] == -1).all()) and not w[~some].any()
    want = top.values[some] / top.values[some].sum(1, keepdim=True)
    assert bool(((w[some].double() - want).abs() <= 1.01 * 2.0 ** -24 * want).all())
    flat = ids.reshape(-1)
    n = int(off[-1])
    assert n == int((flat >= 0).sum())
    by = torch.sort(torch.where(flat >= 0, flat, E), stable=True).indices[:n]
    assert torch.equal(order[:n].long(), by)
    assert torch.equal(off[1:].long(), torch.bincount(flat[flat >= 0], minlength=E).cumsum(0))


def test_scored_route_without_sorting_and_without_tokens():
    report("scored route: no order, no tokens")
    l = torch.randn(9, 40, generator=rc.gen(1), device="cuda")
    ids = torch.empty(9, 5, dtype=torch.int32, device="cuda")
    w = torch.empty(9, 5, device="cuda")
    pm.pm_route_scored_device(pm.pm_route_rule(), l, None, 5, ids, w)
    assert np.array_equal(ids.cpu().numpy(), fc.scored_plain(l, None, 5, "sigmoid")[0])
    off = torch.full((41,), 9, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 40, device="cuda")
    pm.pm_route_scored_device(pm.pm_route_rule(), e, None, 5, ids, w, off,
                              torch.empty(0, dtype=torch.int32, device="cuda"))
    assert not off.any()


# ---------------------------------------------------------------- encoder
def check_encode(x, block_rows, ldq=None, what=""):
    shape = x.shape if x.dim() == 3 else (1, *x.shape)
    n, r, c = shape
    buf = torch.full((n * r, (ldq or c) + 16), 0x55, dtype=torch.uint8, device="cuda")
    q = buf[:, :c].unflatten(0, (n, r)) if x.dim() == 3 else buf[:, :c]
    scales = torch.full((n, -(-r // block_rows), -(-c // 128)), -7.0, device="cuda")
    pm.pm_encode_fp8_device(x, q, scales, block_rows)
    wq, wsc = fc.encode_plain(x.reshape(shape) if x.dim() == 2 else x, block_rows)
    assert np.array_equal(scales.cpu().numpy(), wsc), what
    got = q.contiguous().view(fc.F8).double().cpu().numpy().reshape(shape)
    assert np.array_equal(got, wq, equal_nan=True), (
        what, np.argwhere((got != wq) & ~(np.isnan(got) & np.isnan(wq)))[:4])
    assert bool((buf[:, c:] == 0x55).all()), what


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (8, 4096), (333, 1008),
                                       (17, 112), (2, 8208), (1000, 256), (129, 400)])
def test_encode_rows(ty, rows, cols):
    report(f"encode rows {rows} x {cols} {ty}")
    g = rc.gen(rows + cols)
    buf = torch.randn(rows, cols + 32, generator=g, device="cuda").to(rc.TYPES[ty])
    buf[rows // 2, :cols // 2] *= 64.0
    buf[-1, :] = 0.0
    check_encode(buf[:, 16:16 + cols], 1)
    check_encode(buf[:, :cols].contiguous(), 1)


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 16), (1, 128, 128), (3, 127, 144), (2, 256, 1008),
                                         (5, 129, 256), (1, 1426, 1008), (40, 16, 112)])
def test_encode_squares(ty, n, rows, cols):
    report(f"encode squares {n} x {rows} x {cols} {ty}")
    g = rc.gen(rows + cols)
    x = torch.randn(n, rows, cols + 16, generator=g, device="cuda").mul_(0.02).to(rc.TYPES[ty])
    check_encode(x[:, :, :cols], 128)
    if n == 1:
        check_encode(x[0, :, :cols], 128)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
def test_encode_ends_of_the_types(ty, block_rows):
    """Infinities and NaN, blocks of zeros, of the smallest and the largest
    values, quotients on the borders of two codes, and below the smallest."""
    report(f"encode ends {ty} {block_rows}")
    dt = rc.TYPES[ty]
    fi = torch.finfo(dt)
    g = rc.gen(9)
    x = torch.randn(260, 512, generator=g, device="cuda")
    x[0, 5] = float("inf")
    x[0, 200] = -float("inf")
    x[1, 130] = float("nan")
    x[2, :128] = float("nan")                      # nothing finite in a block
    x[3] = 0.0
    x[4] = -0.0
    x = x.to(dt)
    x[5] = fi.max
    x[6, ::2] = fi.min
    x[7] = fi.smallest_normal
    x[8, :256] = fi.smallest_normal * fi.eps       # the smallest subnormal number
    x[8, 256:] = -fi.smallest_normal * 3 * fi.eps
    # every midpoint of two codes, where the largest is 448 times a power of two
    mids = torch.arange(1, 512, dtype=torch.float32)
    x[9] = torch.cat([torch.tensor([448.0]), mids / 2.0]).to(dt).cuda().clamp(max=448)
    x[10] = torch.cat([torch.tensor([448.0]), mids * 2.0 ** -11]).to(dt).cuda()
    x[11] = torch.cat([torch.tensor([448.0]), -mids / 16.0]).to(dt).cuda()
    # quotients by a largest value that is a multiple of 7: ties in exact numbers
    x[12] = torch.cat([torch.tensor([3.5]), mids * 2.0 ** -8]).to(dt).cuda().clamp(max=3.5)
    check_encode(x, block_rows)


def test_encode_far_rows():
    """Rows of x and q beyond 2^32 bytes."""
    report("encode far rows")
    r, c, ld = 70_000, 256, 32_768
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("too little memory")
    x = torch.zeros(r, ld, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(r, ld * 2 - 16, dtype=torch.uint8, device="cuda")
    rows = [0, 1, 35_000, 65_535, 65_536, 69_999]
    v = torch.randn(len(rows), c, generator=rc.gen(4), device="cuda").bfloat16()
    x[rows, :c] = v
    s = torch.empty(r, 2, device="cuda")
    pm.pm_encode_fp8_device(x[:, :c], q[:, :c], s)
    wq, wsc = fc.encode_plain(v[:, None], 1)
    assert np.array_equal(s[rows].cpu().numpy(), wsc[:, 0])
    assert np.array_equal(q[rows, :c].contiguous().view(fc.F8).double().cpu().numpy(), wq[:, 0])
    q[rows, :c] = 0
    assert not q[::997].any()


# ---------------------------------------------------------------- products
def run_grouped8(counts, R, C, y_ty, top_k, flags, seed=0, n_rows=None, order=True, pad=0, wide=0,
                 make_x=fc.make_x, make_w=fc.make_weights):
    """One call against the plain form.  pad: extra elements per row of x (times
    16) and y; wide: columns of y kept from the right of the output."""
    E = len(counts)
    off, ordr = rc.groups(counts, seed, n_rows)
    n = ordr.numel()
    if not order:
        ordr = None
    nx = (n + top_k - 1) // top_k if flags & GATHER else n
    out = R // 2 if flags & SWIGLU else R
    W, ws = make_w(E, R, C, seed + 1)
    x, xs = make_x(nx, C, seed + 2, C + 16 * pad)
    ybuf = torch.full((n, out + pad + wide), -7.0, dtype=rc.TYPES[y_ty], device="cuda")
    y = ybuf[:, :out]
    pm.pm_grouped_gemm_fp8(W, ws, x, xs, y, off, ordr, top_k, flags)
    want = fc.grouped_plain(W, ws, x, xs, off, ordr, n, top_k, flags & GATHER, flags & SCATTER,
                            flags & SWIGLU, y_ty == "bf16")
    rc.check_grouped(y, -7.0, want, f"{counts[:8]} {R}x{C} {y_ty} flags {flags}")
    assert bool((ybuf[:, out:] == -7.0).all())
    # twice gives the same bits
    again = torch.full_like(ybuf, -7.0)
    pm.pm_grouped_gemm_fp8(W, ws, x, xs, again[:, :out], off, ordr, top_k, flags)
    assert torch.equal(ybuf, again)


FLAGS = [0, GATHER, SCATTER, SWIGLU, GATHER | SWIGLU, GATHER | SCATTER | SWIGLU]
PATTERNS = {"one": [1], "few": [1, 0, 2, 5, 0, 0, 3], "sixteens": [16, 17, 15, 32, 33],
            "uneven": [0, 130, 1, 260, 40, 0, 7], "many": [300, 513, 129]}


@pytest.mark.parametrize("y_ty", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pattern", list(PATTERNS))
@pytest.mark.parametrize("R,C", [(128, 256), (142, 144), (1426, 1008), (20, 16), (258, 400)])
def test_grouped8(y_ty, pattern, R, C):
    for flags in FLAGS:
        report(f"fp8 {pattern} {R} x {C} {y_ty} flags {flags}")
        run_grouped8(PATTERNS[pattern], R, C, y_ty, 3, flags, seed=R + flags, pad=flags % 3,
                     wide=flags & 1)


@pytest.mark.parametrize("C", [128, 512, 1024, 1152, 2048, 2304, 4096, 4112, 5120, 8192])
@pytest.mark.parametrize("y_ty", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[3, 1, 2], [40, 9], [1, 300]])
def test_grouped8_inputs(C, y_ty, counts):
    """Input sizes of every split, small and large groups."""
    report(f"fp8 {counts} 96 x {C} {y_ty}")
    run_grouped8(counts, 96, C, y_ty, 1, GATHER | SWIGLU, seed=C)
    run_grouped8(counts, 96, C, y_ty, 1, SCATTER, seed=C)


@pytest.mark.parametrize("R,C", [(4096, 144), (4120, 400), (3000, 16), (4096, 2048)])
def test_grouped8_large_tiles(R, C):
    """Groups of many rows and more tiles of 256 x 256 than twice the compute
    units, the last round not full; weight rows whose gate and up begin inside
    a block of 128."""
    for counts in ([4500, 4200], [2300, 257, 0, 6200, 255]):
        for flags in (0, GATHER | SWIGLU, SCATTER):
            report(f"fp8 large tiles {R} x {C} {counts} flags {flags}")
            run_grouped8(counts, R, C, "bf16", 2, flags, seed=R + C, pad=flags & 1)


def test_grouped8_many_experts():
    """512 and 4096 experts, most without rows; more rows than offsets end at."""
    g = np.random.default_rng(3)
    for E, n in ((512, 80), (4096, 300), (512, 3000)):
        report(f"fp8 {E} experts {n} rows")
        counts = np.bincount(g.integers(0, E, n), minlength=E).tolist()
        run_grouped8(counts, 64, 128, "bf16", 10, GATHER | SWIGLU, n_rows=n + 17)
        run_grouped8(counts, 48, 256, "f32", 10, SCATTER, n_rows=n + 5)


@pytest.mark.parametrize("y_ty", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[3, 1, 2], [700, 300], [140, 1, 90]])
def test_grouped8_exact(y_ty, counts):
    """Products of small whole numbers: every partial sum is exact, on every
    path (products of at most 64 keep all bits beside each other), so results
    are equal and not only near.  Scales are powers of two."""
    report(f"fp8 exact {counts} {y_ty}")
    for C in (144, 1024, 4096):
        off, ordr = rc.groups(counts, 5)
        n, E, R = ordr.numel(), len(counts), 160
        g = rc.gen(C)

        def ints(*shape):
            return torch.randint(-8, 9, shape, generator=g, device="cuda").float().to(fc.F8)

        W, x = ints(E, R, C), ints(n, C)
        ws = torch.exp2(torch.randint(-3, 1, (E, 2, -(-C // 128)), generator=g, device="cuda")
                        .float())
        xs = torch.exp2(torch.randint(-2, 2, (n, -(-C // 128)), generator=g, device="cuda").float())
        y = torch.full((n, R), -7.0, dtype=rc.TYPES[y_ty], device="cuda")
        pm.pm_grouped_gemm_fp8(W, ws, x, xs, y, off, ordr, 1, SCATTER)
        want = fc.grouped_plain(W, ws, x, xs, off, ordr, n, 1, False, True, False, False)
        for at, p, _ in want:
            assert torch.equal(y[at], p.to(y.dtype))


def test_grouped8_masked_nan_and_infinite_weights():
    """NaN codes and scales in rows of x that no use maps to, in experts without
    rows and past the last input reach no output; NaN in a row of x reaches that
    row alone."""
    report("fp8 NaN")
    for counts in ([2, 0, 3], [200, 0, 80]):
        C, R = 144, 80
        off, ordr = rc.groups(counts, 6, sum(counts) + 9)
        n = ordr.numel()
        W, ws = fc.make_weights(3, R, C, 1)
        W.view(torch.uint8)[1] = 0x7F
        ws[1] = float("nan")
        x, xs = fc.make_x(n, C, 2, C + 32)
        x.view(torch.uint8)
        buf = x.untyped_storage()
        full = torch.empty(0, dtype=torch.uint8, device="cuda").set_(buf).reshape(n, C + 32)
        full[:, C:] = 0x7F
        full[sum(counts):] = 0x7F
        xs[sum(counts):] = float("nan")
        for y_ty in ("f32", "bf16"):
            y = torch.full((n, R), -7.0, dtype=rc.TYPES[y_ty], device="cuda")
            pm.pm_grouped_gemm_fp8(W, ws, x, xs, y, off, None, 1, 0)
            ok = x.clone()
            ok.view(torch.uint8)[sum(counts):] = 0
            sc = torch.where(xs.isnan(), torch.ones_like(xs), xs)
            want = fc.grouped_plain(W, ws, ok, sc, off, None, n, 1, False, False, False,
                                    y_ty == "bf16")
            rc.check_grouped(y, -7.0, want)
            z = x.clone()
            z.view(torch.uint8)[1, 17] = 0xFF
            y2 = torch.full_like(y, -7.0)
            pm.pm_grouped_gemm_fp8(W, ws, z, xs, y2, off, None, 1, 0)
            assert bool(y2[1].isnan().all())
            rest = [i for i in range(n) if i != 1]
            assert torch.equal(y2[rest], y[rest])


def test_grouped8_bad_offsets_and_order():
    """Offsets that decrease or pass the rows, entries of the order outside the
    rows: nothing outside y is written, and rows of good groups are right."""
    report("fp8 bad offsets")
    E, R, C, n = 6, 96, 256, 200
    W, ws = fc.make_weights(E, R, C, 1)
    x, xs = fc.make_x(n, C, 2)
    big = torch.full((n + 64, R), -7.0, dtype=torch.bfloat16, device="cuda")
    for off in ([0, 40, 20, 200, 100, 150, 300], [-5, 10, 20, 30, 40, 50, 60],
                [0, 2 ** 31 - 1, 0, 5, -2 ** 31, 7, 9], [0, 300, 400, 500, 600, 700, 800]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        pm.pm_grouped_gemm_fp8(W, ws, x, xs, big[32:32 + n], o, None, 1, 0)
        torch.cuda.synchronize()
        assert bool((big[:32] == -7.0).all()) and bool((big[32 + n:] == -7.0).all())
    order = torch.arange(n, dtype=torch.int32, device="cuda")
    order[5], order[77], order[150] = -1, n, 2 ** 31 - 1
    for counts in ([10, 20, 30, 40, 50, 50], [3, 0, 1, 0, 2, 0]):
        off, _ = rc.groups(counts, 0)
        for flags in (GATHER, SCATTER, GATHER | SCATTER):
            y = torch.full((n, R), -7.0, dtype=torch.float32, device="cuda")
            pm.pm_grouped_gemm_fp8(W, ws, x, xs, y, off, order, 1, flags)
            want = fc.grouped_plain(W, ws, x, xs, off, order, n, 1, flags & GATHER,
                                    flags & SCATTER, False, False)
            rc.check_grouped(y, -7.0, want)


def test_grouped8_no_inputs_and_no_rows():
    report("fp8 empty")
    W = torch.empty(2, 32, 0, dtype=torch.uint8, device="cuda")
    s0 = torch.empty(0, device="cuda")
    off, ordr = rc.groups([3, 2], 0)
    y = torch.full((5, 32), -7.0, device="cuda")
    pm.pm_grouped_gemm_fp8(W, s0, torch.empty(5, 0, dtype=torch.uint8, device="cuda"), s0, y, off,
                           ordr, 1, 0)
    assert not y.any()
    W, ws = fc.make_weights(2, 32, 128, 0)
    x, xs = fc.make_x(5, 128, 1)
    off0 = torch.zeros(3, dtype=torch.int32, device="cuda")
    y.fill_(-7.0)
    pm.pm_grouped_gemm_fp8(W, ws, x, xs, y, off0, ordr, 1, 0)
    assert bool((y == -7.0).all())


def test_grouped8_far_rows():
    """Rows of x and y beyond 2^32 bytes."""
    report("fp8 far rows")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("too little memory")
    n, C, R, ld = 70_000, 128, 64, 65_536
    xb = torch.zeros(n, ld, dtype=torch.uint8, device="cuda")
    x, xs = fc.make_x(n, C, 2)
    xb[:, :C] = x.view(torch.uint8)
    W, ws = fc.make_weights(2, R, C, 1)
    off, ordr = rc.groups([40_000, 30_000], 3)
    yb = torch.zeros(n, ld // 2, dtype=torch.bfloat16, device="cuda")
    want = torch.full((n, R), 0.0, dtype=torch.bfloat16, device="cuda")
    for flags in (GATHER | SCATTER, 0):
        pm.pm_grouped_gemm_fp8(W, ws, xb[:, :C], xs, yb[:, :R], off, ordr, 1, flags)
        want = fc.grouped_plain(W, ws, x, xs, off, ordr, n, 1, flags & GATHER, flags & SCATTER,
                                False, True)
        rc.check_grouped(yb[:, :R], -7.0, want)
    del xb, yb


# ---------------------------------------------------------------- layers
def layer(rule, bias, logits, x, W1, s1, W2, s2, top_k, bufs, stream):
    """Scored routing, encoder, gate and up, encoder, down, combine."""
    ids, w, off, order, ws, xq, xs, h, hq, hs, z, y = bufs
    pm.pm_route_scored_device(rule, logits, bias, top_k, ids, w, off, order, ws, stream)
    pm.pm_encode_fp8_device(x, xq, xs, 1, stream)
    pm.pm_grouped_gemm_fp8(W1, s1, xq, xs, h, off, order, top_k, GATHER | SWIGLU, stream)
    pm.pm_encode_fp8_device(h, hq, hs, 1, stream)
    pm.pm_grouped_gemm_fp8(W2, s2, hq, hs, z, off, order, top_k, SCATTER, stream)
    pm.pm_combine_uses(z, w, y, stream)


def layer_buffers(T, E, K, hidden, inter):
    d = "cuda"
    u = T * K
    return (torch.empty(T, K, dtype=torch.int32, device=d), torch.empty(T, K, device=d),
            torch.empty(E + 1, dtype=torch.int32, device=d),
            torch.empty(u, dtype=torch.int32, device=d),
            torch.empty(pm.pm_route_workspace_bytes(T, E, K), dtype=torch.uint8, device=d),
            torch.empty(T, hidden, dtype=fc.F8, device=d),
            torch.empty(T, -(-hidden // 128), device=d),
            torch.full((u, inter), float("nan"), dtype=torch.bfloat16, device=d),
            torch.empty(u, inter, dtype=fc.F8, device=d), torch.empty(u, -(-inter // 128), device=d),
            torch.full((u, hidden), float("nan"), dtype=torch.bfloat16, device=d),
            torch.empty(T, hidden, dtype=torch.bfloat16, device=d))


def check_layer(rule_kw, bias, logits, x, W1, s1, W2, s2, K, bufs):
    """Every step against the plain form of that step on the step's own inputs."""
    ids, w, off, order, ws, xq, xs, h, hq, hs, z, y = bufs
    check_scored(logits, bias, K, got=(ids, w, off, torch.where(
        torch.arange(order.numel(), device="cuda") < off[-1], order, -7)), **rule_kw)
    qx, sx = fc.encode_plain(x[None], 1)
    assert np.array_equal(xs.cpu().numpy(), sx[0])
    assert np.array_equal(xq.double().cpu().numpy(), qx[0])
    n, used = order.numel(), int(off[-1])
    want = fc.grouped_plain(W1, s1, xq, xs, off, order, n, K, True, False, True, True)
    rc.check_grouped(h[:used], 0.0, want)
    qh, sh = fc.encode_plain(h[None, :used], 1)
    assert np.array_equal(hs[:used].cpu().numpy(), sh[0])
    assert np.array_equal(hq[:used].double().cpu().numpy(), qh[0])
    one = torch.ones_like(hs[:1])
    hs2 = torch.cat([hs[:used], one.expand(n - used, -1)])
    want = fc.grouped_plain(W2, s2, hq, hs2, off, order, n, K, False, True, False, True)
    for at, p, tol in want:
        lim = tol + 2.0 ** -8 * (p.abs() + tol) + 2.0 ** -130
        assert bool(((z[at].double() - p).abs() <= lim).all())
    zc = torch.where((ids.reshape(-1) >= 0)[:, None], z.double(), 0.0).reshape(*ids.shape, -1)
    yy = (zc * w.double()[:, :, None]).sum(1)
    mag = (zc.abs() * w.double()[:, :, None].abs()).sum(1)
    lim = (K + 1) * 2.0 ** -23 * mag + 2.0 ** -8 * yy.abs() + 2.0 ** -130
    assert bool(((y.double() - yy).abs() <= lim).all())


@pytest.mark.parametrize("T", [1, 6, 40, 300])
def test_layer_of_8_bit_experts(T):
    """A layer as it is used, on a stream of its own, with a padded token; then
    captured once and replayed for other tokens, with eager work between."""
    report(f"fp8 layer of {T} tokens")
    E, K, hidden, inter = 32, 4, 272, 144
    kw = dict(score="sigmoid", n_groups=4, top_groups=2, group_best=2, renorm=True, scale=2.5)
    rule = pm.pm_route_rule(SCORES["sigmoid"], 4, 2, 2, pm.PM_ROUTE_RENORM, 2.5)
    g = rc.gen(T)
    bias = torch.randn(E, generator=g, device="cuda").mul_(0.1)
    W1, s1 = fc.make_weights(E, 2 * inter, hidden, 1)
    W2, s2 = fc.make_weights(E, hidden, inter, 2)
    bufs = layer_buffers(T, E, K, hidden, inter)
    logits = torch.empty(T, E, device="cuda")
    x = torch.empty(T, hidden, dtype=torch.bfloat16, device="cuda")

    def fresh(seed):
        g = rc.gen(seed)
        logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
        x.copy_(torch.randn(T, hidden, generator=g, device="cuda").bfloat16())
        if T > 5:
            logits[T // 2] = -float("inf")

    side = torch.cuda.Stream()
    fresh(1)
    torch.cuda.synchronize()
    layer(rule, bias, logits, x, W1, s1, W2, s2, K, bufs, side)
    side.synchronize()
    check_layer(kw, bias, logits, x, W1, s1, W2, s2, K, bufs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            layer(rule, bias, logits, x, W1, s1, W2, s2, K, bufs, side)
    for seed in (2, 3, 4):
        fresh(seed)
        for b in bufs[:4]:
            b.fill_(-3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_layer(kw, bias, logits, x, W1, s1, W2, s2, K, bufs)
        eager = layer_buffers(T, E, K, hidden, inter)
        layer(rule, bias, logits, x, W1, s1, W2, s2, K, eager, None)
        torch.cuda.synchronize()
        assert torch.equal(eager[-1], bufs[-1])


def test_two_streams_at_once():
    """Two calls of each operator at once, on two streams, with buffers of their
    own."""
    report("fp8 two streams")
    T, E, K, hidden, inter = 64, 32, 4, 256, 128
    rule = pm.pm_route_rule(SCORES["softmax"], 4, 2, 1, 0, 1.0)
    W1, s1 = fc.make_weights(E, 2 * inter, hidden, 1)
    W2, s2 = fc.make_weights(E, hidden, inter, 2)
    sets = []
    for i in range(2):
        g = rc.gen(50 + i)
        sets.append((torch.randn(T, E, generator=g, device="cuda"),
                     torch.randn(T, hidden, generator=g, device="cuda").bfloat16(),
                     layer_buffers(T, E, K, hidden, inter), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for logits, x, bufs, st in sets:
            layer(rule, None, logits, x, W1, s1, W2, s2, K, bufs, st)
    torch.cuda.synchronize()
    for logits, x, bufs, st in sets:
        check_layer(dict(score="softmax", n_groups=4, top_groups=2, group_best=1), None, logits, x,
                    W1, s1, W2, s2, K, bufs)


def test_encoded_weights_serve():
    """Weights through the encoder and the product against the product of the
    weights themselves: e4m3 keeps each value to half a step of 2^-4 of it, or
    of its block's smallest normal code."""
    report("fp8 encoded weights")
    E, R, C, n = 3, 200, 400, 30
    g = rc.gen(8)
    w = torch.randn(E, R, C, generator=g, device="cuda").mul_(0.02)
    W = torch.empty(E, R, C, dtype=fc.F8, device="cuda")
    ws = torch.empty(E, 2, 4, device="cuda")
    pm.pm_encode_fp8_device(w, W, ws, 128)
    dec = fc.decode(W, ws, 128)
    lim = w.double().abs() * 2.0 ** -4 * (1 + 2.0 ** -20) + \
        fc.decode(torch.ones_like(w), ws, 128) * 2.0 ** -10
    assert bool(((dec - w.double()).abs() <= lim).all())
    x, xs = fc.make_x(n, C, 3)
    off, ordr = rc.groups([10, 12, 8], 1)
    y = torch.full((n, R), -7.0, device="cuda")
    pm.pm_grouped_gemm_fp8(W, ws, x, xs, y, off, ordr, 1, SCATTER)
    rc.check_grouped(y, -7.0, fc.grouped_plain(W, ws, x, xs, off, ordr, n, 1, False, True, False,
                                               False))


def test_binding_refusals():
    W, ws = fc.make_weights(2, 32, 128, 0)
    x, xs = fc.make_x(4, 128, 1)
    off, ordr = rc.groups([2, 2], 0)
    y = torch.empty(4, 32, device="cuda")
    call = pm.pm_grouped_gemm_fp8
    for bad in ((W[:, ::2], ws, x, xs, y, off), (W, ws[:1], x, xs, y, off),
                (W, ws, x, xs[:3], y, off), (W.float(), ws, x, xs, y, off),
                (W, ws, x.float(), xs, y, off), (W, ws, x[:, :64], xs, y, off),
                (W, ws, x, xs, y[:, :31], off), (W, ws, x, xs, y.double(), off),
                (W, ws, x, xs, y[:3], off, ordr),
                (W, ws, x, xs, y, off[:2]), (W, ws.half(), x, xs, y, off),
                (W, ws, x, xs.double(), y, off), (W, ws.cpu(), x, xs, y, off),
                (W, ws, x, xs.t(), y, off.cpu())):
        with pytest.raises(ValueError):
            call(*bad)
    q, s = torch.empty(4, 128, dtype=fc.F8, device="cuda"), torch.empty(4, 1, device="cuda")
    v = torch.randn(4, 128, device="cuda")
    for bad in ((v, q[:3], s), (v, q, s[:3]), (v.double(), q, s), (v, q.float(), s), (v[0], q[0], s),
                (v.t(), q.t(), s), (v.cpu(), q, s), (v, q, s.half())):
        with pytest.raises(ValueError):
            pm.pm_encode_fp8_device(*bad)
    with pytest.raises(pm.PMError, match="1 or 128"):
        pm.pm_encode_fp8_device(v, q, s, 4)
    l = torch.randn(4, 16, device="cuda")
    ids, w = torch.empty(4, 2, dtype=torch.int32, device="cuda"), torch.empty(4, 2, device="cuda")
    b = torch.zeros(16, device="cuda")
    for bad in (b[:15], b.half(), b.cpu(), torch.zeros(32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            pm.pm_route_scored_device(pm.pm_route_rule(), l, bad, 2, ids, w)
    with pytest.raises(pm.PMError, match="group_best"):
        pm.pm_route_scored_device(pm.pm_route_rule(group_best=3), l, b, 2, ids, w)
