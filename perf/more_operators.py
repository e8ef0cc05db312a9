"""Routed experts in 8-bit floating point as measured workloads.

A layer whose experts are kept in 8-bit floating point (e4m3, one scale for
each block of 128 inputs) runs three operators beside the combine: a router
that scores every expert and picks within the best groups of experts, the
encoder that gives activations (and, offline, weights) their 8-bit form, and
the products grouped by expert of such activations and weights.  Every case is
one call of one of them.

`run` computes a case in elementary torch operations in fp32, the router's
scores in fp64 (own False), or calls the library's entry point (own True);
`exact` computes it in fp64.
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_F8 = torch.float8_e4m3fn
BLOCK = 128


# ---------------------------------------------------------------- cases
def listed():
    """The shapes are those of the repository's workloads (512 experts, hidden
    4096, intermediate 1024, top-10; hidden 256, intermediate 128), of common
    smaller layers, and odd ones."""
    return [
        # one decode token's routing: sigmoid scores, a bias that balances the
        # load, the best 4 of 8 groups.  Latency only
        _route("score-decode", 1, 512, 10, "sigmoid", True, 8, 4, 2, True, 2.5, "f32"),
        # an odd batch over few experts, softmax over all of them, bf16 logits
        # with many equal ones
        _route("score-ragged", 1003, 60, 4, "softmax", False, 1, 1, 1, False, 1.0, "bf16"),
        # a prefill's routing
        _route("score-prefill", 16384, 512, 10, "sigmoid", True, 8, 4, 2, True, 2.5, "f32"),

        # a decode batch's activations, one scale per row and 128 inputs
        _encode("encode-decode", 1, 8, 4096, 1, "bf16"),
        # a prefill's activations
        _encode("encode-prefill", 1, 16384, 4096, 1, "bf16"),
        # the weights of a layer of odd sizes, one scale per 128 x 128
        _encode("encode-weights", 40, 1426, 1008, BLOCK, "f32"),

        # gate and up of one token in the small expert: the smallest product
        _gemm("fp8-tiny", 1, 16, 2, 256, 128, "gateup", "f32"),
        # eight decode tokens over 512 experts: about one row per expert
        _gemm("fp8-decode", 8, 512, 10, 4096, 1024, "gateup", "bf16"),
        # a decode batch's way down: every weight once
        _gemm("fp8-batch", 64, 512, 10, 4096, 1024, "down", "f32"),
        # sizes that fit no tile, a batch of a few rows per expert and more
        _gemm("fp8-odd", 333, 40, 6, 1008, 713, "gateup", "f16"),
        # prefill over 512 experts: about 80 rows per expert
        _gemm("fp8-prefill", 4096, 512, 10, 4096, 1024, "down", "bf16"),
        # prefill over few experts: thousands of rows per expert, uneven
        _gemm("fp8-large", 8192, 32, 8, 4096, 1024, "gateup", "bf16", skew=0.5),
    ]


def _route(name, tokens, experts, top_k, score, bias, n_groups, top_groups, group_best, renorm,
           scale, logits):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k,
            "score": score, "bias": bias, "n_groups": n_groups, "top_groups": top_groups,
            "group_best": group_best, "renorm": renorm, "scale": scale, "logits": logits}


def _encode(name, matrices, rows, cols, block_rows, x):
    return {"name": name, "op": "encode", "matrices": matrices, "rows": rows, "cols": cols,
            "block_rows": block_rows, "x": x}


def _gemm(name, tokens, experts, top_k, hidden, inter, stage, y, skew=0.0):
    return {"name": name, "op": "gemm", "tokens": tokens, "experts": experts, "top_k": top_k,
            "hidden": hidden, "inter": inter, "stage": stage, "y": y, "skew": skew}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_route(rng):
    n_groups = rng.choice([1, 1, 2, 4, 8])
    size = _log_int(rng, 4, 512 // n_groups)
    top_groups = rng.randint(1, n_groups)
    return _route(None, _log_int(rng, 1, 16384), n_groups * size,
                  rng.randint(1, min(10, top_groups * size)), rng.choice(["sigmoid", "softmax"]),
                  rng.random() < 0.5, n_groups, top_groups, rng.randint(1, 2),
                  rng.random() < 0.5, rng.choice([1.0, 2.5]), rng.choice(["f32", "bf16", "f16"]))


def _draw_encode(rng):
    x = rng.choice(["f32", "bf16", "f16"])
    # rows of whole 16-byte pieces of codes
    cols = 16 * _log_int(rng, 8, 512)
    if rng.random() < 0.5:
        return _encode(None, 1, _log_int(rng, 1, 16384), cols, 1, x)
    return _encode(None, _log_int(rng, 1, 64), _log_int(rng, 64, 4096), cols, BLOCK, x)


def _draw_gemm(rng):
    experts = _log_int(rng, 4, 512)
    stage = rng.choice(["gateup", "down"])
    # rows of whole 16-byte pieces of codes; the output side is free
    hidden = 16 * _log_int(rng, 8, 256)
    inter = 16 * _log_int(rng, 4, 128)
    if stage == "gateup":
        inter = max(64, inter - rng.randint(0, 15))
    else:
        hidden = max(64, hidden - rng.randint(0, 15))
    return _gemm(None, _log_int(rng, 1, 8192), experts, rng.randint(1, min(10, experts)), hidden,
                 inter, stage, rng.choice(["f32", "bf16", "f16"]), rng.choice([0.0, 0.5]))


def draw(rng):
    make = rng.choice([_draw_route, _draw_encode, _draw_gemm, _draw_gemm])
    case = make(rng)
    most = [work(c) for c in listed() if c["op"] == case["op"]]
    while any(work(case)[m] > max(w[m] for w in most) for m in ("bytes", "flops")):
        case = make(rng)
    return case


# ---------------------------------------------------------------- sizes
def _dims(case):
    """Rows and columns of one expert's weight matrix and the output width."""
    if case["stage"] == "gateup":
        return 2 * case["inter"], case["hidden"], case["inter"]
    return case["hidden"], case["inter"], case["hidden"]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _active(case):
    """Experts that get a row, as expected of independent even routing."""
    e, k, t = case["experts"], case["top_k"], case["tokens"]
    return e * (1.0 - (1.0 - k / e) ** t)


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        # logits and bias in; ids, weights and sorted order out, offsets out;
        # an exponential, a division and two comparisons per logit
        return {"bytes": t * e * _SIZE[case["logits"]] + 4 * e * case["bias"] + t * k * 12 +
                (e + 1) * 4, "flops": 4 * t * e}
    if case["op"] == "encode":
        n, r, c = case["matrices"], case["rows"], case["cols"]
        scales = n * (-(-r // case["block_rows"])) * _blocks(c)
        # a maximum and a division per value
        return {"bytes": n * r * c * (_SIZE[case["x"]] + 1) + 4 * scales, "flops": 2 * n * r * c}
    t, uses = case["tokens"], case["tokens"] * case["top_k"]
    rows, cols, out = _dims(case)
    matrix = rows * cols + 4 * _blocks(rows) * _blocks(cols)
    x_rows = t if case["stage"] == "gateup" else uses
    return {"bytes": int(_active(case) * matrix) + x_rows * (cols + 4 * _blocks(cols)) +
            uses * out * _SIZE[case["y"]] + uses * 4 + (case["experts"] + 1) * 4,
            "flops": 2 * uses * rows * cols}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _plan(g, case):
    """A router's result over this case's experts: uses sorted by expert.
    skew > 0 makes some experts more popular than others."""
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    logits = _randn(g, t, e) + case["skew"] * _randn(g, 1, e)
    ids = torch.topk(logits, k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices.to(torch.int32)
    counts = torch.bincount(ids, minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, order


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        s["logits"] = _randn(g, t, e).to(_T[case["logits"]])
        s["bias"] = 0.05 * _randn(g, e) if case["bias"] else None
        s["ids"] = torch.empty(t, k, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(t, k, device="cuda")
        s["offsets"] = torch.empty(e + 1, dtype=torch.int32, device="cuda")
        s["order"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
        # a workspace that serves every size of these ranges
        s["ws"] = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        return s
    if case["op"] == "encode":
        n, r, c, b = case["matrices"], case["rows"], case["cols"], case["block_rows"]
        if b == 1:
            # activations: normalised, a few inputs much larger than the others
            s["x"] = _randn(g, r, c)
            s["x"][:, torch.randperm(c, generator=g, device="cuda")[:max(1, c // 256)]] *= 30.0
            s["x"] = s["x"].to(_T[case["x"]])
        else:
            s["x"] = (0.02 * _randn(g, n, r, c)).to(_T[case["x"]])
        s["q"] = torch.empty(s["x"].shape, dtype=_F8, device="cuda")
        s["scales"] = torch.empty(*s["x"].shape[:-2], -(-r // b), _blocks(c), device="cuda")
        return s
    rows, cols, out = _dims(case)
    e, t, k = case["experts"], case["tokens"], case["top_k"]
    s["offsets"], s["order"] = _plan(g, case)
    # gate/up reads its tokens' rows; down reads h, already in sorted order
    # and smaller than a normalised activation
    if case["stage"] == "gateup":
        x = _randn(g, t, cols)
    else:
        x = _randn(g, t * k, cols) * _randn(g, t * k, cols).abs() * 0.5
    s["x"], s["xs"] = _plain_encode(x[None], 1)
    s["x"], s["xs"] = s["x"][0], s["xs"][0]
    # weights of deviation 0.02 whose largest in a block is some 4 deviations
    s["ws"] = (0.02 * 4.2 / 448.0) * (0.9 + 0.2 * torch.rand(
        e, _blocks(rows), _blocks(cols), generator=g, device="cuda"))
    s["W"] = torch.empty(e, rows, cols, dtype=_F8, device="cuda")
    step = max(1, (1 << 28) // (rows * cols))
    for e0 in range(0, e, step):
        n = min(step, e - e0)
        v = _randn(g, n, rows, cols, dtype=torch.float16)
        s["W"][e0:e0 + n] = v.mul_(448.0 / 4.2).clamp_(-448.0, 448.0).to(_F8)
    s["y"] = torch.zeros(t * k, out, dtype=_T[case["y"]], device="cuda")
    return s


# ---------------------------------------------------------------- passes
def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "route":
        return _plain_route(s, case)
    if case["op"] == "encode":
        x = s["x"] if s["x"].dim() == 3 else s["x"][None]
        q, scales = _plain_encode(x, case["block_rows"])
        return q.reshape(s["q"].shape), scales.reshape(s["scales"].shape)
    return _plain_grouped(s, case)


def _own(s, case):
    import bitplane_quantized_expert_amd as pm
    stream = torch.cuda.current_stream()
    if case["op"] == "route":
        if "rule" not in s:
            # the model's routing rule, made once
            s["rule"] = pm.pm_route_rule(
                pm.PM_SCORE_SIGMOID if case["score"] == "sigmoid" else pm.PM_SCORE_SOFTMAX,
                case["n_groups"], case["top_groups"], case["group_best"],
                pm.PM_ROUTE_RENORM if case["renorm"] else 0, case["scale"])
        pm.pm_route_scored_device(s["rule"], s["logits"], s["bias"], case["top_k"], s["ids"],
                                  s["w"], s["offsets"], s["order"], s["ws"], stream)
        return s["ids"], s["w"], s["offsets"], s["order"]
    if case["op"] == "encode":
        pm.pm_encode_fp8_device(s["x"], s["q"], s["scales"], case["block_rows"], stream)
        return s["q"], s["scales"]
    # gate/up gathers its tokens' rows and forms SiLU(gate) * up; down writes
    # its rows back in the order of the uses
    if case["stage"] == "gateup":
        flags = pm.PM_GROUPED_GATHER | pm.PM_GROUPED_SWIGLU
    else:
        flags = pm.PM_GROUPED_SCATTER
    pm.pm_grouped_gemm_fp8(s["W"], s["ws"], s["x"], s["xs"], s["y"], s["offsets"], s["order"],
                           case["top_k"], flags, stream)
    return s["y"]


def _plain_route(s, case):
    """Scores and choices in fp64: whole numbers have to come out the same."""
    t, e, k, n = case["tokens"], case["experts"], case["top_k"], case["n_groups"]
    l = s["logits"].double()
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        score = p / p.sum(1, keepdim=True)
    c = score if s["bias"] is None else score + s["bias"].double()
    if n > 1:
        best = torch.topk(c.reshape(t, n, e // n), min(case["group_best"], e // n), dim=2).values
        kept = torch.sort(best.sum(2), dim=1, descending=True,
                          stable=True).indices[:, :case["top_groups"]]
        keep = (kept[:, :, None] == torch.arange(n, device=l.device)).any(1)
        c = torch.where(keep.repeat_interleave(e // n, 1), c, -math.inf)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k].contiguous()
    w = torch.gather(score, 1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * case["scale"]).float()
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=l.device)
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=e), 0)
    return ids.to(torch.int32), w, offsets, order.to(torch.int32)


def _plain_encode(x, block_rows):
    """Codes and scales of x [n][rows][cols], one scale per block of block_rows
    x 128: the largest of a block is 448, e4m3's largest."""
    n, r, c = x.shape
    rb, cb = -(-r // block_rows), _blocks(c)
    v = torch.nn.functional.pad(x.float(), (0, cb * BLOCK - c, 0, rb * block_rows - r))
    v = v.reshape(n, rb, block_rows, cb, BLOCK)
    # (no smaller than the least normal number: a block of zeros has codes of 0)
    scales = (v.abs().amax((2, 4)) / 448.0).clamp(min=2.0 ** -126)
    v = v / scales[:, :, None, :, None]
    q = v.reshape(n, rb * block_rows, cb * BLOCK)[:, :r, :c].to(_F8)
    return q, scales


def _plain_decode(q, scales, block_rows):
    """fp32 values of codes q [n][rows][cols]."""
    n, r, c = q.shape
    scales = scales.repeat_interleave(BLOCK, 2)[:, :, :c]
    if block_rows > 1:
        scales = scales.repeat_interleave(block_rows, 1)[:, :r]
    return q.float().mul_(scales)


def _plain_grouped(s, case):
    """The experts that have rows, each group padded to the longest, as one
    batched fp32 product."""
    off, order, y = s["offsets"].long(), s["order"].long(), s["y"]
    counts = off[1:] - off[:-1]
    active = counts.nonzero()[:, 0]
    at = torch.arange(int(counts.max()), device=y.device)
    valid = at < counts[active][:, None]
    pos = torch.where(valid, off[active][:, None] + at, 0)
    gateup = case["stage"] == "gateup"
    xr = order[pos] // case["top_k"] if gateup else pos
    x = _plain_decode(s["x"][None], s["xs"][None], 1)[0][xr]
    w = _plain_decode(s["W"].view(torch.uint8)[active].view(_F8), s["ws"][active], BLOCK)
    p = torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2)[valid]
    if gateup:
        gate, up = p[:, :case["inter"]], p[:, case["inter"]:]
        y.copy_(gate / (1.0 + torch.exp(-gate)) * up)
    else:
        y[order] = p.to(y.dtype)
    return y


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s, case)
    if case["op"] == "encode":
        return _exact_encode(s, case)
    rows, cols, out = _dims(case)
    uses = case["tokens"] * case["top_k"]
    y = torch.zeros(uses, out, dtype=torch.float64, device="cuda")
    row, col = torch.arange(rows, device="cuda"), torch.arange(cols, device="cuda")
    x = s["x"].double() * s["xs"].double()[:, col // BLOCK]
    ends = s["offsets"].tolist()
    for e in range(case["experts"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        use = s["order"][a:b].long()
        w = s["W"][e].double() * s["ws"][e].double()[row // BLOCK][:, col // BLOCK]
        if case["stage"] == "gateup":
            xs = x[torch.div(use, case["top_k"], rounding_mode="floor")]
            gate, up = torch.matmul(xs, w.T).split(case["inter"], dim=1)
            y[a:b] = gate * torch.sigmoid(gate) * up
        else:
            y[use] = torch.matmul(x[a:b], w.T)
    return y


def _exact_route(s, case):
    t, e, k, n = case["tokens"], case["experts"], case["top_k"], case["n_groups"]
    l = s["logits"].double()
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    c = score.clone()
    if s["bias"] is not None:
        c += s["bias"].double()
    rows = torch.arange(t, device="cuda")
    # groups and experts one at a time, the first of the largest
    value = torch.zeros(t, n, dtype=torch.float64, device="cuda")
    left = c.reshape(t, n, e // n).clone()
    for _ in range(min(case["group_best"], e // n)):
        top = left.max(2)
        value += top.values
        left.scatter_(2, top.indices[:, :, None], -math.inf)
    closed = torch.ones(t, n, dtype=torch.bool, device="cuda")
    for _ in range(case["top_groups"]):
        first = _first_largest(value)
        closed[rows, first] = False
        value[rows, first] = -math.inf
    c[closed.repeat_interleave(e // n, 1)] = -math.inf
    ids = torch.empty(t, k, dtype=torch.int64, device="cuda")
    for j in range(k):
        ids[:, j] = _first_largest(c)
        c[rows, ids[:, j]] = -math.inf
    w = score.gather(1, ids)
    if case["renorm"]:
        w /= w.sum(1, keepdim=True)
    by_expert = torch.sort(ids.reshape(-1), stable=True)
    offsets = torch.searchsorted(by_expert.values, torch.arange(e + 1, device="cuda"))
    return (ids.to(torch.int32), w * case["scale"], offsets.to(torch.int32),
            by_expert.indices.to(torch.int32))


def _first_largest(v):
    at = torch.arange(v.shape[1], device=v.device)
    return torch.where(v == v.max(1, keepdim=True).values, at, v.shape[1]).min(1).values


def _exact_encode(s, case):
    """Codes are those of x over the scale as it is held, in 32 bits."""
    r, c, b = case["rows"], case["cols"], case["block_rows"]
    x = s["x"].double().reshape(-1, r, c)
    q, scales = torch.empty_like(x), []
    for j in range(0, c, BLOCK):
        for i in range(0, r, b if b > 1 else r):
            v = x[:, i:i + (b if b > 1 else r), j:j + BLOCK]
            top = v.abs().amax((1, 2) if b > 1 else 2, keepdim=True)
            scale = (top / 448.0).clamp(min=2.0 ** -126)
            scales.append(scale[:, :, 0])
            v = v / scale.float().double()
            # steps of 2^-3 of the power of two below the value, 2^-9 at least
            step = torch.exp2(torch.frexp(v)[1].clamp(min=-5).double() - 4.0)
            q[:, i:i + v.shape[1], j:j + BLOCK] = torch.round(v / step) * step
    cb = _blocks(c)
    if b > 1:
        scales = torch.cat(scales, 1).reshape(-1, cb, -(-r // b)).transpose(1, 2)
    else:
        scales = torch.stack(scales, 2)
    return q.reshape(s["q"].shape), scales.reshape(s["scales"].shape)
