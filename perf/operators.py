"""The routed expert layer's operators as measured workloads.

A layer that keeps its experts as 16-bit or 4-bit matrices runs four
operators on the device: the router (top-k, softmax over the selected, uses
sorted by expert), the products grouped by expert with 16-bit weights, the
same products with 4-bit weights and group scales, and the routing-weighted
combine.  Every case is one call of one of them.

`run` computes a case in elementary torch operations in fp32 (own False) or
calls the library's entry point (own True); `exact` computes it in fp64.
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- cases
def listed():
    """The shapes are those of the repository's workloads (512 experts, hidden
    4096, intermediate 1024, top-10; hidden 256, intermediate 128), of common
    smaller layers, and odd ones."""
    return [
        # one decode token's routing: latency only
        _route("route-decode", 1, 512, 10, "f32"),
        # bf16 logits of an odd batch over few experts: many equal logits
        _route("route-ragged", 1003, 60, 4, "bf16"),
        # a prefill's routing
        _route("route-prefill", 16384, 512, 10, "f32"),

        # gate and up of one token in the small expert: the smallest product
        _gemm("gemm-tiny", 1, 16, 2, 256, 128, "gateup", "f16", "f32"),
        # eight decode tokens over 512 experts: about one row per expert
        _gemm("gemm-decode", 8, 512, 10, 4096, 1024, "gateup", "f16", "f16"),
        # sizes that fit no tile, a batch of a few rows per expert and more
        _gemm("gemm-odd", 333, 40, 6, 1000, 713, "gateup", "bf16", "f32"),
        # prefill over 512 experts: about 80 rows per expert, weights dominate
        _gemm("gemm-prefill", 4096, 512, 10, 4096, 1024, "down", "bf16", "bf16"),
        # prefill over few experts: thousands of rows per expert, uneven
        _gemm("gemm-large", 8192, 32, 8, 4096, 1024, "gateup", "bf16", "bf16", skew=0.5),

        # one decode token with 4-bit experts, fp32 activations as in the
        # prefix path
        _w4("w4-decode", 1, 512, 10, 4096, 1024, 128, "gateup", False, "f32", "f32"),
        # a decode batch with 4-bit experts and zero points
        _w4("w4-batch", 64, 512, 10, 4096, 1024, 128, "down", True, "bf16", "bf16"),

        # a decode batch's combine
        _combine("combine-decode", 8, 10, 4096, "f32", "f32"),
        # a prefill's combine
        _combine("combine-prefill", 8191, 10, 4096, "bf16", "bf16"),
    ]


def _route(name, tokens, experts, top_k, logits):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k,
            "logits": logits}


def _gemm(name, tokens, experts, top_k, hidden, inter, stage, w, y, skew=0.0):
    return {"name": name, "op": "gemm", "tokens": tokens, "experts": experts, "top_k": top_k,
            "hidden": hidden, "inter": inter, "stage": stage, "w": w, "x": w, "y": y,
            "skew": skew}


def _w4(name, tokens, experts, top_k, hidden, inter, group, stage, zeros, x, y):
    return {"name": name, "op": "w4", "tokens": tokens, "experts": experts, "top_k": top_k,
            "hidden": hidden, "inter": inter, "group": group, "stage": stage, "zeros": zeros,
            "x": x, "y": y, "skew": 0.0}


def _combine(name, tokens, top_k, hidden, z, y):
    return {"name": name, "op": "combine", "tokens": tokens, "top_k": top_k, "hidden": hidden,
            "z": z, "y": y}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "gemm", "gemm", "gemm", "w4", "w4", "combine"])
    if op == "route":
        experts = _log_int(rng, 4, 512)
        return _route(None, _log_int(rng, 1, 16384), experts,
                      rng.randint(1, min(10, experts)), rng.choice(["f32", "f32", "bf16", "f16"]))
    if op == "combine":
        top_k = rng.randint(1, 10)
        t = rng.choice(["f32", "bf16", "f16"])
        return _combine(None, _log_int(rng, 1, 8191 if t != "f32" else 4000), top_k,
                        _log_int(rng, 128, 4096), t, rng.choice([t, "f32"]))
    top = {c["name"]: work(c) for c in listed() if c["op"] == op}
    flops = max(v["flops"] for v in top.values())
    nbytes = max(v["bytes"] for v in top.values())
    while True:
        experts = _log_int(rng, 4, 512)
        top_k = rng.randint(1, min(10, experts))
        stage = rng.choice(["gateup", "down"])
        if op == "gemm":
            w = rng.choice(["f16", "bf16"])
            # 16-bit rows are multiples of 8 inputs; the output side is free
            hidden = 8 * _log_int(rng, 16, 512)
            inter = 8 * _log_int(rng, 8, 256)
            if stage == "gateup":
                inter = max(64, inter - rng.randint(0, 7))
            else:
                hidden = max(64, hidden - rng.randint(0, 7))
            case = _gemm(None, _log_int(rng, 1, 8192), experts, top_k, hidden, inter, stage, w,
                         rng.choice([w, "f32"]), rng.choice([0.0, 0.5]))
        else:
            # the input side is whole groups, the output side is free
            group = rng.choice([32, 64, 128, 128])
            if stage == "gateup":
                hidden = group * _log_int(rng, 1, 4096 // group)
                inter = _log_int(rng, 64, 2048)
            else:
                hidden = _log_int(rng, 64, 4096)
                inter = group * _log_int(rng, 1, 2048 // group)
            x = rng.choice(["f32", "bf16", "f16"])
            case = _w4(None, _log_int(rng, 1, 256), experts, top_k, hidden, inter, group, stage,
                       rng.random() < 0.5, x, rng.choice([x, "f32"]))
        v = work(case)
        if v["flops"] <= flops and v["bytes"] <= nbytes:
            return case


# ---------------------------------------------------------------- sizes
def _dims(case):
    """Rows and columns of one expert's weight matrix and the output width."""
    if case["stage"] == "gateup":
        return 2 * case["inter"], case["hidden"], case["inter"]
    return case["hidden"], case["inter"], case["hidden"]


def _active(case):
    """Experts that get a row, as expected of independent even routing."""
    e, k, t = case["experts"], case["top_k"], case["tokens"]
    return e * (1.0 - (1.0 - k / e) ** t)


def work(case):
    t = case["tokens"]
    if case["op"] == "route":
        e, k = case["experts"], case["top_k"]
        # logits in; ids, weights and sorted order out, offsets out; one
        # comparison per logit
        return {"bytes": t * e * _SIZE[case["logits"]] + t * k * 12 + (e + 1) * 4,
                "flops": t * e}
    if case["op"] == "combine":
        k, h = case["top_k"], case["hidden"]
        return {"bytes": t * k * (h * _SIZE[case["z"]] + 4) + t * h * _SIZE[case["y"]],
                "flops": 2 * t * k * h}
    rows, cols, out = _dims(case)
    uses = t * case["top_k"]
    if case["op"] == "gemm":
        matrix = rows * cols * _SIZE[case["w"]]
    else:
        matrix = rows * cols // 2 + rows * (cols // case["group"]) * (3 if case["zeros"] else 2)
    x_rows = t if case["stage"] == "gateup" else uses
    return {"bytes": int(_active(case) * matrix) + x_rows * cols * _SIZE[case["x"]] +
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
    t = case["tokens"]
    s = {"case": case}
    if case["op"] == "route":
        e, k = case["experts"], case["top_k"]
        s["logits"] = _randn(g, t, e).to(_T[case["logits"]])
        s["ids"] = torch.empty(t, k, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(t, k, device="cuda")
        s["offsets"] = torch.empty(e + 1, dtype=torch.int32, device="cuda")
        s["order"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
        if own:
            import bitplane_quantized_expert_amd as pm
            s["ws"] = torch.empty(max(1, pm.pm_route_workspace_bytes(t, e, k)),
                                  dtype=torch.uint8, device="cuda")
        return s
    if case["op"] == "combine":
        k, h = case["top_k"], case["hidden"]
        s["z"] = _randn(g, t * k, h).to(_T[case["z"]])
        s["w"] = torch.softmax(_randn(g, t, k), dim=1)
        s["y"] = torch.empty(t, h, dtype=_T[case["y"]], device="cuda")
        return s
    rows, cols, out = _dims(case)
    e, k = case["experts"], case["top_k"]
    s["offsets"], s["order"] = _plan(g, case)
    # gate/up reads its tokens' rows; down reads h, already in sorted order
    # and smaller than a normalised activation
    if case["stage"] == "gateup":
        s["x"] = _randn(g, t, cols).to(_T[case["x"]])
    else:
        s["x"] = (_randn(g, t * k, cols) * _randn(g, t * k, cols).abs() * 0.5).to(_T[case["x"]])
    s["y"] = torch.zeros(t * k, out, dtype=_T[case["y"]], device="cuda")
    if case["op"] == "gemm":
        s["W"] = torch.empty(e, rows, cols, dtype=_T[case["w"]], device="cuda")
        s["W"].normal_(0.0, 0.02, generator=g)
        return s
    group = case["group"]
    s["q"] = torch.empty(e, rows, cols // 2, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (rows * cols))
    for e0 in range(0, e, step):
        n = min(step, e - e0)
        v = _randn(g, n, rows, cols, dtype=torch.float16)
        v = v.mul_(2.7).add_(8.0).round_().clamp_(0, 15).to(torch.uint8)
        s["q"][e0:e0 + n] = v[..., 0::2] | (v[..., 1::2] << 4)
    s["scales"] = (0.005 + 0.005 * torch.rand(e, rows, cols // group, generator=g, device="cuda")
                   ).to(torch.float16)
    s["zeros"] = None
    if case["zeros"]:
        s["zeros"] = torch.randint(6, 11, (e, rows, cols // group), generator=g, device="cuda",
                                   dtype=torch.uint8)
    return s


# ---------------------------------------------------------------- passes
def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "route":
        return _plain_route(s, case)
    if case["op"] == "combine":
        t, k = case["tokens"], case["top_k"]
        z = s["z"].float().reshape(t, k, -1)
        return (z * s["w"][:, :, None]).sum(1).to(_T[case["y"]])
    return _plain_grouped(s, case)


def _own(s, case):
    import bitplane_quantized_expert_amd as pm
    stream = torch.cuda.current_stream()
    if case["op"] == "route":
        pm.pm_route_topk_device(s["logits"], case["top_k"], s["ids"], s["w"], s["offsets"],
                                s["order"], s["ws"], stream)
        return s["ids"], s["w"], s["offsets"], s["order"]
    if case["op"] == "combine":
        pm.pm_combine_uses(s["z"], s["w"], s["y"], stream)
        return s["y"]
    # gate/up gathers its tokens' rows and forms SiLU(gate) * up; down writes
    # its rows back in the order of the uses
    if case["stage"] == "gateup":
        flags = pm.PM_GROUPED_GATHER | pm.PM_GROUPED_SWIGLU
    else:
        flags = pm.PM_GROUPED_SCATTER
    if case["op"] == "gemm":
        pm.pm_grouped_gemm(s["W"], s["x"], s["y"], s["offsets"], s["order"], case["top_k"],
                           flags, stream)
    else:
        pm.pm_grouped_gemm_w4(s["q"], s["scales"], s["zeros"], case["group"], s["x"], s["y"],
                              s["offsets"], s["order"], case["top_k"], flags, stream)
    return s["y"]


def _plain_route(s, case):
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    l = s["logits"].float()
    # one integer per logit that orders as (logit, lower index first)
    bits = (l + 0.0).view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = bits * 65536 + (65535 - torch.arange(e, device=l.device))
    ids = torch.topk(key, k, dim=1, sorted=True).indices
    v = torch.gather(l, 1, ids)
    p = torch.exp(v - v[:, :1])
    w = p / p.sum(1, keepdim=True)
    flat = ids.reshape(-1)
    order = torch.topk(-(flat * (t * k) + torch.arange(t * k, device=l.device)), t * k,
                       sorted=True).indices
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=l.device)
    offsets[1:] = torch.cumsum((flat[None] == torch.arange(e, device=l.device)[:, None]).sum(1),
                               0)
    return ids.to(torch.int32), w, offsets, order.to(torch.int32)


def _decode4(q, scales, zeros, group, dtype):
    """The values of one matrix: (code - zero) * scale of its group."""
    rows = q.shape[0]
    v = torch.stack((q & 15, q >> 4), dim=2).reshape(rows, -1, group).to(dtype)
    z = 8 if zeros is None else zeros.to(dtype)[:, :, None]
    return ((v - z) * scales.to(dtype)[:, :, None]).reshape(rows, -1)


def _plain_grouped(s, case):
    off = s["offsets"].tolist()
    order = s["order"].long()
    x, y = s["x"], s["y"]
    gateup = case["stage"] == "gateup"
    for e in range(case["experts"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        if case["op"] == "gemm":
            w = s["W"][e].float()
        else:
            w = _decode4(s["q"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e],
                         case["group"], torch.float32)
        if gateup:
            p = x[order[a:b] // case["top_k"]].float() @ w.t()
            gate, up = p[:, :case["inter"]], p[:, case["inter"]:]
            y[a:b] = (gate / (1.0 + torch.exp(-gate)) * up).to(y.dtype)
        else:
            y[order[a:b]] = (x[a:b].float() @ w.t()).to(y.dtype)
    return y


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    s = prepare(case, seed)
    t = case["tokens"]
    if case["op"] == "route":
        e, k = case["experts"], case["top_k"]
        srt = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
        ids = srt.indices[:, :k].contiguous()
        w = torch.softmax(srt.values[:, :k], dim=1)
        by_expert = torch.sort(ids.reshape(-1), stable=True)
        offsets = torch.searchsorted(by_expert.values, torch.arange(e + 1, device="cuda"))
        return (ids.to(torch.int32), w, offsets.to(torch.int32),
                by_expert.indices.to(torch.int32))
    if case["op"] == "combine":
        y = torch.zeros(t, case["hidden"], dtype=torch.float64, device="cuda")
        z = s["z"].reshape(t, case["top_k"], -1)
        for j in range(case["top_k"]):
            y += s["w"][:, j:j + 1].double() * z[:, j].double()
        return y
    rows, cols, out = _dims(case)
    y = torch.zeros(t * case["top_k"], out, dtype=torch.float64, device="cuda")
    counts = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    pos = 0
    for e, n in enumerate(counts):
        at = torch.arange(pos, pos + n, device="cuda")
        use = s["order"][pos:pos + n].long()
        pos += n
        if n == 0:
            continue
        if case["op"] == "gemm":
            w = s["W"][e].double()
        else:
            q, g = s["q"][e], case["group"]
            w = torch.empty(rows, cols, dtype=torch.float64, device="cuda")
            w[:, 0::2] = (q % 16).double()
            w[:, 1::2] = torch.div(q, 16, rounding_mode="floor").double()
            zero = 8.0 if s["zeros"] is None else s["zeros"][e].double().repeat_interleave(g, 1)
            w = (w - zero) * s["scales"][e].double().repeat_interleave(g, 1)
        if case["stage"] == "gateup":
            xs = s["x"].double()[torch.div(use, case["top_k"], rounding_mode="floor")]
            gate, up = torch.matmul(xs, w.T).split(case["inter"], dim=1)
            y[at] = gate * torch.sigmoid(gate) * up
        else:
            y[use] = torch.matmul(s["x"][at].double(), w.T)
    return y
