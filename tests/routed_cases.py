"""Plain fp64 forms of the routed experts' device operators, and their inputs."""
import numpy as np
import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def route_plain(logits, top_k):
    """ids, w (fp64), offsets and order of logits [T][E] (any float type), on
    the host: -inf and NaN are never selected."""
    l = logits.double().cpu().numpy()
    T, E = l.shape
    ids = np.full((T, top_k), -1, np.int32)
    w = np.zeros((T, top_k))
    ok = ~np.isnan(l) & (l > -np.inf)
    for t in range(T):
        cand = np.nonzero(ok[t])[0]
        # descending logit, ties by ascending id
        cand = cand[np.lexsort((cand, -l[t, cand]))][:top_k]
        n = len(cand)
        if n == 0:
            continue
        v = l[t, cand]
        ex = np.array([1.0 if a == v[0] else np.exp(a - v[0]) for a in v])
        ids[t, :n] = cand
        w[t, :n] = ex / ex.sum()
    flat = ids.reshape(-1)
    order = np.concatenate([np.nonzero(flat == e)[0] for e in range(E)]).astype(np.int32)
    counts = np.array([(flat == e).sum() for e in range(E)])
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return ids, w, offsets, order


def groups(counts, seed, n_rows=None):
    """offsets (int32) of the given group sizes and a shuffled order over
    n_rows uses (the sum of the counts by default)."""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(off[-1]) if n_rows is None else n_rows
    order = np.random.default_rng(seed).permutation(n).astype(np.int32)
    return torch.from_numpy(off).cuda(), torch.from_numpy(order).cuda()


def decode_w4(q, scales, zeros, group):
    """fp64 weights [..., cols] of 4-bit codes."""
    q = q.long()
    v = torch.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1).double()
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, -1)
    return (v - z) * scales.double().repeat_interleave(group, -1)


def grouped_plain(w64, x, offsets, order, n_rows, top_k, gather, scatter, swiglu, bad=()):
    """For fp64 weights [E][R][C] (a function of e): a list of (y row, values,
    bound) over the rows the call has to write, where bound is the largest
    allowed error of fp32 sums in any order: with u = 2^-24, a sum of C exact
    (16-bit) products is off by at most C * 2u * S, S = sum |w x|, when every
    addition rounds or cuts off at one fp32 step; 16 more such steps cover the
    scales, the split of an fp32 x and the joining of parts."""
    off = offsets.tolist()
    ordl = list(range(n_rows)) if order is None else order.tolist()
    out = []
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        w = w64(e)
        us = ordl[a:b]
        xr = [u // top_k for u in us] if gather else list(range(a, b))
        yr = us if scatter else list(range(a, b))
        keep = [i for i, u in enumerate(us) if 0 <= u < n_rows]
        if not keep:
            continue
        xs = x[torch.tensor([xr[i] for i in keep], device=x.device)].double()
        p = xs @ w.T
        tol = (w.shape[1] + 16) * 2.0 ** -23 * (xs.abs() @ w.abs().T) + 2.0 ** -126
        if swiglu:
            h = w.shape[0] // 2
            g, v, dg, dv = p[:, :h], p[:, h:], tol[:, :h], tol[:, h:]
            s = g * torch.sigmoid(g)
            # |SiLU'| < 1.1; 16 steps for the exponential, division and products
            tol = 1.1 * dg * (v.abs() + dv) + s.abs() * dv + 16 * 2.0 ** -24 * (s * v).abs() + \
                2.0 ** -126
            p = s * v
        out.append((torch.tensor([yr[i] for i in keep], device=x.device), p, tol))
    return out


def check_grouped(y, fill, want, what=""):
    """y against grouped_plain's rows; every other row still holds `fill`."""
    half = HALF_STEP[y.dtype]
    tiny = torch.finfo(y.dtype).smallest_normal * half
    touched = torch.zeros(y.shape[0], dtype=torch.bool, device=y.device)
    for rows, p, tol in want:
        got = y[rows].double()
        touched[rows] = True
        lim = tol + half * (p.abs() + tol) + tiny
        # beyond the type's largest value the rounded result is an infinity
        big = p.abs() + lim > torch.finfo(y.dtype).max
        bad = ~((got - p).abs() <= lim) & ~big
        assert not bad.any(), (
            f"{what}: {int(bad.sum())} of {bad.numel()} off; worst "
            f"{float(((got - p).abs() / lim)[~big].max()):.3g} of the bound; first at "
            f"{bad.nonzero()[0].tolist()}")
    rest = y[~touched].float()
    assert torch.equal(rest, torch.full_like(rest, fill)), f"{what}: rows outside the groups"
