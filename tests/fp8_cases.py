"""Plain fp64 forms of the scored router and the 8-bit operators, on the host
or the device, with bounds that follow from the steps of the sums."""
import numpy as np
import torch

import routed_cases as rc

F8 = torch.float8_e4m3fn
BLOCK = 128


# ---------------------------------------------------------------- scored router
def scored_plain(logits, bias, top_k, score, n_groups=1, top_groups=1, group_best=1, renorm=False,
                 scale=1.0):
    """ids, w (fp64), offsets and order of logits [T][E], token by token in
    NumPy fp64."""
    l = logits.double().cpu().numpy()
    T, E = l.shape
    b = np.zeros(E) if bias is None else bias.double().cpu().numpy()
    size = E // n_groups
    ids = np.full((T, top_k), -1, np.int32)
    w = np.zeros((T, top_k))
    for t in range(T):
        seen = ~np.isnan(l[t]) & (l[t] > -np.inf)
        s = np.zeros(E)
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s[seen] = 1.0 / (1.0 + np.exp(-l[t, seen]))
            elif seen.any():
                top = l[t, seen].max()
                s[seen] = [1.0 if v == top else np.exp(v - top) for v in l[t, seen]]
                s[seen] /= s[seen].sum()
        ok = seen & ~np.isnan(b) & (b > -np.inf)
        c = np.where(ok, s + np.where(ok, b, 0.0), -np.inf)
        if n_groups > 1:
            value = np.full(n_groups, -np.inf)
            for g in range(n_groups):
                best = np.sort(c[g * size:(g + 1) * size])[::-1][:group_best]
                best = best[best > -np.inf]
                if len(best):
                    value[g] = best.sum()
            kept = [g for g in np.lexsort((np.arange(n_groups), -value)) if value[g] > -np.inf]
            keep = np.zeros(n_groups, bool)
            keep[kept[:top_groups]] = True
            c = np.where(np.repeat(keep, size), c, -np.inf)
        cand = np.nonzero(c > -np.inf)[0]
        cand = cand[np.lexsort((cand, -c[cand]))][:top_k]
        n = len(cand)
        if n == 0:
            continue
        v = s[cand]
        if renorm:
            v = v / v.sum() if v.sum() > 0 else np.zeros(n)
        ids[t, :n] = cand
        w[t, :n] = v * scale
    flat = ids.reshape(-1)
    order = np.concatenate([np.nonzero(flat == e)[0] for e in range(E)]).astype(np.int32)
    counts = np.array([(flat == e).sum() for e in range(E)])
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return ids, w, offsets, order


# ---------------------------------------------------------------- encoder
def round_e4m3(v):
    """fp64 values rounded to the nearest e4m3 (ties to the even code), on a
    grid of 2^-3 of the power of two below, 2^-9 at least."""
    step = np.exp2(np.clip(np.frexp(v)[1], -5, None) - 4.0)
    return np.rint(v / step) * step


def encode_plain(x, block_rows):
    """Values of the codes (fp64, NaN where x is not finite) and fp32 scales of
    x [n][rows][cols].  Quotients of fp32 numbers in fp64: their 53 bits tell
    every quotient from the borders of two codes (which differ from it by 2^-29
    of it at least, or not at all), and round to fp32 as the exact ones do."""
    x = x.double().cpu().numpy()
    n, r, c = x.shape
    rb, cb = -(-r // block_rows), -(-c // BLOCK)
    q = np.empty_like(x)
    scales = np.empty((n, rb, cb), np.float32)
    for i in range(rb):
        for j in range(cb):
            v = x[:, i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            fin = np.isfinite(v)
            top = np.where(fin, np.abs(v), 0.0).max((1, 2))
            s = np.maximum((top / 448.0).astype(np.float32), np.float32(2.0 ** -126))
            scales[:, i, j] = s
            d = (np.where(fin, v, 0.0) / s.astype(np.float64)[:, None, None])
            d = round_e4m3(d)
            q[:, i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK] = \
                np.where(fin, d, np.nan)
    return q, scales


# ---------------------------------------------------------------- products
def make_weights(E, R, C, seed):
    """Codes of normal weights (every finite code occurs) and their scales."""
    g = rc.gen(seed)
    w = torch.randn(E, R, C, generator=g, device="cuda").mul_(100.0).clamp_(-448.0, 448.0).to(F8)
    s = 0.0002 * (0.5 + torch.rand(E, -(-R // BLOCK), -(-C // BLOCK), generator=g, device="cuda"))
    return w, s


def make_x(n, C, seed, ld=None, spread=True):
    """Codes of n rows (in a buffer of `ld` columns) and their scales."""
    g = rc.gen(seed)
    x = torch.randn(n, ld or C, generator=g, device="cuda").mul_(60.0)
    if spread:
        x[:, ::37] *= 40.0                          # a few much larger inputs
    x = x.clamp_(-448.0, 448.0).to(F8)[:, :C]
    s = 0.01 * (0.25 + torch.rand(n, -(-C // BLOCK), generator=g, device="cuda"))
    return x, s


def decode(q, scales, block_rows):
    """fp64 values of codes q [..., rows, cols]."""
    r, c = q.shape[-2:]
    s = scales.double().repeat_interleave(BLOCK, -1)[..., :c]
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, -2)[..., :r, :]
    return q.double() * s


def grouped_plain(W, ws, x, xs, offsets, order, n_rows, top_k, gather, scatter, swiglu, bf16):
    """Rows, values and bounds as in routed_cases.grouped_plain.  Beside its
    (cols + 16) fp32 steps there is, for bf16 results, what the matrix cores
    cut off: of any 8 adjacent products each loses less than 2^-13 of the
    largest one's power of two, where codes below 2^-6 count as 2^-6: at most
    7 * 2^-13 of that product, so less than 2^-10 of the sum of all products of
    codes of at least 2^-6."""
    off = offsets.tolist()
    ordl = list(range(n_rows)) if order is None else order.tolist()
    x64 = decode(x, xs[:x.shape[0]], 1)
    one = torch.ones((), dtype=torch.float64, device=x.device)

    def up(q):
        return torch.where(q.double().abs() < 2.0 ** -6, one * 2.0 ** -6, q.double().abs())

    x_up = up(x) * xs[:x.shape[0]].double().repeat_interleave(BLOCK, -1)[:, :x.shape[1]]
    out = []
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        us = ordl[a:b]
        xr = [u // top_k for u in us] if gather else list(range(a, b))
        yr = us if scatter else list(range(a, b))
        keep = [i for i, u in enumerate(us) if 0 <= u < n_rows]
        if not keep:
            continue
        w = decode(W[e], ws[e], BLOCK)
        rows = torch.tensor([xr[i] for i in keep], device=x.device)
        p = x64[rows] @ w.T
        tol = (w.shape[1] + 16) * 2.0 ** -23 * (x64[rows].abs() @ w.abs().T) + 2.0 ** -126
        if bf16:
            w_up = up(W[e]) * decode(torch.ones_like(W[e].float()), ws[e], BLOCK)
            tol = tol + 2.0 ** -10 * (x_up[rows] @ w_up.T)
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
