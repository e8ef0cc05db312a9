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
