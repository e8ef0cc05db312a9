"""Argument checks of the scored router and the 8-bit operators, without a GPU:
every refusal happens before any HIP call, so made-up addresses are never
used; and the plain forms of the tests against torch's own e4m3 type."""
import concurrent.futures
import os
import subprocess

import numpy as np
import pytest
import torch

import bitplane_quantized_expert_amd as pm
import fp8_cases as fc
from bitplane_quantized_expert_amd import build
import test_routed_host as routed
from test_routed_host import A, B, D, OFF, ORD, WS, refused, rows, shape, status

S1, S2 = A + (1 << 35), B + (1 << 35)


def rule(score=pm.PM_SCORE_SIGMOID, n_groups=4, top_groups=2, group_best=2, flags=0, scale=1.0):
    return pm.pm_route_rule(score, n_groups, top_groups, group_best, flags, scale)


def scored(T=4, E=16, K=2, r=None, l=A, ty=pm.PM_F32, ld=16, bias=S1, ids=B, w=B + 4096, off=OFF,
           order=ORD, ws=WS, wsb=1 << 20):
    return status("pm_route_scored_device", T, E, K, r or rule(), l, ty, ld, bias, ids, w, off,
                  order, ws, wsb, None)


def test_scored_route_refusals():
    refused(scored(T=-1), pm.PM_ERR_ARG)
    refused(scored(E=0), pm.PM_ERR_ARG)
    refused(scored(K=0), pm.PM_ERR_ARG)
    refused(scored(K=17), pm.PM_ERR_ARG)
    refused(scored(E=4100, ld=4100), pm.PM_ERR_SHAPE)
    refused(scored(E=100, ld=100, K=65), pm.PM_ERR_SHAPE)
    refused(scored(T=1 << 30, K=2), pm.PM_ERR_ARG)
    refused(scored(ty=3), pm.PM_ERR_ARG, "type")
    refused(scored(ld=15), pm.PM_ERR_ARG, "distance")
    refused(scored(order=None), pm.PM_ERR_ARG, "together")
    for k in ("l", "ids", "w"):
        refused(scored(**{k: None}), pm.PM_ERR_ARG, "null")
    refused(scored(l=A + 2), pm.PM_ERR_ARG, "misaligned")
    refused(scored(bias=S1 + 2), pm.PM_ERR_ARG, "misaligned")
    refused(scored(ws=None), pm.PM_ERR_ARG, "workspace")
    refused(scored(ids=A + 16), pm.PM_ERR_ARG, "overlap")
    refused(scored(ids=S1 + 8), pm.PM_ERR_ARG, "bias")
    refused(scored(r=rule(score=2)), pm.PM_ERR_ARG, "score")
    refused(scored(r=rule(flags=2)), pm.PM_ERR_ARG, "flags")
    refused(scored(r=rule(group_best=0)), pm.PM_ERR_ARG, "group_best")
    refused(scored(r=rule(group_best=3)), pm.PM_ERR_ARG, "group_best")
    refused(scored(r=rule(n_groups=0)), pm.PM_ERR_ARG, "groups")
    refused(scored(r=rule(top_groups=0)), pm.PM_ERR_ARG, "groups")
    refused(scored(r=rule(top_groups=5)), pm.PM_ERR_ARG, "groups")
    refused(scored(r=rule(n_groups=5)), pm.PM_ERR_SHAPE, "one size")
    refused(scored(E=130, ld=130, r=rule(n_groups=65, top_groups=65)), pm.PM_ERR_SHAPE, "at most")
    refused(scored(K=9), pm.PM_ERR_ARG, "top_k")
    for s in (float("nan"), float("inf"), -float("inf")):
        refused(scored(r=rule(scale=s)), pm.PM_ERR_ARG, "scale")
    assert scored(T=0, off=None, order=None, l=None, ids=None, w=None) == pm.PM_OK


def fp8(s=None, w=A, wsc=S1, r=None, x=B, xsc=S2, ldx=None, y=D, yt=pm.PM_BF16, ldy=None, flags=0):
    s = s or shape()
    return status("pm_grouped_gemm_fp8", s, w, wsc, r or rows(), x, xsc,
                  s.cols if ldx is None else ldx, y, yt, s.rows if ldy is None else ldy, flags,
                  None)


def test_grouped_fp8_refusals():
    refused(fp8(s=shape(e=0)), pm.PM_ERR_SHAPE)
    refused(fp8(s=shape(e=pm.PM_GROUPED_MAX_EXPERTS + 1)), pm.PM_ERR_SHAPE, "experts")
    refused(fp8(s=shape(r=-1)), pm.PM_ERR_SHAPE)
    refused(fp8(s=shape(r=1 << 15, c=1 << 15)), pm.PM_ERR_SHAPE, "2^30")
    refused(fp8(s=shape(c=136)), pm.PM_ERR_SHAPE, "multiple of 16")
    refused(fp8(s=shape(r=63), flags=pm.PM_GROUPED_SWIGLU), pm.PM_ERR_SHAPE, "gate")
    refused(fp8(flags=8), pm.PM_ERR_ARG, "flags")
    refused(fp8(r=rows(n=-1)), pm.PM_ERR_ARG)
    refused(fp8(r=rows(k=0)), pm.PM_ERR_ARG)
    refused(fp8(r=rows(n=pm.PM_ROUTED_MAX_USES + 1)), pm.PM_ERR_ARG, "n_rows")
    refused(fp8(yt=3), pm.PM_ERR_ARG, "type")
    refused(fp8(ldx=127), pm.PM_ERR_ARG, "distance")
    refused(fp8(ldy=63), pm.PM_ERR_ARG, "distance")
    refused(fp8(ldx=136), pm.PM_ERR_ARG, "16-byte")
    refused(fp8(x=B + 8), pm.PM_ERR_ARG, "16-byte")
    refused(fp8(y=D + 1), pm.PM_ERR_ARG, "misaligned")
    for k in ("x", "y"):
        refused(fp8(**{k: None}), pm.PM_ERR_ARG, "null")
    for k in ("w", "wsc", "xsc"):
        refused(fp8(**{k: None}), pm.PM_ERR_ARG, "codes or scales")
    refused(fp8(w=A + 8), pm.PM_ERR_ARG, "misaligned")
    refused(fp8(wsc=S1 + 2), pm.PM_ERR_ARG, "misaligned")
    refused(fp8(xsc=S2 + 2), pm.PM_ERR_ARG, "misaligned")
    refused(fp8(r=rows(off=None)), pm.PM_ERR_ARG, "null")
    refused(fp8(y=B + 256), pm.PM_ERR_ARG, "overlap")
    refused(fp8(y=A + 4 * 64 * 128 - 2), pm.PM_ERR_ARG, "overlap")
    refused(fp8(y=S1 + 12), pm.PM_ERR_ARG, "overlap")
    refused(fp8(y=S2 + 28), pm.PM_ERR_ARG, "overlap")
    assert fp8(r=rows(n=0, off=None, order=None), x=None, y=None) == pm.PM_OK
    assert fp8(s=shape(r=0), y=None) == pm.PM_OK


def test_fp32_sums_flag():
    """PM_GROUPED_FP32_SUMS is of the 8-bit products alone, and goes with every
    other flag and type."""
    many = pm.PM_GROUPED_GATHER | pm.PM_GROUPED_SCATTER | pm.PM_GROUPED_SWIGLU
    for yt in (pm.PM_F32, pm.PM_F16, pm.PM_BF16):
        for flags in (0, many):
            assert fp8(r=rows(n=0), yt=yt, flags=flags | pm.PM_GROUPED_FP32_SUMS) == pm.PM_OK
    refused(fp8(flags=pm.PM_GROUPED_FP32_SUMS | 8), pm.PM_ERR_ARG, "flags")
    refused(fp8(flags=pm.PM_GROUPED_FP32_SUMS, y=B), pm.PM_ERR_ARG, "overlap")
    refused(routed.gemm(flags=pm.PM_GROUPED_FP32_SUMS), pm.PM_ERR_ARG, "flags")
    refused(routed.w4(flags=pm.PM_GROUPED_FP32_SUMS), pm.PM_ERR_ARG, "flags")


def test_encode_fp8_refusals():
    def enc(n=1, r=2, c=64, g=128, b=1, x=A, ty=pm.PM_F32, ldx=64, q=B, ldq=64, s=D):
        return status("pm_encode_fp8_device", n, pm.mshape(r, c, g), b, x, ty, ldx, q, ldq, s,
                      None)
    refused(enc(n=-1), pm.PM_ERR_ARG)
    refused(enc(r=-1), pm.PM_ERR_SHAPE)
    refused(enc(c=72), pm.PM_ERR_SHAPE)
    refused(enc(g=64), pm.PM_ERR_SHAPE)
    refused(enc(b=2), pm.PM_ERR_ARG, "1 or 128")
    refused(enc(n=1 << 20, r=1 << 20), pm.PM_ERR_ARG, "matrices")
    refused(enc(ty=3), pm.PM_ERR_ARG, "type")
    refused(enc(ldx=63), pm.PM_ERR_ARG, "distance")
    refused(enc(ldq=63), pm.PM_ERR_ARG, "distance")
    refused(enc(ldx=66), pm.PM_ERR_ARG, "misaligned")
    refused(enc(ldq=72), pm.PM_ERR_ARG, "misaligned")
    for k in ("x", "q", "s"):
        refused(enc(**{k: None}), pm.PM_ERR_ARG, "null")
    refused(enc(x=A + 8), pm.PM_ERR_ARG, "misaligned")
    refused(enc(q=B + 8), pm.PM_ERR_ARG, "misaligned")
    refused(enc(s=D + 2), pm.PM_ERR_ARG, "misaligned")
    refused(enc(q=A + 496), pm.PM_ERR_ARG, "overlap")
    refused(enc(s=B + 124), pm.PM_ERR_ARG, "overlap")
    for k in ("n", "r"):
        assert enc(**{k: 0}, x=None) == pm.PM_OK


def test_binding_refusals_without_a_gpu():
    x, q, s = torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="device"):
        pm.pm_encode_fp8_device(x, q, s)
    with pytest.raises(ValueError, match="device"):
        pm.pm_route_scored_device(rule(), torch.zeros(4, 16), None, 2,
                                  torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))


def test_plain_e4m3_is_torchs():
    """The tests' own rounding against torch's cast, ties and both ends among
    the values."""
    v = torch.cat([torch.linspace(-464, 464, 40001), torch.randn(40000) * 0.01,
                   torch.arange(-1200, 1200) * 2.0 ** -11, torch.arange(-500, 500) / 2.0])
    v = v[v.abs() <= 448]
    assert np.array_equal(fc.round_e4m3(v.double().numpy()), v.to(fc.F8).double().numpy())


SOURCES = [s for s in build.TARGETS[0][1]
           if os.path.basename(s).startswith(("pm_fp8", "pm_scored"))]


def test_entry_points_have_nothing_that_throws(tmp_path):
    """The host code of the operators neither allocates nor locks: no C++
    exception can leave a C entry point."""
    assert len(SOURCES) >= 3

    def undefined(src):
        obj = tmp_path / (os.path.basename(src) + ".o")
        subprocess.run([build.hipcc(), *build.COMPILE_FLAGS, "--cuda-host-only", "-x", "hip", "-c",
                        src, "-o", str(obj)], check=True, capture_output=True)
        return subprocess.run(["nm", "-u", str(obj)], check=True, capture_output=True,
                              text=True).stdout
    with concurrent.futures.ThreadPoolExecutor(4) as ex:
        for src, names in zip(SOURCES, ex.map(undefined, SOURCES)):
            for bad in ("_Znw", "_Zna", "__cxa_throw", "__cxa_allocate_exception", "_ZSt", "malloc",
                        "pthread_mutex"):
                assert bad not in names, (src, bad, names)
