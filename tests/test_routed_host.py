"""Argument checks of the routed experts' device operators, without a GPU:
every refusal happens before any HIP call, so made-up addresses are never
used."""
import concurrent.futures
import ctypes
import os
import subprocess

import pytest
import torch

import bitplane_quantized_expert_amd as pm
from bitplane_quantized_expert_amd import build

A = 1 << 40                   # made-up device addresses, far apart
B = A + (1 << 36)
D = B + (1 << 36)
OFF, ORD, WS = D + (1 << 36), D + (2 << 36), D + (3 << 36)


def status(f, *args):
    return getattr(pm.lib(), f)(*args)


def refused(st, want, text=""):
    assert st == want, (st, pm.lib().pm_last_error())
    assert text.encode() in pm.lib().pm_last_error()


def route(T=4, E=16, K=2, l=A, ty=pm.PM_F32, ld=16, ids=B, w=B + 4096, off=OFF, order=ORD, ws=WS,
          wsb=1 << 20):
    return status("pm_route_topk_device", T, E, K, l, ty, ld, ids, w, off, order, ws, wsb, None)


def test_route_refusals():
    refused(route(T=-1), pm.PM_ERR_ARG)
    refused(route(E=0), pm.PM_ERR_ARG)
    refused(route(K=0), pm.PM_ERR_ARG)
    refused(route(K=17), pm.PM_ERR_ARG)
    refused(route(E=4097, ld=4097), pm.PM_ERR_SHAPE)
    refused(route(E=100, ld=100, K=65), pm.PM_ERR_SHAPE)
    refused(route(T=1 << 30, K=2), pm.PM_ERR_ARG)
    refused(route(T=pm.PM_ROUTED_MAX_USES + 1, K=1), pm.PM_ERR_ARG)
    refused(route(ty=3), pm.PM_ERR_ARG, "type")
    refused(route(ld=15), pm.PM_ERR_ARG, "distance")
    refused(route(order=None), pm.PM_ERR_ARG, "together")
    refused(route(off=None), pm.PM_ERR_ARG, "together")
    for k in ("l", "ids", "w"):
        refused(route(**{k: None}), pm.PM_ERR_ARG, "null")
    refused(route(l=A + 2), pm.PM_ERR_ARG, "misaligned")
    refused(route(ids=B + 2), pm.PM_ERR_ARG, "misaligned")
    refused(route(ws=WS + 4), pm.PM_ERR_ARG, "misaligned")
    refused(route(ws=None), pm.PM_ERR_ARG, "workspace")
    refused(route(wsb=pm.pm_route_workspace_bytes(4, 16, 2) - 1), pm.PM_ERR_ARG, "workspace")
    refused(route(ids=A + 16), pm.PM_ERR_ARG, "overlap")
    refused(route(w=B + 4), pm.PM_ERR_ARG, "overlap")
    refused(route(ws=ORD), pm.PM_ERR_ARG, "overlap")
    assert route(T=0, off=None, order=None, l=None, ids=None, w=None) == pm.PM_OK


def test_route_workspace_sizes():
    assert pm.pm_route_workspace_bytes(0, 16, 2) == 0
    assert pm.pm_route_workspace_bytes(1, 16, 2) > 0
    assert pm.pm_route_workspace_bytes(-1, 16, 2) == 0
    assert pm.pm_route_workspace_bytes(4, 16, 17) == 0
    # one 16-bit count per (block of tokens, expert), however many tokens
    assert pm.pm_route_workspace_bytes(1 << 22, 512, 10) <= 256 * 512 * 2


def shape(e=4, r=64, c=128):
    return pm.pm_grouped_shape(e, r, c)


def rows(n=8, k=2, off=OFF, order=ORD):
    return pm.pm_grouped_rows(n, k, off, order)


def gemm(s=None, ty=pm.PM_BF16, w=A, r=None, x=B, ldx=None, y=D, yt=pm.PM_BF16, ldy=None, flags=0):
    s = s or shape()
    return status("pm_grouped_gemm", s, ty, w, r or rows(), x, s.cols if ldx is None else ldx, y,
                  yt, s.rows if ldy is None else ldy, flags, None)


def w4(s=None, group=32, q=A, sc=A + (1 << 34), z=None, r=None, x=B, xt=pm.PM_F32, ldx=None, y=D,
       yt=pm.PM_F32, ldy=None, flags=0):
    s = s or shape()
    return status("pm_grouped_gemm_w4", s, group, q, sc, z, r or rows(), x, xt,
                  s.cols if ldx is None else ldx, y, yt, s.rows if ldy is None else ldy, flags,
                  None)


@pytest.mark.parametrize("call", [gemm, w4])
def test_grouped_refusals(call):
    refused(call(s=shape(e=0)), pm.PM_ERR_SHAPE)
    refused(call(s=shape(e=pm.PM_GROUPED_MAX_EXPERTS + 1)), pm.PM_ERR_SHAPE, "experts")
    refused(call(s=shape(r=-1)), pm.PM_ERR_SHAPE)
    refused(call(s=shape(r=1 << 15, c=1 << 15)), pm.PM_ERR_SHAPE, "2^30")
    refused(call(s=shape(r=1 << 30, c=0)), pm.PM_ERR_SHAPE, "2^30")
    refused(call(r=rows(n=pm.PM_ROUTED_MAX_USES + 1)), pm.PM_ERR_ARG, "n_rows")
    refused(call(s=shape(r=63), flags=pm.PM_GROUPED_SWIGLU), pm.PM_ERR_SHAPE, "gate")
    refused(call(flags=8), pm.PM_ERR_ARG, "flags")
    refused(call(r=rows(n=-1)), pm.PM_ERR_ARG)
    refused(call(r=rows(k=0)), pm.PM_ERR_ARG)
    refused(call(yt=pm.PM_F16), pm.PM_ERR_ARG, "type")
    refused(call(ldx=127), pm.PM_ERR_ARG, "distance")
    refused(call(ldy=63), pm.PM_ERR_ARG, "distance")
    refused(call(ldy=31, flags=pm.PM_GROUPED_SWIGLU), pm.PM_ERR_ARG, "distance")
    refused(call(ldx=130), pm.PM_ERR_ARG, "16-byte")
    refused(call(x=B + 8), pm.PM_ERR_ARG, "16-byte")
    refused(call(y=D + 1), pm.PM_ERR_ARG, "misaligned")
    refused(call(x=None), pm.PM_ERR_ARG, "null")
    refused(call(y=None), pm.PM_ERR_ARG, "null")
    refused(call(r=rows(off=None)), pm.PM_ERR_ARG, "null")
    refused(call(r=rows(off=OFF + 2)), pm.PM_ERR_ARG, "misaligned")
    refused(call(y=B + 256), pm.PM_ERR_ARG, "overlap")
    # nothing to do: no launch, no pointers needed
    assert call(r=rows(n=0, off=None, order=None), x=None, y=None) == pm.PM_OK
    assert call(s=shape(r=0), y=None) == pm.PM_OK


def test_grouped_gemm_refusals():
    refused(gemm(ty=pm.PM_F32, yt=pm.PM_F32), pm.PM_ERR_ARG, "type")
    refused(gemm(s=shape(c=132)), pm.PM_ERR_SHAPE, "multiple of 8")
    refused(gemm(w=None), pm.PM_ERR_ARG, "weights")
    refused(gemm(w=A + 8), pm.PM_ERR_ARG, "weights")


def test_grouped_w4_refusals():
    refused(w4(xt=5), pm.PM_ERR_ARG, "type")
    for g in (0, -32, 16, 48, 96):
        refused(w4(group=g), pm.PM_ERR_SHAPE, "group")
    refused(w4(q=None), pm.PM_ERR_ARG, "codes")
    refused(w4(q=A + 4), pm.PM_ERR_ARG, "codes")
    refused(w4(sc=None), pm.PM_ERR_ARG, "scales")
    refused(w4(sc=A + 1), pm.PM_ERR_ARG, "scales")


def test_encode_w4_refusals():
    def enc(r=2, c=64, g=32, w=A, ty=pm.PM_F32, q=B, s=D, z=None):
        return status("pm_encode_w4_device", pm.mshape(r, c, g), w, ty, q, s, z, None)
    refused(enc(r=-1), pm.PM_ERR_SHAPE)
    refused(enc(g=48), pm.PM_ERR_SHAPE)
    refused(enc(c=65), pm.PM_ERR_SHAPE)
    refused(enc(ty=7), pm.PM_ERR_ARG)
    refused(enc(w=None), pm.PM_ERR_ARG, "null")
    refused(enc(q=B + 8), pm.PM_ERR_ARG, "misaligned")
    refused(enc(q=A + 16), pm.PM_ERR_ARG, "overlap")
    refused(enc(z=D), pm.PM_ERR_ARG, "overlap")
    assert enc(r=0, w=None) == pm.PM_OK


def test_combine_refusals():
    def comb(T=3, K=2, H=16, z=A, zt=pm.PM_BF16, ldz=16, w=B, y=D, yt=pm.PM_F32, ldy=16):
        return status("pm_combine_uses", T, K, H, z, zt, ldz, w, y, yt, ldy, None)
    refused(comb(T=-1), pm.PM_ERR_ARG)
    refused(comb(K=0), pm.PM_ERR_ARG)
    refused(comb(H=-1), pm.PM_ERR_ARG)
    refused(comb(T=1 << 30), pm.PM_ERR_ARG)
    refused(comb(T=pm.PM_ROUTED_MAX_USES + 1, K=1), pm.PM_ERR_ARG)
    refused(comb(zt=3), pm.PM_ERR_ARG, "type")
    refused(comb(yt=pm.PM_F16), pm.PM_ERR_ARG, "type")
    refused(comb(ldz=15), pm.PM_ERR_ARG, "distance")
    refused(comb(ldy=15), pm.PM_ERR_ARG, "distance")
    for k in ("z", "w", "y"):
        refused(comb(**{k: None}), pm.PM_ERR_ARG, "null")
    refused(comb(z=A + 1), pm.PM_ERR_ARG, "misaligned")
    refused(comb(y=D + 2), pm.PM_ERR_ARG, "misaligned")
    refused(comb(y=A + 64), pm.PM_ERR_ARG, "overlap")
    refused(comb(y=B), pm.PM_ERR_ARG, "overlap")
    assert comb(T=0, z=None) == pm.PM_OK


def test_binding_refuses_tensors_it_cannot_pass():
    """Types, shapes, strides and devices are checked in Python before the call."""
    f = torch.zeros
    i32 = torch.int32
    with pytest.raises(ValueError, match="device"):
        pm.pm_route_topk_device(f(2, 8), 2, f(2, 2, dtype=i32), f(2, 2))
    with pytest.raises(ValueError, match="adjacent"):
        pm.pm_route_topk_device(f(8, 2).t(), 2, f(2, 2, dtype=i32), f(2, 2))
    with pytest.raises(ValueError, match="w: contiguous"):
        pm.pm_grouped_gemm(f(2, 8), f(1, 8), f(1, 8), f(3, dtype=i32))
    with pytest.raises(ValueError, match="weights"):
        pm.pm_grouped_gemm(f(2, 8, 8, dtype=torch.float16), f(1, 8), f(1, 8), f(3, dtype=i32))
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        pm.pm_grouped_gemm(f(2, 8, 8, dtype=torch.float64), f(1, 8), f(1, 8), f(3, dtype=i32))
    with pytest.raises(ValueError, match="uint8"):
        pm.pm_grouped_gemm_w4(f(2, 8, 8), f(2), None, 32, f(1, 16), f(1, 8), f(3, dtype=i32))
    with pytest.raises(ValueError, match="device"):
        pm.pm_combine_uses(f(4, 8), f(2, 2), f(2, 8))
    with pytest.raises(ValueError, match="2-D"):
        pm.pm_combine_uses(f(4, 8), f(4), f(2, 8))
    with pytest.raises(ValueError, match="contiguous"):
        pm.pm_encode_w4_device(f(8, 64).t(), 32, f(8), f(8))


@pytest.mark.parametrize("call", [gemm, w4])
def test_grouped_outputs_over_other_inputs_are_refused(call):
    """y in the offsets, the order or the weights would change them under the
    running call."""
    near = D + 8 * 64 * 4 - 4                        # the last element of y
    for kw in ({"r": rows(off=D)}, {"r": rows(off=near, order=None)}, {"r": rows(order=D + 16)},
               {"y": OFF}, {"y": ORD + 28, "r": rows()}, {"y": OFF + 16}, {"y": ORD - 64}):
        refused(call(yt=pm.PM_F32, **kw), pm.PM_ERR_ARG, "offsets or the order")


def test_grouped_outputs_over_weights_are_refused():
    E, R, C, G = 4, 64, 128, 32
    last = A + E * R * C * 2 - 2
    refused(gemm(y=A), pm.PM_ERR_ARG, "overlaps the weights")
    refused(gemm(y=last), pm.PM_ERR_ARG, "overlaps the weights")
    S, Z = A + (1 << 34), A + (2 << 34)
    for y in (A, A + E * R * C // 2 - 4, S, S + E * R * (C // G) * 2 - 4, Z,
              Z + E * R * (C // G) - 4):
        refused(w4(y=y, sc=S, z=Z), pm.PM_ERR_ARG, "overlaps the codes")


ROUTED_SOURCES = [s for s in build.TARGETS[0][1] if "pm_rout" in s or "pm_grouped" in s or
                  s.endswith("pm_combine.hip")]


def test_entry_points_have_nothing_that_throws(tmp_path):
    """The host code of the operators neither allocates nor locks: no C++
    exception can leave a C entry point."""
    assert len(ROUTED_SOURCES) == 9

    def undefined(src):
        obj = tmp_path / (os.path.basename(src) + ".o")
        subprocess.run([build.hipcc(), *build.COMPILE_FLAGS, "--cuda-host-only", "-x", "hip", "-c",
                        src, "-o", str(obj)], check=True, capture_output=True)
        return subprocess.run(["nm", "-u", str(obj)], check=True, capture_output=True,
                              text=True).stdout
    with concurrent.futures.ThreadPoolExecutor(4) as ex:
        for src, names in zip(ROUTED_SOURCES, ex.map(undefined, ROUTED_SOURCES)):
            assert "hipLaunchKernel" in names or src.endswith(("pm_routed.cpp", "pm_grouped.hip"))
            for bad in ("_Znw", "_Zna", "__cxa_throw", "__cxa_allocate_exception", "_ZSt", "malloc",
                        "pthread_mutex"):
                assert bad not in names, (src, bad, names)
