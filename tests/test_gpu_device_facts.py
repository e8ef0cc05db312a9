"""What the kernels assume of the hardware, tried on it: the error of the scored
router's fp32 sigmoid over every logit, and the sums of the 8-bit matrix
instruction over random groups of products."""
import ctypes
import os

import pytest
import torch

import fp8_cases as fc
import routed_cases as rc
from test_gpu_fp8 import report

pytestmark = pytest.mark.gpu
LIB = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "libpmfacts.so")


@pytest.fixture(scope="module")
def facts():
    lib = ctypes.CDLL(LIB)
    P = ctypes.c_void_p
    lib.facts_sigmoid.argtypes = [P, P]
    lib.facts_products.argtypes = [ctypes.c_int, P, P, P, P]
    return lib


def test_sigmoid_of_every_logit(facts):
    """The constants of pm_rank.h: 2^-23, and 1.125 * 2^-18 of the sigmoid itself
    where that is 2^-125 or more.  (Below 2^-126 the reciprocal gives 0, all of it;
    the router allows for 2^-125 there.)"""
    report("fp32 sigmoid over all logits")
    out = torch.full((1 << 18, 2), float("nan"), dtype=torch.float64, device="cuda")
    torch.cuda.synchronize()
    assert facts.facts_sigmoid(out.data_ptr(), None) == 0
    torch.cuda.synchronize()
    error, relative = out.max(0).values.tolist()
    assert error <= 2.0 ** -23 and relative <= 1.125 * 2.0 ** -18, (error, relative)


def exponent(q):
    return torch.frexp(q.double().abs().clamp(min=2.0 ** -6))[1].double() - 1.0


@pytest.mark.parametrize("seed", range(8))
def test_sums_of_eight_products(facts, seed):
    """Products of 8 random codes in each row, of all exponents: each is cut off
    towards 0 at 2^-13 of the largest power of two of two codes (no less than
    2^-6 each) whose product is not 0, and their sum is exact."""
    report(f"sums of eight products, seed {seed}")
    n, g = 1024, rc.gen(seed)

    def codes():
        q = torch.randint(0, 256, (n, 16, 8), dtype=torch.uint8, device="cuda", generator=g)
        full = torch.zeros(n, 16, 128, dtype=torch.uint8, device="cuda")
        at = 8 * (seed * 5 % 16)
        full[:, :, at:at + 8] = torch.where((q & 127) == 127, 0, q)
        return full, full[:, :, at:at + 8].contiguous().view(fc.F8)

    (a, a8), (b, b8) = codes(), codes()
    d = torch.full((n, 16, 16), float("nan"), device="cuda")
    torch.cuda.synchronize()
    assert facts.facts_products(n, a.data_ptr(), b.data_ptr(), d.data_ptr(), None) == 0
    torch.cuda.synchronize()
    p = a8.double()[:, :, None] * b8.double()[:, None]
    e = (exponent(a8)[:, :, None] + exponent(b8)[:, None]).masked_fill(p == 0, -99.0)
    unit = torch.exp2(e.amax(-1, keepdim=True) - 13.0)
    assert torch.equal(d.double(), (torch.trunc(p / unit) * unit).sum(-1))
