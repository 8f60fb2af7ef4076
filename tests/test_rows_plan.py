"""moe_gemm_plan on the host, and that the GPU tests' list of kernels has one
case for each that ordinary sizes reach."""
import ctypes as C
import math
import random

import pytest

from moe_layer_amd import ops

from rows_plan_cases import KERNELS, planned

BF16, FP8 = ops.MOE_WDTYPE_BF16, ops.MOE_WDTYPE_FP8_E4M3
OK, BAD, NOT = ops.MOE_OK, ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_each_case_takes_its_kernel(kernel):
    assert planned(ops, kernel[0], *KERNELS[kernel]) == kernel


def test_sizes_at_large_reach_no_other_kernel():
    rng = random.Random(3)

    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    missing = {}
    for _ in range(60000):
        fp8 = rng.random() < 0.5
        E = 0 if fp8 and rng.random() < 0.4 else rng.choice([1, 2, 4, 8, 16, 32, 64, 100, 128, 256, 512, 1024])
        rows, N = spread(1, 200000), spread(1, 200000)
        K = 128 * spread(1, 160) if fp8 else 64 * spread(1, 320)
        kernel = planned(ops, fp8, rows, E, N, K)
        if kernel not in KERNELS:
            missing[kernel] = (rows, E, N, K)
    assert not missing


def test_a_plan_depends_on_its_sizes_alone():
    a = ops.moe_gemm_plan(8192, 4096, 7168)
    ops.moe_gemm_plan(1, 16, 128, 4, BF16)
    assert ops.moe_gemm_plan(8192, 4096, 7168) == a


def plan(rows=4, E=3, N=256, K=256, wd=FP8, out=True):
    info = ops.GemmPlanInfo()
    return ops.lib().moe_gemm_plan(rows, E, N, K, wd, C.byref(info) if out else None)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(E=0), OK), (dict(E=1024), OK), (dict(wd=BF16, K=64), OK), (dict(rows=1 << 30, N=1 << 30), OK),
    (dict(rows=0), BAD), (dict(rows=-1), BAD), (dict(E=-1), BAD), (dict(E=1025), BAD), (dict(N=0), BAD),
    (dict(K=0), BAD), (dict(wd=3), BAD), (dict(wd=-1), BAD), (dict(out=False), BAD),
    (dict(wd=2), NOT), (dict(E=0, wd=BF16), NOT), (dict(K=192), NOT), (dict(K=96, wd=BF16), NOT),
    (dict(rows=(1 << 30) + 1), NOT), (dict(N=(1 << 30) + 1), NOT), (dict(K=(1 << 20) + 128), NOT),
])
def test_refusals(kw, status):
    assert plan(**kw) == status
