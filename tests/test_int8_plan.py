"""The GPU tests' list of int8 kernels has one case for each that ordinary
sizes reach (host only)."""
import math
import random

import pytest

from moe_layer_amd import ops

from int8_plan_cases import KERNELS, planned


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_each_case_takes_its_kernel(kernel):
    assert planned(ops, *KERNELS[kernel]) == kernel


def test_sizes_at_large_reach_no_other_kernel():
    rng = random.Random(4)

    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    missing = {}
    for _ in range(60000):
        E = rng.choice([0, 0, 0, 1, 2, 4, 8, 16, 32, 64, 100, 128, 256, 512, 1024])
        rows, N, K = spread(1, 200000), spread(1, 200000), 16 * spread(1, 2048)
        kernel = planned(ops, rows, E, N, K)
        if kernel not in KERNELS:
            missing[kernel] = (rows, E, N, K)
    assert not missing


def test_the_other_types_take_one_workgroup_a_cu():
    """moe_gemm_plan's answer 2 is for int8 alone."""
    rng = random.Random(5)
    for _ in range(5000):
        rows, N, K = rng.randint(1, 40000), rng.randint(1, 8000), 128 * rng.randint(1, 16)
        for E, wd in ((0, ops.MOE_WDTYPE_FP8_E4M3), (64, ops.MOE_WDTYPE_FP8_E4M3), (64, ops.MOE_WDTYPE_BF16)):
            assert ops.moe_gemm_plan(rows, N, K, E, wd)["split"] in (0, 1)
