"""NaN and infinities through the SiLU-gated multiply: what the definition
gives, with and without the clamp, in every position of gate and up."""
import numpy as np
import pytest
import torch

import oracle as O
from moe_layer_amd import ops

from gpu_util import bf16_to_f64, dev

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("limit", [0.0, 2.5])
def test_silu_mul_special_values(limit):
    special = [NAN, -NAN, INF, -INF, 0.0, -0.0, 1.0, -3.0, 1e30, -1e30]
    pairs = [(g, u) for g in special for u in special]
    h = torch.full((len(pairs), 2 * 8), 0.5)
    for i, (g, u) in enumerate(pairs):
        h[i, i % 8], h[i, 8 + i % 8] = g, u
    h = h.bfloat16()
    y, _, _ = ops.moe_silu_mul(h.to(dev()), clamp_limit=limit)
    # -inf's SiLU is its limit, -0 (the formula's inf / inf)
    f = bf16_to_f64(h)
    with np.errstate(invalid="ignore", over="ignore"):
        want = O.silu_mul(np.where(np.isneginf(f) & (np.arange(16) < 8), -1e30, f), limit)
    np.testing.assert_array_equal(bf16_to_f64(y), want)


@pytest.mark.parametrize("quant", ["fp8", "mxfp8"])
@pytest.mark.parametrize("limit", [0.0, 2.5])
@pytest.mark.parametrize("half", [0, 1])
def test_silu_mul_codes_keep_a_nan(quant, limit, half):
    """A NaN of gate or up is a NaN code, and other groups are as without it."""
    g = torch.Generator().manual_seed(5)
    rows, cols, group = 4, 256, 128 if quant == "fp8" else 32
    h = (2 * torch.randn(rows, 2 * cols, generator=g)).bfloat16().to(dev())
    _, clean, scales = ops.moe_silu_mul(h, quant=quant, clamp_limit=limit)
    bad = h.clone()
    bad[2, half * cols + 70] = NAN
    _, codes, s2 = ops.moe_silu_mul(bad, quant=quant, clamp_limit=limit)
    assert int(codes[2, 70]) & 0x7f == 0x7f                # E4M3FN's NaN
    keep = torch.ones(rows, cols, dtype=torch.bool, device=dev())
    keep[2, 70 // group * group: 70 // group * group + group] = False
    assert torch.equal(codes[keep], clean[keep])
    assert torch.equal(s2.flatten()[keep[:, ::group].flatten()], scales.flatten()[keep[:, ::group].flatten()])
