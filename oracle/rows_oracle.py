"""fp64 definitions of the operators around the fused layer: RMSNorm with the
residual's addition, the SiLU-gated multiply, and the dense and grouped
products (plain NumPy, from the formulas in include/moe.h)."""
from __future__ import annotations

import numpy as np

from .moe_oracle import dequant_block, e4m3_decode, fl32, round_bf16

__all__ = ["rmsnorm", "silu_mul", "act_values", "block_values", "grouped_product"]


def rmsnorm(x, residual, weight, eps: float):
    """(y, residual_out) of bf16 values given in fp64; y rounded to fp32 and
    then bf16, residual_out None without a residual."""
    x = np.asarray(x, dtype=np.float64)
    s = x if residual is None else fl32(x + np.asarray(residual, dtype=np.float64))
    inv = 1.0 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + float(np.float32(eps)))
    with np.errstate(invalid="ignore"):
        y = round_bf16(fl32(s * inv * np.asarray(weight, dtype=np.float64)[None, :]))
    return y, None if residual is None else round_bf16(s)


def silu_mul(h, clamp_limit: float = 0.0):
    """bf16(bf16(silu(gate)) * up) of h = [gate | up], after the clamp."""
    h = np.asarray(h, dtype=np.float64)
    cols = h.shape[1] // 2
    g, u = h[:, :cols], h[:, cols:]
    if clamp_limit > 0:
        g = np.minimum(g, clamp_limit)
        u = np.clip(u, -clamp_limit, clamp_limit)
    with np.errstate(over="ignore"):
        s = round_bf16(g / (1.0 + np.exp(-g)))
    return round_bf16(s * u)


def act_values(codes, scales, group: int = 128):
    """Quantised rows as their values: e4m3(code) * scale of its group."""
    return e4m3_decode(codes) * np.repeat(np.asarray(scales, dtype=np.float64), group, axis=-1)


def block_values(codes, scales):
    """Block-scaled weights [.., N, K] as their values, N not necessarily a
    multiple of 128 (the last row of blocks is cut)."""
    n = codes.shape[-2]
    pad = [(0, 0)] * (codes.ndim - 2) + [(0, -n % 128), (0, 0)]
    return dequant_block(np.pad(codes, pad), scales)[..., :n, :]


def grouped_product(a, w, offsets):
    """[rows, N] products of rows offsets[e] .. offsets[e+1] with w[e]; NaN on
    rows outside every group."""
    out = np.full((a.shape[0], w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            out[lo:hi] = a[lo:hi] @ w[e].T
    return out
