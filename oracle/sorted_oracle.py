"""64-bit definitions of the operators that sort a batch by expert, bring it
back and run its products in 8-bit integers (plain NumPy, from the formulas in
include/moe.h)."""
from __future__ import annotations

import numpy as np

from .moe_oracle import fl32, round_bf16

__all__ = ["sort_slots", "combine_rows", "combine_rows_grads", "quant_int8", "int8_product", "int8_grouped_product"]


def sort_slots(topk_ids, E: int):
    """(offsets [E+1], inv [T, k], token [offsets[E]]): where each slot goes and
    which token each sorted row is, slot by slot."""
    ids = np.asarray(topk_ids)
    flat = ids.reshape(-1)
    lists = [[] for _ in range(E)]
    for f, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(f)
    offsets = np.zeros(E + 1, dtype=np.int32)
    offsets[1:] = np.cumsum([len(x) for x in lists])
    order = [f for x in lists for f in x]
    inv = np.full(flat.shape, -1, dtype=np.int32)
    for p, f in enumerate(order):
        inv[f] = p
    return offsets, inv.reshape(ids.shape), np.array(order, dtype=np.int64) // max(ids.shape[1], 1)


def combine_rows(rows, inv, weights=None):
    """(sum, sum of magnitudes) over a token's slots of weight * row, unrounded."""
    T, k = inv.shape
    out = np.zeros((T, rows.shape[1]))
    size = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            if 0 <= inv[t, j] < rows.shape[0]:
                v = (1.0 if weights is None else float(weights[t, j])) * rows[inv[t, j]]
                out[t] += v
                size[t] += np.abs(v)
    return out, size


def combine_rows_grads(grad_out, rows, inv, weights=None):
    """(grad_rows with NaN where no slot has a row, grad_weights, sums of the
    magnitudes behind grad_weights), unrounded."""
    T, k = inv.shape
    grad_rows = np.full(rows.shape, np.nan)
    grad_w, size = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = inv[t, j]
            if 0 <= r < rows.shape[0]:
                grad_rows[r] = (1.0 if weights is None else float(weights[t, j])) * grad_out[t]
                grad_w[t, j] = np.sum(grad_out[t] * rows[r])
                size[t, j] = np.sum(np.abs(grad_out[t] * rows[r]))
    return grad_rows, grad_w, size


def quant_int8(x):
    """(codes int8, scales fp64) of rows given in fp64: fp32 quotients rounded
    once, and the nearest whole number of the exact product, ties to even."""
    most = np.maximum(np.abs(x).max(axis=1), float(np.float32(1e-10)))
    scale, inverse = fl32(most / 127.0), fl32(127.0 / most)
    # a value has 8 significant bits and the inverse 24: the product is exact
    return np.rint(x * inverse[:, None]).astype(np.int8), scale


def int8_product(a, a_scale, w, w_scale):
    """bf16(fl32(fl32(S) a_scale) w_scale) with S exact."""
    S = (a.astype(np.int64) @ w.astype(np.int64).T).astype(np.float64)
    with np.errstate(all="ignore"):
        v = fl32(S) * np.asarray(a_scale, dtype=np.float64)[:, None]
        return round_bf16(fl32(fl32(v) * np.asarray(w_scale, dtype=np.float64)[None, :]))


def int8_grouped_product(a, a_scale, w, w_scale, offsets):
    """The same with w[e] for rows offsets[e] .. offsets[e+1]; NaN outside."""
    out = np.full((a.shape[0], w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            out[lo:hi] = int8_product(a[lo:hi], a_scale[lo:hi], w[e], w_scale[e])
    return out
