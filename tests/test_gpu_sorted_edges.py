"""Rows sorted by expert on the GPU where the forms end: values that are no
numbers, the form with scratch replayed, on two streams and with a caller's
scratch, and launches that a size cuts in two."""
import numpy as np
import pytest
import torch

import oracle as O
from moe_layer_amd import ops

from gpu_util import dev

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def special_rows(T, cols, seed):
    """bf16 rows whose 128-column groups hold, in turn: numbers, zeros, values under
    the scale's floor, the largest numbers, an infinity, a NaN of either sign and of
    the smallest and the largest bits, both, NaN alone, and negative zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, cols // 128, 128, generator=g).bfloat16()
    bits = x.view(torch.int16)
    for i in range(T * (cols // 128)):
        t, b, at = i // (cols // 128), i % (cols // 128), (37 * i) % 128
        kind = i % 13
        if kind == 1:
            x[t, b] = 0.0
        elif kind == 2:
            x[t, b] *= 2.0 ** -60
        elif kind == 3:
            x[t, b] = torch.where(x[t, b] > 0, 3.3e38, -3.3e38).bfloat16()
        elif kind in (4, 5):
            x[t, b, at] = INF if kind == 4 else -INF
        elif kind in (6, 7, 8, 9):
            bits[t, b, at] = (0x7fc0, 0xffc0 - 0x10000, 0x7f81, 0xffff - 0x10000)[kind - 6]
        elif kind == 10:
            x[t, b, at], x[t, b, (at + 64) % 128] = INF, NAN
        elif kind == 11:
            x[t, b] = NAN
        elif kind == 12:
            x[t, b], x[t, b, at] = -0.0, 2.0 ** -130
    return x.view(T, cols)


@pytest.mark.parametrize("T,k,cols", [
    (1, 8, 7168), (40, 3, 1664),              # every workgroup compares the ids
    (2600, 2, 128), (2600, 3, 512), (1700, 8, 1664), (1100, 4, 20480),   # tokens share a workgroup
    (52000, 1, 128), (26000, 2, 640), (7000, 8, 2048)])                  # counted
def test_sort_to_fp8_is_moe_quant_act_whatever_the_values(T, k, cols):
    """Codes and scales bit for bit, in every form of the sort.  A signaling NaN is
    taken for a quiet one: moe_quant_act's fmaxf of one is a NaN, which drops the
    columns before it from the maximum, so what that makes is a matter of its order."""
    d, E = dev(), 5
    x = special_rows(min(T, 300), cols, T).repeat(-(-T // 300), 1)[:T].contiguous().to(d)
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(k), dtype=torch.int32).to(d)
    quiet = torch.where(x.isnan(), x.view(torch.int16) | 0x40, x.view(torch.int16)).view(torch.bfloat16)
    codes, scales = ops.moe_quant_act(quiet)
    rows, row_scales, _, inv = ops.moe_sort_rows(x, ids, E, quant="fp8")
    for j in range(k):
        at = inv[:, j].long()
        assert torch.equal(rows[at], codes)
        assert torch.equal(row_scales[at].view(torch.int32), scales.view(torch.int32))
