"""The sums of the dense and grouped products are 32-bit sums whatever the
operands' type.

Operands whose products are 2^8 or 2^-6: every 128-block of K holds two columns
of magnitude 16 on both sides, whose products cancel, and small values of
magnitude 2^-3 or 0 else.  A block's partial sums are at most 2 2^14 + 126 units
of 2^-6 and the cancelled blocks' at most 126, times scales of 1 to 4 in units
of the smallest: exact fp32 values in every order for K <= 2^16, so outputs are
compared bit for bit.  A dot product that keeps fewer bits below the largest of
its terms loses the small ones.
"""
import numpy as np
import pytest
import torch

import oracle as O
from moe_layer_amd import ops

from gpu_util import bf16_to_f64, dev, log
from test_gpu_rows import put, sizes_to_offsets

pytestmark = pytest.mark.gpu


def wide_operands(rng, rows, E, N, K, fp8):
    a = (rng.integers(-1, 2, (rows, K)) / 8).astype(np.float32)
    w = (rng.integers(-1, 2, (E, N, K)) / 8).astype(np.float32)
    sign = rng.choice([-16.0, 16.0], rows).astype(np.float32)
    for b in range(0, K, 128):
        plus, minus = b + rng.choice(min(128, K - b), 2, replace=False)
        a[:, plus] = a[:, minus] = sign
        w[:, :, plus], w[:, :, minus] = 16.0, -16.0
    at, wt = torch.from_numpy(a), torch.from_numpy(w)
    if not fp8:
        return at.bfloat16(), wt.bfloat16(), None, None, a.astype(np.float64), w.astype(np.float64)
    nb = -(-N // 128)
    sa = rng.choice([0.5, 1.0], (rows, K // 128)).astype(np.float32)
    sw = rng.choice([1.0, 2.0], (E, nb, K // 128)).astype(np.float32)
    ac, wc = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (at, wt))
    return (ac, wc, torch.from_numpy(sa), torch.from_numpy(sw), O.act_values(ac.numpy(), sa),
            O.block_values(wc.numpy(), sw))


# from one row to the largest tiles
@pytest.mark.parametrize("M,N,K", [(1, 40, 128), (1, 4096, 2048), (9, 300, 512), (40, 1000, 2048), (64, 7168, 512),
                                   (129, 255, 384), (300, 520, 2304), (520, 2000, 640), (770, 4741, 128),
                                   (1500, 2001, 1152), (2300, 4100, 512)])
def test_gemm_fp8(M, N, K):
    rng = np.random.default_rng(M + N + K)
    a, w, sa, sw, av, wv = wide_operands(rng, M, 1, N, K, True)
    out = ops.moe_gemm_fp8(*put(a, sa, w[0], sw[0]))
    np.testing.assert_array_equal(bf16_to_f64(out), O.round_bf16(av @ wv[0].T))


@pytest.mark.parametrize("sizes,N,K", [([5, 0, 1, 18], 130, 256), ([1] * 90, 256, 1024), ([64, 1, 0, 65, 129], 257, 384),
                                       ([300, 0, 7, 511], 640, 256), ([600, 500, 90], 1536, 512),
                                       ([2048 + 65, 1024 + 129, 0, 1, 768 + 64], 2601, 256)])
@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_gemm(sizes, N, K, fp8):
    rng = np.random.default_rng(sum(sizes) + N + K)
    a, w, sa, sw, av, wv = wide_operands(rng, sum(sizes), len(sizes), N, K, fp8)
    off = sizes_to_offsets(sizes)
    out = ops.moe_grouped_gemm(*put(a, w, torch.from_numpy(off), sa, sw))
    np.testing.assert_array_equal(bf16_to_f64(out), O.round_bf16(O.grouped_product(av, wv, off)))


@pytest.mark.parametrize("M,N,K", [(1, 40, 256), (40, 300, 256), (300, 520, 384), (1500, 2001, 256)])
@pytest.mark.parametrize("low", [True, False])
def test_scale_products_at_the_ends_of_the_range(M, N, K, low):
    """a_scale w_scale = 2^-126 and 2^127, the smallest and largest powers of two
    that are normal fp32 values, and zero scales.  Sums of values -1, 0, 1 times
    2^-9 (low: 1), below 2^11 of their unit, are exact."""
    rng = np.random.default_rng(M + K)
    unit = 1.0 if low else 2.0 ** -9
    a, w = (rng.integers(-1, 2, s).astype(np.float32) for s in ((M, K), (N, K)))
    ac, wc = (torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8) for v in (a * np.float32(unit), w))
    sa = np.full((M, K // 128), 2.0 ** (-100 if low else 100), np.float32)
    sa[M // 2] = 0.0
    sw = np.full((-(-N // 128), K // 128), 2.0 ** (-26 if low else 27), np.float32)
    ref = O.act_values(ac.numpy(), sa) @ O.block_values(wc.numpy(), sw).T
    args = put(ac, torch.from_numpy(sa), wc, torch.from_numpy(sw))
    np.testing.assert_array_equal(bf16_to_f64(ops.moe_gemm_fp8(*args)), O.round_bf16(ref))
    off = torch.tensor([0, M // 3, M], dtype=torch.int32, device=dev())
    two = [args[2].expand(2, -1, -1).contiguous(), args[3].expand(2, -1, -1).contiguous()]
    out = ops.moe_grouped_gemm(args[0], two[0], off, args[1], two[1])
    np.testing.assert_array_equal(bf16_to_f64(out), O.round_bf16(ref))


@pytest.mark.parametrize("rows,E,N,K,fp8", [(3, 0, 40, 2 ** 20, True), (300, 0, 260, 2 ** 16, True), (70, 0, 130, 2 ** 17 + 128, True),
                                            (40, 3, 70, 2 ** 18, True), (20, 1, 40, 2 ** 18, False),
                                            (520, 2, 300, 2 ** 15 + 64, False), (9, 2, 33, 2 ** 20, False)])
def test_long_sums_are_complete(rows, E, N, K, fp8):
    """One product of magnitude 1 for every 128 of K, at a place that moves
    through the block, so that a lost step changes every output by 1; most sums,
    of up to 2^13 random signs, stay below 256, where bf16 shows a difference of 1."""
    rng = np.random.default_rng(K + rows)
    groups = max(E, 1)
    a = np.zeros((rows, K), np.float32)
    w = rng.choice([-1.0, 1.0], (groups, N, K)).astype(np.float32)
    steps = -(-K // 128)
    for r in range(rows):
        at = 128 * np.arange(steps) + (37 * np.arange(steps) + 11 * r) % 128
        at[0], at[-1] = 0, K - 1                            # the first and the last of K
        a[r, at] = rng.choice([-1.0, 1.0], steps)
    off = sizes_to_offsets(rng.multinomial(rows, [1 / groups] * groups))
    ref = O.grouped_product(a.astype(np.float64), w.astype(np.float64), off)
    assert (np.abs(ref) < 256).mean() > 0.9
    at, wt = torch.from_numpy(a), torch.from_numpy(w)
    if not fp8:
        out = ops.moe_grouped_gemm(*put(at.bfloat16(), wt.bfloat16(), torch.from_numpy(off)))
    else:
        ac, wc = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (at, wt))
        sa, sw = torch.ones(rows, K // 128), torch.ones(groups, -(-N // 128), K // 128)
        if E == 0:
            out = ops.moe_gemm_fp8(*put(ac, sa, wc[0], sw[0]))
        else:
            out = ops.moe_grouped_gemm(*put(ac, wc, torch.from_numpy(off), sa, sw))
    np.testing.assert_array_equal(bf16_to_f64(out), O.round_bf16(ref))


@pytest.mark.parametrize("grouped", [False, True])
def test_codes_behind_a_product(grouped):
    """The codes that moe_silu_mul makes of a gate/up product are those of its
    64-bit sum, but for values next to a rounding border.  A 32-bit sum of 4096
    random products is off by about 2^-25 sqrt(128) = 3e-7 of itself, so about
    3e-7 / 2^-8 = 1e-4 of the bf16 gate and up values round the other way, and one
    in 16 of those moves a 4-bit code: 1e-5 of the codes.  20 times that is
    allowed (a sum that loses 2^-14 of its largest products flips 2e-3 of them)."""
    rng = np.random.default_rng(41)
    rows, E, K, I = 128, 2, 4096, 512
    a = (rng.standard_normal((rows, K)) * 60).clip(-448, 448).astype(np.float32)
    w = (rng.standard_normal((E, 2 * I, K)) * 60).clip(-448, 448).astype(np.float32)
    ac, wc = (torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8) for v in (a, w))
    sa = (2.0 ** rng.integers(-9, -6, (rows, K // 128))).astype(np.float32)
    sw = (1e-4 * (1 + rng.random((E, 2 * I // 128, K // 128)))).astype(np.float32)
    av, wv = O.act_values(ac.numpy(), sa), O.block_values(wc.numpy(), sw)
    if grouped:
        off = np.array([0, 50, rows], np.int32)
        ref = O.grouped_product(av, wv, off)
        h = ops.moe_grouped_gemm(*put(ac, wc, torch.from_numpy(off), torch.from_numpy(sa), torch.from_numpy(sw)))
    else:
        ref = av @ wv[0].T
        h = ops.moe_gemm_fp8(*put(ac, torch.from_numpy(sa), wc[0], torch.from_numpy(sw[0])))
    _, codes, _ = ops.moe_silu_mul(h, quant="fp8")
    want, _, _ = O.quant_act(O.silu_mul(O.round_bf16(O.fl32(ref))))
    off_by = int((codes.cpu().numpy() != want).sum())
    log(f"codes behind a product: {off_by} of {want.size} differ")
    assert off_by <= 2e-4 * want.size
