"""Pins of the 64-bit definitions of the operators around the layer, by hand
and against torch's own functions on the CPU."""
import numpy as np
import pytest
import torch

import oracle as O


def test_rmsnorm_by_hand():
    # s = (3, 4): mean square 12.5; weight (1, 2), eps 0
    y, res = O.rmsnorm([[1.0, 1.5]], [[2.0, 2.5]], [1.0, 2.0], 0.0)
    np.testing.assert_array_equal(res, [[3.0, 4.0]])
    np.testing.assert_array_equal(y, O.round_bf16(O.fl32(np.array([[3.0, 8.0]]) / np.sqrt(12.5))))
    y, res = O.rmsnorm([[0.0, 0.0]], None, [1.0, 1.0], 1e-6)
    assert res is None and not y.any()


def test_rmsnorm_matches_torch():
    g = torch.Generator().manual_seed(3)
    x, r = (torch.randn(5, 96, generator=g, dtype=torch.float64).bfloat16().double() for _ in range(2))
    w = torch.randn(96, generator=g, dtype=torch.float64).bfloat16().double()
    ref = torch.nn.functional.rms_norm(x + r, (96,), w, eps=float(np.float32(1e-5))).numpy()
    y, res = O.rmsnorm(x.numpy(), r.numpy(), w.numpy(), 1e-5)
    # two roundings, fp32 and bf16: 2^-24 + 2^-8 of the value (and s rounded to fp32, 2^-24)
    assert np.all(np.abs(y - ref) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ref))
    assert np.all(np.abs(res - (x + r).numpy()) <= (2.0 ** -8 + 2.0 ** -24) * np.abs((x + r).numpy()))


def test_silu_mul_by_hand_and_torch():
    np.testing.assert_array_equal(O.silu_mul([[1.0, 0.0, 2.0, 5.0]]), [[1.4609375, 0.0]])
    # the clamp caps the gate above and the up value on both sides
    a = O.silu_mul([[10.0, -10.0, 20.0, -20.0]], 7.0)
    s = O.round_bf16(np.array([7.0, -10.0]) / (1 + np.exp([-7.0, 10.0])))
    np.testing.assert_array_equal(a, O.round_bf16(s * [7.0, -7.0])[None])
    g = torch.Generator().manual_seed(4)
    h = torch.randn(7, 64, generator=g, dtype=torch.float64).bfloat16().double()
    ref = (torch.nn.functional.silu(h[:, :32]) * h[:, 32:]).numpy()
    got = O.silu_mul(h.numpy())
    assert np.all(np.abs(got - ref) <= (2 * 2.0 ** -8 + 2.0 ** -16) * np.abs(ref) + 2.0 ** -133)


@pytest.mark.parametrize("n", [1, 128, 200])
def test_values_by_loop(n):
    rng = np.random.default_rng(n)
    codes = rng.integers(0, 127, (n, 256)).astype(np.uint8)
    blocks = rng.random((-(-n // 128), 2)).astype(np.float32)
    v = O.block_values(codes, blocks)
    rows = rng.random((n, 2)).astype(np.float32)
    a = O.act_values(codes, rows)
    dec = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    for i in range(n):
        for k in (0, 127, 128, 255):
            assert v[i, k] == dec[i, k] * float(blocks[i // 128, k // 128])
            assert a[i, k] == dec[i, k] * float(rows[i, k // 128])


def test_grouped_product_rows_outside_groups():
    a, w = np.arange(8.0).reshape(4, 2), np.ones((3, 1, 2))
    out = O.grouped_product(a, w, [1, 1, 3, 3])
    assert np.isnan(out[0]) and np.isnan(out[3])
    np.testing.assert_array_equal(out[1:3, 0], [5.0, 9.0])
