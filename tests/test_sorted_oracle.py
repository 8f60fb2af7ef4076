"""Pins of oracle/sorted_oracle.py: hand examples, other formulations, and
differences for the gradients."""
import numpy as np
import torch

import oracle as O


def test_sort_slots_by_hand():
    ids = np.array([[2, 0], [0, 5], [2, 2], [-1, 0]])
    offsets, inv, token = O.sort_slots(ids, 3)
    assert offsets.tolist() == [0, 3, 3, 6]
    assert inv.tolist() == [[3, 0], [1, -1], [4, 5], [-1, 2]]
    assert token.tolist() == [0, 1, 3, 0, 2, 2]


def test_sort_slots_is_moe_aligns_order():
    """Blocks of one row have no padding: moe_align's oracle sorts the same way."""
    rng = np.random.default_rng(1)
    ids = rng.integers(-1, 9, (57, 5))
    offsets, inv, token = O.sort_slots(ids, 8)
    al = O.align(ids.astype(np.int32), 8, 1)
    order, experts, inverse = al["sorted_token_ids"], al["expert_ids"], al["inv"]
    total = int(np.ravel(al["num_tokens_post_padded"])[0])
    assert total == offsets[-1]
    np.testing.assert_array_equal(np.asarray(order)[:total] // 5, token)
    np.testing.assert_array_equal(np.asarray(inverse).reshape(57, 5), inv)
    np.testing.assert_array_equal(np.bincount(np.asarray(experts)[:total], minlength=8), np.diff(offsets))


def test_combine_rows_is_a_product_with_the_routing_matrix():
    rng = np.random.default_rng(2)
    T, k, n, H = 9, 3, 20, 5
    inv = rng.permutation(40)[: T * k].reshape(T, k).astype(np.int32)
    inv[inv >= n] = -1
    rows, w = rng.normal(size=(n, H)), rng.normal(size=(T, k))
    G = np.zeros((T, n))
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                G[t, inv[t, j]] += w[t, j]
    out, size = O.combine_rows(rows, inv, w)
    np.testing.assert_allclose(out, G @ rows, atol=1e-12)
    np.testing.assert_allclose(size, np.abs(G) @ np.abs(rows), atol=1e-12)


def test_gradients_are_the_differences():
    """Central differences of <grad_out, combine(rows, w)>, which is linear in
    each of rows and w: exact but for rounding."""
    rng = np.random.default_rng(3)
    T, k, n, H = 4, 2, 9, 3
    inv = np.array([[0, 5], [7, -1], [2, 8], [-1, -1]], dtype=np.int32)
    rows, w, g = rng.normal(size=(n, H)), rng.normal(size=(T, k)), rng.normal(size=(T, H))
    d_rows, d_w, _ = O.combine_rows_grads(g, rows, inv, w)
    for t in range(T):
        for j in range(k):
            up, down = w.copy(), w.copy()
            up[t, j] += 0.5
            down[t, j] -= 0.5
            diff = np.sum(g * (O.combine_rows(rows, inv, up)[0] - O.combine_rows(rows, inv, down)[0]))
            assert abs(diff - d_w[t, j]) < 1e-12
    for r in range(n):
        for h in range(H):
            up, down = rows.copy(), rows.copy()
            up[r, h] += 0.5
            down[r, h] -= 0.5
            diff = np.sum(g * (O.combine_rows(up, inv, w)[0] - O.combine_rows(down, inv, w)[0]))
            assert abs(diff - (0.0 if r in (1, 3, 4, 6) else d_rows[r, h])) < 1e-12
            assert np.isnan(d_rows[r, h]) == (r in (1, 3, 4, 6))


def test_quant_int8_by_hand():
    """127 / 1 is whole: codes are 127 x.  Half-way codes go to even, the largest
    magnitude to 127, a row of zeros to zeros."""
    x = np.array([[1.0, -1.0, 0.5, -0.25, 0.0], [0.0] * 5, [254.0, 1.0, -3.0, 5.0, -254.0], [2.0 ** -120] * 5])
    codes, scales = O.quant_int8(x)
    assert codes[0].tolist() == [127, -127, 64, -32, 0]
    assert codes[1].tolist() == [0] * 5
    assert codes[2].tolist() == [127, 0, -2, 2, -127]      # 0.5, 1.5 and 2.5 to even
    assert codes[3].tolist() == [0] * 5                    # far below the floor of the scale
    assert scales[2] == 2.0 and scales[0] == float(np.float32(1 / 127))


def test_quant_int8_every_magnitude():
    """The largest value of a row is code 127 for every bf16 magnitude from the
    floor on, so no code leaves [-127, 127]; the scale is within half a step."""
    bits = np.arange(0x80, 0x7F80, dtype=np.uint32) << 16
    v = bits.view(np.float32).astype(np.float64)
    v = v[v >= 1e-10]
    codes, scales = O.quant_int8(np.stack([v, -v], 1))
    assert (codes[:, 0] == 127).all() and (codes[:, 1] == -127).all()
    assert (np.abs(scales * 127 - v) <= 2.0 ** -24 * v * (1 + 2.0 ** -20)).all()


def test_int8_products_against_torch():
    rng = np.random.default_rng(5)
    a, w = rng.integers(-128, 128, (7, 48)).astype(np.int8), rng.integers(-128, 128, (5, 48)).astype(np.int8)
    sa, sw = rng.random(7).astype(np.float32), rng.random(5).astype(np.float32)
    S = torch.from_numpy(a).int() @ torch.from_numpy(w).int().t()
    want = (S.float() * torch.from_numpy(sa)[:, None] * torch.from_numpy(sw)).bfloat16()
    np.testing.assert_array_equal(O.int8_product(a, sa, w, sw), want.double().numpy())
    g = O.int8_grouped_product(a, sa, np.stack([w, w[::-1]]), np.stack([sw, sw[::-1]]), [1, 4, 6])
    assert np.isnan(g[[0, 6]]).all()
    np.testing.assert_array_equal(g[1:4], want.double().numpy()[1:4])
    np.testing.assert_array_equal(g[4:6], want.double().numpy()[4:6, ::-1])
