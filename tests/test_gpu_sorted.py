"""Rows sorted by expert and back on the GPU against their 64-bit definitions
(oracle/sorted_oracle.py).

Comparison rules, fixed before the first run
  * moe_sort_rows: bit for bit, quantised or not (every rounding is one
    rounding of an exact value).
  * moe_combine_rows, per output: 2^-8 |o| (half a step of bf16) and
    2^-24 (k + 1) S (one fp32 rounding per slot), S the sum of magnitudes, both
    times 1 + 2^-8 for the rounding of the rounded.
  * grad_rows: bit for bit the bf16 rounding of fl32(w g): a weight has 24 bits
    and a bf16 value 8, so the oracle rounds the exact product to fp32 and then
    to bf16, as the kernel does.
  * grad_weights: 2^-24 cols S, the worst order of an fp32 sum of cols products
    that are exact in fp32 (8 + 8 bits).
"""
import numpy as np
import pytest
import torch

import oracle as O
from moe_layer_amd import ops

from gpu_util import bf16_to_f64, dev

pytestmark = pytest.mark.gpu


def routing(rng, T, k, E, away=0.0, repeats=False, skew=0.0):
    """int32 ids [T, k]: without repeats in a token unless asked, a share of them
    outside [0, E) on either side."""
    load = np.exp(skew * rng.normal(size=E))
    if repeats or k > E:
        ids = rng.choice(E, (T, k), p=load / load.sum())
    else:
        ids = np.argsort(-(np.log(load) + rng.gumbel(size=(T, E))), axis=1)[:, :k]
    ids = ids.astype(np.int64)
    out = rng.random((T, k)) < away
    return np.where(out, rng.choice([-1, E, -2 ** 31, 2 ** 31 - 1, -7], (T, k)), ids).astype(np.int32)


def source(g, T, cols, kind):
    """(x, x_scale) of a type, x with rows of very different sizes."""
    x = (torch.randn(T, cols, generator=g) * torch.logspace(-3, 3, max(T, 1))[:T, None]).bfloat16()
    if kind == "bf16":
        return x, None
    if kind == "int8":
        return torch.randint(-128, 128, (T, cols), generator=g).to(torch.int8), torch.rand(T, generator=g)
    return (torch.randint(0, 256, (T, cols), generator=g).to(torch.uint8), torch.rand(T, cols // 128, generator=g))


def expected(x, x_scale, kind, quant):
    """(rows' source, scales' source) per token as NumPy arrays."""
    if quant == "int8":
        return O.quant_int8(bf16_to_f64(x))
    if quant == "fp8":
        c, s, _ = O.quant_act(bf16_to_f64(x), 128)
        return c, s
    return (x.view(torch.int16) if kind == "bf16" else x).numpy(), None if x_scale is None else x_scale.numpy()


def check_sort(T, k, E, cols, kind, quant, ids, seed):
    g, d = torch.Generator().manual_seed(seed), dev()
    x, x_scale = source(g, T, cols, kind)
    offsets, inv, token = O.sort_slots(ids, E)
    n = int(offsets[-1])
    xd, ids_d = x.to(d), torch.from_numpy(ids).to(d)
    sd = None if x_scale is None else x_scale.to(d)
    out = quant or kind
    dtype = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.uint8}[out]
    rows = torch.full((T * k, cols), 7, dtype=dtype, device=d)
    scales = None if out == "bf16" else torch.full((T * k,) if out == "int8" else (T * k, cols // 128), 7.0, device=d)
    got = ops.moe_sort_rows(xd, ids_d, E, x_scale=sd, quant=quant, rows=rows, scales=scales)
    assert got[0] is rows and got[1] is scales
    np.testing.assert_array_equal(got[2].cpu().numpy(), offsets)
    np.testing.assert_array_equal(got[3].cpu().numpy(), inv)
    want, want_s = expected(x, x_scale, kind, quant)
    have = (rows.view(torch.int16) if out == "bf16" else rows).cpu().numpy()
    np.testing.assert_array_equal(have[:n], want[token])
    assert (rows[n:] == 7).all(), "rows behind the last one were written"
    if scales is not None:
        np.testing.assert_array_equal(scales.cpu().numpy()[:n], want_s[token].astype(np.float32))
        assert (scales[n:] == 7).all()
    # allocated outputs, and codes as float8
    again = ops.moe_sort_rows(xd.view(torch.float8_e4m3fn) if kind == "fp8" else xd, ids_d, E, x_scale=sd, quant=quant)
    assert torch.equal(again[0][:n].view(torch.uint8), rows[:n].view(torch.uint8))
    assert torch.equal(again[2], got[2]) and torch.equal(again[3], got[3])


KINDS = [("bf16", None), ("bf16", "int8"), ("bf16", "fp8"), ("fp8", None), ("int8", None)]


@pytest.mark.parametrize("kind,quant", KINDS)
@pytest.mark.parametrize("T,k,E,cols", [
    (1, 1, 1, 128), (1, 8, 256, 7168), (2, 3, 5, 128), (7, 2, 4, 256), (33, 8, 8, 384), (64, 8, 128, 4096),
    (300, 6, 60, 640), (9, 64, 64, 128), (1, 64, 1024, 2176), (513, 4, 1000, 128), (1031, 8, 256, 512),
    (5000, 1, 3, 128), (4100, 5, 1024, 128)])
def test_sort_rows(T, k, E, cols, kind, quant):
    rng = np.random.default_rng(T * 31 + k)
    check_sort(T, k, E, cols, kind, quant, routing(rng, T, k, E, skew=1.0), T + cols)


@pytest.mark.parametrize("T", [50, 3000])
@pytest.mark.parametrize("away,repeats", [(0.4, False), (0.0, True), (0.5, True), (1.0, False)])
def test_sort_rows_unrouted_and_repeated(T, away, repeats):
    """Ids on either side of [0, E), all of them too; experts twice in a token."""
    rng = np.random.default_rng(T + int(8 * away))
    for kind, quant in KINDS:
        check_sort(T, 6, 7, 128, kind, quant, routing(rng, T, 6, 7, away, repeats), T)


@pytest.mark.parametrize("cols", [8, 16, 24, 1000, 2056, 4104, 16384, 40008])
def test_sort_rows_widths(cols):
    rng = np.random.default_rng(cols)
    for T in (3, 700):
        if T * cols > 1 << 22:
            continue
        check_sort(T, 4, 9, cols, "bf16", None, routing(rng, T, 4, 9), cols)
        if cols % 16 == 0 and cols <= ops.MOE_MAX_INT8_K:
            check_sort(T, 4, 9, cols, "bf16", "int8", routing(rng, T, 4, 9), cols)
            check_sort(T, 4, 9, cols, "int8", None, routing(rng, T, 4, 9), cols)


@pytest.mark.parametrize("cols", [2048, 2064, 4096, 8192, 8208, 16400, 32768])
def test_sort_rows_int8_of_every_row_size(cols):
    rng = np.random.default_rng(cols + 1)
    check_sort(5, 3, 4, cols, "bf16", "int8", routing(rng, 5, 3, 4), cols)


@pytest.mark.parametrize("kind,quant", KINDS)
@pytest.mark.parametrize("cols", [8448, 16640, 24576])
def test_sort_rows_long_rows_of_many_tokens(cols, kind, quant):
    """Rows longer than a wave holds, in a batch of more tokens than workgroups compare ids for."""
    rng = np.random.default_rng(cols)
    check_sort(1100, 4, 9, cols, kind, quant, routing(rng, 1100, 4, 9, away=0.3), cols)


@pytest.mark.parametrize("T,k", [(1619, 1), (1620, 1), (572, 8), (573, 8), (809, 4), (810, 4), (257, 64),
                                 (2051, 8), (4095, 7)])
def test_sort_rows_between_the_forms(T, k):
    """Batches around the size from which tokens share a workgroup, and of several tokens a wave."""
    rng = np.random.default_rng(T)
    check_sort(T, k, 33, 64, "bf16", "int8", routing(rng, T, k, 33, away=0.1), T)


# columns whose rows are up to 8, 16, 32, 64 and more pieces of 16 stored bytes
NARROW = {("bf16", None): (8, 64, 72, 256, 504, 512, 520), ("bf16", "int8"): (16, 128, 144, 400, 512, 528, 1024, 1040),
          ("bf16", "fp8"): (128, 256, 384, 512, 896, 1152), ("fp8", None): (128, 256, 384, 512, 1024, 1152),
          ("int8", None): (16, 128, 144, 256, 496, 1024, 1040)}


@pytest.mark.parametrize("kind,quant", KINDS)
@pytest.mark.parametrize("T,k", [(2501, 3), (6260, 4), (13001, 4), (17001, 3)])
def test_sort_rows_narrow(T, k, kind, quant):
    """Rows that a part of a wave takes, in the two forms for many ids; the last
    tokens leave lanes of a wave without one."""
    rng = np.random.default_rng(T + k)
    ids = routing(rng, T, k, 20, away=0.2)
    for cols in NARROW[kind, quant]:
        check_sort(T, k, 20, cols, kind, quant, ids, cols)


def test_sort_rows_ids_anywhere():
    """Ids that start at every 4-byte place of a 16-byte piece."""
    rng, d = np.random.default_rng(8), dev()
    for T, k in ((3, 3), (700, 5)):
        ids = routing(rng, T, k, 12, away=0.2)
        want_off, want_inv, _ = O.sort_slots(ids, 12)
        x = torch.randn(T, 64, device=d).bfloat16()
        for at in range(4):
            buf = torch.full((T * k + 8,), 5, dtype=torch.int32, device=d)
            view = buf[at: at + T * k].view(T, k)
            view.copy_(torch.from_numpy(ids))
            _, _, off, inv = ops.moe_sort_rows(x, view, 12)
            np.testing.assert_array_equal(off.cpu().numpy(), want_off)
            np.testing.assert_array_equal(inv.cpu().numpy(), want_inv)


def test_sort_rows_sizes_around_the_forms():
    """Slots on both sides of where the counted form begins, and of its blocks."""
    rng = np.random.default_rng(17)
    T = 1
    while ops.moe_sort_scratch_bytes(T + 1, 1, 16) == 0:
        T += 1
    for t in (T - 1, T, T + 1, T + 63, 2 * T + 1, 4 * T):
        check_sort(t, 1, 16, 16, "bf16", None, routing(rng, t, 1, 16), t)


@pytest.mark.parametrize("T,k,E", [(200000, 2, 100), (40000, 8, 1024)])
def test_sort_rows_many_slots(T, k, E):
    """Blocks of more slots than the smallest."""
    rng = np.random.default_rng(T)
    ids = routing(rng, T, k, E, away=0.1, repeats=True, skew=2.0)
    d = dev()
    x = torch.arange(T, dtype=torch.int32).view(torch.int16).view(T, 2).repeat(1, 4).view(torch.bfloat16).contiguous()
    rows, _, offsets, inv = ops.moe_sort_rows(x.to(d), torch.from_numpy(ids).to(d), E)
    want_off, want_inv, token = O.sort_slots(ids, E)
    np.testing.assert_array_equal(offsets.cpu().numpy(), want_off)
    np.testing.assert_array_equal(inv.cpu().numpy(), want_inv)
    n = int(want_off[-1])
    np.testing.assert_array_equal(rows[:n].view(torch.int16).cpu().numpy(), x.view(torch.int16).numpy()[token])


def test_sort_rows_of_no_tokens():
    d = dev()
    offsets = torch.full((6,), 9, dtype=torch.int32, device=d)
    rows, scales, off, inv = ops.moe_sort_rows(torch.empty(0, 64, dtype=torch.bfloat16, device=d),
                                               torch.empty(0, 2, dtype=torch.int32, device=d), 5, quant="int8",
                                               offsets=offsets)
    assert rows.shape == (0, 64) and scales.shape == (0,) and inv.shape == (0, 2)
    assert off is offsets and off.tolist() == [0] * 6


def test_sort_rows_special_values():
    """int8 rows of zeros, of one large value, of values below the scale's floor,
    and a row with an infinity or a NaN, whose scale is NaN; the other rows and
    the copies of any bits stay what they are."""
    d, cols = dev(), 64
    x = torch.zeros(6, cols, dtype=torch.bfloat16)
    x[1, 3], x[2] = 3.0e38, 2.0 ** -130
    x[3, 5], x[4, 6] = float("inf"), float("nan")
    x[5] = torch.linspace(-2, 2, cols).bfloat16()
    ids = torch.tensor([[0], [1], [2], [0], [1], [2]], dtype=torch.int32)
    rows, scales, _, inv = ops.moe_sort_rows(x.to(d), ids.to(d), 3, quant="int8")
    p = inv[:, 0].long()
    good = [0, 1, 2, 5]
    c, s = O.quant_int8(bf16_to_f64(x[good]))
    np.testing.assert_array_equal(rows[p][good].cpu().numpy(), c)
    np.testing.assert_array_equal(scales[p][good].cpu().numpy(), s.astype(np.float32))
    assert scales[p][[3, 4]].isnan().all()
    copy, _, _, inv = ops.moe_sort_rows(x.to(d), ids.to(d), 3)
    assert torch.equal(copy[inv[:, 0].long()].view(torch.int16).cpu(), x.view(torch.int16))


# ------------------------------------------------------------------ combine ---

def combine_case(rng, g, T, k, n, cols, away):
    """inv of distinct rows, a share of the slots without one."""
    inv = np.full(T * k, -1, dtype=np.int64)
    live = rng.permutation(T * k)[: min(n, int(round(T * k * (1 - away))))]
    inv[live] = rng.permutation(n)[: len(live)]
    inv[inv < 0] = rng.choice([-1, n, 2 ** 31 - 1, -2 ** 31], int((inv < 0).sum()))
    rows = torch.randn(n, cols, generator=g).bfloat16()
    w = torch.rand(T, k, generator=g) * torch.logspace(-2, 1, T)[:, None]
    return inv.reshape(T, k).astype(np.int32), rows, w


COMBINE = [(1, 1, 1, 8, 0.0), (1, 8, 8, 7168, 0.0), (3, 5, 17, 40, 0.2), (64, 8, 512, 4096, 0.0), (5, 64, 320, 128, 0.5),
           (9, 9, 81, 512, 0.1), (200, 2, 300, 1032, 0.4), (1031, 8, 8248, 512, 0.0), (40, 17, 700, 520, 0.0),
           (2100, 3, 6300, 64, 0.3), (6, 4, 24, 20480, 0.0), (30, 4, 120, 2056, 1.0)]


@pytest.mark.parametrize("T,k,n,cols,away", COMBINE)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_rows(T, k, n, cols, away, weighted):
    rng, g, d = np.random.default_rng(T + cols), torch.Generator().manual_seed(T + k), dev()
    inv, rows, w = combine_case(rng, g, T, k, n, cols, away)
    ref, size = O.combine_rows(bf16_to_f64(rows), inv, w.numpy() if weighted else None)
    buf = torch.full((T + 2, cols), 5.0, dtype=torch.bfloat16, device=d)
    out = ops.moe_combine_rows(rows.to(d), torch.from_numpy(inv).to(d), w.to(d) if weighted else None, out=buf[1: T + 1])
    tol = (2.0 ** -8 * np.abs(ref) + 2.0 ** -24 * (k + 1) * size) * (1 + 2.0 ** -8)
    assert (np.abs(bf16_to_f64(out) - ref) <= tol).all()
    assert (buf[0] == 5.0).all() and (buf[T + 1] == 5.0).all()
    assert torch.equal(ops.moe_combine_rows(rows.to(d), torch.from_numpy(inv).to(d), w.to(d) if weighted else None), out)


def test_combine_rows_ignores_rows_of_no_slot():
    """NaN and infinities in rows that no slot has, and a weight of infinity at a
    slot without a row, reach no output; a token without slots is 0."""
    d = dev()
    rows = torch.full((6, 64), float("nan"), dtype=torch.bfloat16)
    rows[2], rows[4] = 1.5, -2.0
    rows[5] = float("inf")
    inv = torch.tensor([[2, -1, 4], [-1, 9, -3], [4, 6, 2]], dtype=torch.int32)
    w = torch.tensor([[2.0, float("inf"), 0.5], [float("nan")] * 3, [1.0, float("nan"), 1.0]])
    out = ops.moe_combine_rows(rows.to(d), inv.to(d), w.to(d))
    assert (out[0] == 2.0).all() and (out[1] == 0.0).all() and (out[2] == -0.5).all()
    none = ops.moe_combine_rows(rows[:0].to(d), inv.to(d), w.to(d))
    assert none.shape == (3, 64) and not none.any()


@pytest.mark.parametrize("T,k,n,cols,away", COMBINE)
@pytest.mark.parametrize("weighted,dots", [(True, True), (False, True), (True, False), (False, False)])
def test_combine_rows_bwd(T, k, n, cols, away, weighted, dots):
    rng, g, d = np.random.default_rng(T + cols), torch.Generator().manual_seed(T + k), dev()
    inv, rows, w = combine_case(rng, g, T, k, n, cols, away)
    grad = torch.randn(T, cols, generator=g).bfloat16()
    want, want_w, size = O.combine_rows_grads(bf16_to_f64(grad), bf16_to_f64(rows), inv, w.numpy() if weighted else None)
    grad_rows = torch.full((n, cols), 5.0, dtype=torch.bfloat16, device=d)
    inv_d, rows_d, w_d = torch.from_numpy(inv).to(d), rows.to(d), w.to(d) if weighted else None
    got, got_w = ops.moe_combine_rows_bwd(grad.to(d), inv_d, rows=rows_d if dots else None, weights=w_d,
                                          grad_rows=grad_rows)
    assert got is grad_rows
    none = np.isnan(want[:, 0])
    assert (grad_rows.cpu()[none] == 5.0).all(), "wrote a row that no slot has"
    np.testing.assert_array_equal(bf16_to_f64(grad_rows)[~none], O.round_bf16(O.fl32(want[~none])))
    if not dots:
        assert got_w is None
        return
    assert (np.abs(got_w.cpu().numpy().astype(np.float64) - want_w) <= 2.0 ** -24 * cols * size).all()
    assert not got_w.cpu().numpy()[(inv < 0) | (inv >= n)].any()
    again = ops.moe_combine_rows_bwd(grad.to(d), inv_d, rows=rows_d, weights=w_d)
    assert torch.equal(again[1], got_w)
    kept = torch.from_numpy(~none).to(d)
    assert torch.equal(again[0][kept], grad_rows[kept])


def test_combine_gradients_against_differences():
    """<grad_out, combine(rows, w)> moved along one weight and along one row: the
    sums are linear in each, so the difference quotient is the gradient but for
    the roundings of the two outputs (half a step each, 2^-8 of |out| times
    |grad_out|), divided by the step."""
    rng, g, d = np.random.default_rng(4), torch.Generator().manual_seed(4), dev()
    T, k, n, cols = 6, 3, 18, 256
    inv, rows, w = combine_case(rng, g, T, k, n, cols, 0.2)
    grad = torch.randn(T, cols, generator=g).bfloat16()
    inv_d, rows_d, w_d = torch.from_numpy(inv).to(d), rows.to(d), w.to(d)
    d_rows, d_w = ops.moe_combine_rows_bwd(grad.to(d), inv_d, rows=rows_d, weights=w_d)
    gd = grad.double().to(d)

    def value(rows, weights):
        out = ops.moe_combine_rows(rows, inv_d, weights).double()
        return float((gd * out).sum()), float((gd * out).abs().sum())

    step = 4.0
    for t in range(T):
        for j in range(k):
            up, down = w_d.clone(), w_d.clone()
            up[t, j] += step
            down[t, j] -= step
            (a, sa), (b, sb) = value(rows_d, up), value(rows_d, down)
            assert abs((a - b) / (2 * step) - float(d_w[t, j])) <= 2.0 ** -8 * (sa + sb) / (2 * step) * 1.01
    for t, j in ((0, 0), (2, 1), (5, 2)):
        r = int(inv[t, j])
        if not 0 <= r < n:
            continue
        move = torch.ones(cols, device=d).bfloat16() * 2 * step
        up, down = rows_d.clone(), rows_d.clone()
        up[r], down[r] = move, -move
        (a, sa), (b, sb) = value(up, w_d), value(down, w_d)
        want = float((d_rows[r].double() * move.double()).sum())
        size = float((d_rows[r].double() * move.double()).abs().sum())
        assert abs((a - b) / 2 - want) <= 2.0 ** -8 * ((sa + sb) / 2 + size) * 1.01


def test_sort_and_combine_are_each_others_gradients():
    """combine without weights of what sort made: every token as often as it was
    routed; and the backward of that combine puts rows where sort puts them."""
    rng, d = np.random.default_rng(12), dev()
    T, k, E, cols = 300, 4, 10, 512
    ids = routing(rng, T, k, E, away=0.3)
    x = torch.randint(-16, 17, (T, cols)).bfloat16().to(d)
    rows, _, offsets, inv = ops.moe_sort_rows(x, torch.from_numpy(ids).to(d), E)
    back = ops.moe_combine_rows(rows, inv)
    times = torch.from_numpy(((ids >= 0) & (ids < E)).sum(1)).to(d)
    assert torch.equal(back, (x.float() * times[:, None]).bfloat16())
    placed, _ = ops.moe_combine_rows_bwd(x, inv)
    n = int(offsets[-1])
    assert torch.equal(placed[:n], rows[:n])


# ---------------------------------------------------------- large and apart ---

@pytest.mark.parametrize("T,k,cols,kind,quant", [
    (4500, 8, 4096, "bf16", None), (9000, 8, 2048, "bf16", None), (9000, 8, 2056, "bf16", None),
    (300000, 2, 256, "bf16", None), (9000, 8, 4096, "bf16", "int8"), (4600, 8, 8192, "bf16", "fp8"),
    (9000, 8, 4096, "int8", None)])
def test_sort_rows_more_than_the_last_cache_holds(T, k, cols, kind, quant):
    """Rows of 256 MiB and more against torch's stable sort and the quantisers' own rows."""
    d, E = dev(), 100
    g = torch.Generator(device=d).manual_seed(T + cols)
    x, xs = (torch.randn(T, cols, generator=g, device=d).bfloat16(), None) if kind == "bf16" else (
        torch.randint(-128, 128, (T, cols), generator=g, device=d, dtype=torch.int8), torch.rand(T, generator=g, device=d))
    ids = torch.randint(-5, E + 5, (T, k), generator=g, device=d, dtype=torch.int32)
    rows, scales, offsets, inv = ops.moe_sort_rows(x, ids, E, x_scale=xs, quant=quant)
    assert rows.nbytes >= 256 << 20
    flat = ids.flatten().long()
    routed = torch.nonzero((flat >= 0) & (flat < E))[:, 0]
    order = routed[torch.sort(flat[routed], stable=True).indices]
    want = torch.full((T * k,), -1, dtype=torch.int32, device=d)
    want[order] = torch.arange(len(order), dtype=torch.int32, device=d)
    assert torch.equal(inv.flatten(), want)
    assert torch.equal(offsets.long(), torch.searchsorted(flat[order].contiguous(), torch.arange(E + 1, device=d)))
    if quant == "int8":
        x, xs = ops.moe_quant_act_int8(x)
    elif quant == "fp8":
        x, xs = ops.moe_quant_act(x)
    for lo in range(0, len(order), 8192):
        part = order[lo: lo + 8192]
        at = slice(lo, lo + len(part))
        assert torch.equal(rows[at].view(torch.uint8), x[part // k].view(torch.uint8))
        assert xs is None or torch.equal(scales[at], xs[part // k])


@pytest.mark.parametrize("T,cols", [(4500, 4096), (17000, 1000), (9001, 2056)])
def test_combine_more_than_the_last_cache_holds(T, cols):
    """The combine of 256 MiB of rows and more, and its gradient: the bits that parts
    of the tokens give, which the definition is checked on, and the definition on some."""
    d, k = dev(), 8
    g = torch.Generator(device=d).manual_seed(T)
    rows = torch.randn(T * k, cols, generator=g, device=d).bfloat16()
    assert rows.nbytes >= 256 << 20
    inv = torch.randperm(T * k, generator=g, device=d).int().view(T, k)
    inv[::7, 3] = -1
    w, grad = torch.rand(T, k, generator=g, device=d), torch.randn(T, cols, generator=g, device=d).bfloat16()
    out = ops.moe_combine_rows(rows, inv, w)
    bare = ops.moe_combine_rows(rows, inv)
    d_rows, d_w = ops.moe_combine_rows_bwd(grad, inv, rows=rows, weights=w)
    for lo in range(0, T, 2000):
        part = slice(lo, min(T, lo + 2000))
        mine = inv[part].flatten()
        slots = torch.where(mine >= 0, torch.arange(len(mine), device=d, dtype=torch.int32), -1).view(-1, k)
        few = rows[mine.clamp(min=0).long()]
        assert torch.equal(ops.moe_combine_rows(few, slots, w[part]), out[part])
        assert torch.equal(ops.moe_combine_rows(few, slots), bare[part])
        g_rows, g_w = ops.moe_combine_rows_bwd(grad[part], slots, rows=few, weights=w[part])
        kept = mine >= 0
        assert torch.equal(g_rows[kept], d_rows[mine[kept].long()]) and torch.equal(g_w, d_w[part])
    some = slice(T - 64, T)
    ref, size = O.combine_rows(bf16_to_f64(rows), inv[some].cpu().numpy(), w[some].cpu().numpy())
    assert (np.abs(bf16_to_f64(out[some]) - ref) <= (2.0 ** -8 * np.abs(ref) + 2.0 ** -24 * (k + 1) * size)
            * (1 + 2.0 ** -8)).all()


def test_beyond_32_bits():
    """Sources, rows and gradients past 2^32 elements: the last tokens of large
    batches (the first ones are not routed)."""
    d = dev()
    T, cols, last = 2 ** 32 // 8192 + 70, 8192, 5
    ids = torch.full((T, 1), -1, dtype=torch.int32, device=d)
    ids[-last:, 0] = torch.tensor([2, 0, 2, 1, 0], dtype=torch.int32, device=d)
    x = torch.zeros(T, cols, dtype=torch.bfloat16, device=d)
    tail = torch.randn(last, cols, generator=torch.Generator().manual_seed(1)).bfloat16().to(d)
    x[-last:] = tail
    rows = torch.empty(T, cols, dtype=torch.bfloat16, device=d)
    _, _, offsets, inv = ops.moe_sort_rows(x, ids, 3, rows=rows)
    assert offsets.tolist() == [0, 2, 3, 5] and inv[-last:, 0].tolist() == [3, 0, 4, 2, 1]
    assert torch.equal(rows[inv[-last:, 0].long()], tail)
    # rows far back in a large buffer, and tokens' outputs as far back
    n = rows.shape[0]
    rows[n - 3] = tail[0]
    far = torch.full((T, 1), -1, dtype=torch.int32, device=d)
    far[-1, 0] = n - 3
    out = ops.moe_combine_rows(rows, far, out=x)
    assert torch.equal(out[-1], tail[0]) and not out[:-1].any()
    grad_rows, grad_w = ops.moe_combine_rows_bwd(x, far, rows=rows, weights=torch.full((T, 1), 2.0, device=d))
    assert torch.equal(grad_rows[n - 3], (2 * tail[0].float()).bfloat16())
    want = float(tail[0].double().square().sum())
    assert abs(float(grad_w[-1, 0]) - want) <= 2.0 ** -24 * cols * want and not grad_w[:-1].any()


def test_views_at_any_offset_of_16_bytes():
    """Operands that start inside other buffers, 16 bytes on."""
    rng, d = np.random.default_rng(3), dev()
    T, k, E, cols = 20, 3, 6, 136
    ids = torch.from_numpy(routing(rng, T, k, E)).to(d)
    flat = torch.randn(T * cols + 8, device=d).bfloat16()
    x = flat[8:].view(T, cols)
    rows, _, off, inv = ops.moe_sort_rows(x, ids, E)
    clean = ops.moe_sort_rows(x.clone(), ids, E)
    assert torch.equal(rows, clean[0]) and torch.equal(inv, clean[3])
    with pytest.raises(ops.MoeError):
        ops.moe_sort_rows(flat[4: 4 + T * cols].view(T, cols), ids, E)
