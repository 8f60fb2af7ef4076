"""The operators around the layer on the GPU against their 64-bit definitions
(oracle/rows_oracle.py).

Comparison rules, fixed before the first run
  * moe_rmsnorm and moe_silu_mul: bit for bit.  The definitions round a 64-bit
    result once to fp32 and then bf16; two orders of a 64-bit sum differ by
    about 2^-50, far less than the distance of these seeded values to a
    rounding border.
  * products of small whole numbers under power-of-two scales: bit for bit
    (every partial sum is an exact fp32 value, and no product is 2^14 times
    another, so the fp8 matrix cores drop nothing).
  * products of random values, per output:
      2^-8 |o|                              half a step of bf16, and
      2^-24 (k/128 + 128 + 16) S            fp32 additions, S the sum of |products|: 128 inside a block,
                                            one per block, up to 16 partial sums joined, and
      fp8: 2^-13 128 sum_b s_b max_k |p_k|  terms below 2^-14 of the largest in their group are dropped; twice that
"""
import threading

import numpy as np
import pytest
import torch

import oracle as O
from moe_layer_amd import ops

from gpu_util import bf16_to_f64, dev, log

pytestmark = pytest.mark.gpu


def rng_bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def check_codes(quant, y_bf16, codes, scales):
    """codes and scales of bf16 y: the oracle's, and moe_quant_act's."""
    group = 128 if quant == "fp8" else 32
    c, s, _ = O.quant_act(bf16_to_f64(y_bf16), group)
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    want = s.astype(np.float32) if quant == "fp8" else O.e8m0_encode(s)
    np.testing.assert_array_equal(scales.cpu().numpy(), want)
    ref = ops.moe_quant_act(y_bf16) if quant == "fp8" else ops.moe_quant_act_mx(y_bf16)
    assert same_bits(codes, ref[0]) and same_bits(scales, ref[1])


# --------------------------------------------------------------------- norm ---

def with_formats(shapes):
    """(rows, cols, quant) for every format whose quantisation groups the columns fill."""
    return [(r, c, q) for r, c in shapes for q, m in ((None, 8), ("fp8", 128), ("mxfp8", 32)) if c % m == 0]


@pytest.mark.parametrize("rows,cols,quant", with_formats(
    [(1, 8), (3, 136), (6, 96), (5, 128), (2, 520), (65, 256), (7, 2048), (9, 2176), (4, 4096), (3, 7168), (2, 8320),
     (2, 16384), (3, 16512), (1, 32768)]))
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(rows, cols, quant, residual):
    g = torch.Generator().manual_seed(rows * 100003 + cols)
    x, r = rng_bf16(g, rows, cols), rng_bf16(g, rows, cols, scale=3.0) if residual else None
    w = (1 + 0.2 * torch.randn(cols, generator=g)).bfloat16()
    x[0, : cols // 8] *= 30
    yo, ro = O.rmsnorm(bf16_to_f64(x), None if r is None else bf16_to_f64(r), bf16_to_f64(w), 1e-5)
    d = dev()
    xd, wd, rd = x.to(d), w.to(d), None if r is None else r.to(d)
    y, res, codes, scales = ops.moe_rmsnorm(xd, wd, 1e-5, residual=rd, quant=quant, with_y=True)
    np.testing.assert_array_equal(bf16_to_f64(y), yo)
    if residual:
        np.testing.assert_array_equal(bf16_to_f64(res), ro)
    else:
        assert res is None
    if quant:
        check_codes(quant, y, codes, scales)
        only = ops.moe_rmsnorm(xd, wd, 1e-5, residual=rd, quant=quant)       # without the bf16 row
        assert only[0] is None and same_bits(only[2], codes) and same_bits(only[3], scales)
    # in place: the residual stream and the row replace their inputs
    if residual:
        x2, r2 = xd.clone(), rd.clone()
        y2, res2, *_ = ops.moe_rmsnorm(x2, wd, 1e-5, residual=r2, y=x2, residual_out=r2)
        assert y2 is x2 and res2 is r2 and same_bits(x2, y) and same_bits(r2, res)


def test_rmsnorm_special_rows():
    """A row of zeros (eps keeps it 0), the smallest and largest bf16
    magnitudes (squares far outside fp32's range), a single large element, and
    negative zeros; a row of zeros with eps 0 is NaN and touches no other."""
    d, cols = dev(), 256
    x = torch.zeros(6, cols, dtype=torch.bfloat16)
    x[1], x[2] = 2.0 ** -130, 3.0e38
    x[3, 17] = 1.0e5
    x[4, ::2], x[4, 1::2] = -0.0, 2.0
    x[5] = torch.linspace(-3, 3, cols).bfloat16()
    w = torch.full((cols,), 1.5).bfloat16()
    for eps in (1e-6, 0.0):
        with np.errstate(all="ignore"):
            yo, _ = O.rmsnorm(bf16_to_f64(x), None, bf16_to_f64(w), eps)
        y, _, codes, scales = ops.moe_rmsnorm(x.to(d), w.to(d), eps, quant="fp8", with_y=True)
        got = bf16_to_f64(y)
        rows = slice(0, 6) if eps else slice(1, 6)
        np.testing.assert_array_equal(got[rows], yo[rows])
        check_codes("fp8", y[1:], codes[1:], scales[1:])
        assert eps or np.isnan(got[0]).all()


def test_rmsnorm_many_rows():
    """More rows than workgroups are resident, each its own scale."""
    g = torch.Generator().manual_seed(8)
    rows, cols = 5003, 640
    x = (torch.randn(rows, cols, generator=g) * torch.logspace(-3, 3, rows)[:, None]).bfloat16()
    w = (1 + 0.1 * torch.randn(cols, generator=g)).bfloat16()
    y, _, codes, scales = ops.moe_rmsnorm(x.to(dev()), w.to(dev()), quant="mxfp8", with_y=True)
    yo, _ = O.rmsnorm(bf16_to_f64(x), None, bf16_to_f64(w), 1e-6)
    np.testing.assert_array_equal(bf16_to_f64(y), yo)
    check_codes("mxfp8", y, codes, scales)


# ---------------------------------------------------------------------- act ---

def test_silu_every_bf16_gate():
    """bf16(silu(g)) is correctly rounded for every finite bf16 g."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    g = O.bf16_bits_to_f64(bits)
    bits = bits[np.isfinite(g)]
    gate = torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).view(-1, 256)
    h = torch.cat([gate, torch.ones_like(gate)], 1).to(dev())
    y, _, _ = ops.moe_silu_mul(h)
    np.testing.assert_array_equal(bf16_to_f64(y), O.silu_mul(bf16_to_f64(h)))


@pytest.mark.parametrize("rows,cols,quant", with_formats(
    [(1, 8), (3, 24), (4, 160), (1, 128), (2, 256), (17, 384), (5, 1536), (129, 2048)]))
@pytest.mark.parametrize("limit", [0.0, 2.5])
def test_silu_mul(rows, cols, quant, limit):
    g = torch.Generator().manual_seed(rows * 31 + cols)
    h = rng_bf16(g, rows, 2 * cols, scale=3.0)
    h[0, :4] = 0.0                                     # zeros of either sign
    h[0, 4:8] = -0.0
    hd = h.to(dev())
    y, codes, scales = ops.moe_silu_mul(hd, quant=quant, clamp_limit=limit, with_y=True)
    np.testing.assert_array_equal(bf16_to_f64(y), O.silu_mul(bf16_to_f64(h), limit))
    if quant:
        check_codes(quant, y, codes, scales)
        only = ops.moe_silu_mul(hd, quant=quant, clamp_limit=limit)
        assert only[0] is None and same_bits(only[1], codes) and same_bits(only[2], scales)


# ----------------------------------------------------------------- products ---

def small_fp8(rng, shape, most):
    """E4M3 codes of whole numbers |v| <= most (<= 15: 4 significant bits)."""
    v = rng.integers(-most, most + 1, shape).astype(np.float32)
    return torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8)


def pow2(rng, shape, lo, hi):
    return torch.from_numpy(np.ldexp(1.0, rng.integers(lo, hi + 1, shape)).astype(np.float32))


def exact_operands(rng, rows, E, N, K, fp8):
    """Operands whose every partial sum is an exact fp32 value: |a| <= 7 and
    |w| <= 15, scales from four neighbouring powers of two on either side, so a
    sum is at most 105 K 2^6 of its smallest unit, below 2^24 for K <= 2304."""
    assert 105 * K * 64 < 2 ** 24
    nb = -(-N // 128)
    if fp8:
        a, w = small_fp8(rng, (rows, K), 7), small_fp8(rng, (E, N, K), 15)
        sa, sw = pow2(rng, (rows, K // 128), -2, 1), pow2(rng, (E, nb, K // 128), -1, 2)
        return a, w, sa, sw, O.act_values(a.numpy(), sa.numpy()), O.block_values(w.numpy(), sw.numpy())
    a = torch.from_numpy(rng.integers(-7, 8, (rows, K)).astype(np.float32)).bfloat16()
    w = torch.from_numpy(rng.integers(-15, 16, (E, N, K)).astype(np.float32)).bfloat16()
    return a, w, None, None, bf16_to_f64(a), bf16_to_f64(w)


def random_operands(rng, rows, E, N, K, fp8):
    nb = -(-N // 128)
    if fp8:
        a = torch.from_numpy(rng.standard_normal((rows, K)).astype(np.float32) * 60).clamp(-448, 448)
        w = torch.from_numpy(rng.standard_normal((E, N, K)).astype(np.float32) * 60).clamp(-448, 448)
        a, w = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (a, w))
        sa = torch.from_numpy((0.002 + rng.random((rows, K // 128)) * 0.05).astype(np.float32))
        sw = torch.from_numpy((0.0002 + rng.random((E, nb, K // 128)) * 0.01).astype(np.float32))
        return a, w, sa, sw, O.act_values(a.numpy(), sa.numpy()), O.block_values(w.numpy(), sw.numpy())
    a = torch.from_numpy(rng.standard_normal((rows, K)).astype(np.float32)).bfloat16()
    w = torch.from_numpy((rng.standard_normal((E, N, K)) / K ** 0.5).astype(np.float32)).bfloat16()
    return a, w, None, None, bf16_to_f64(a), bf16_to_f64(w)


def tolerance(av, wv, out, fp8):
    """The bound of the module's docstring for one group's rows."""
    K = av.shape[1]
    tol = 2.0 ** -8 * np.abs(out) + 2.0 ** -24 * (K / 128 + 144) * (np.abs(av) @ np.abs(wv).T)
    if fp8:
        for b in range(K // 128):
            k = slice(128 * b, 128 * b + 128)
            # max_k |a w| <= max |a| max |w|
            tol += 2.0 ** -6 * np.abs(av[:, k]).max(1)[:, None] * np.abs(wv[:, k]).max(1)[None, :]
    return tol


def put(*ts):
    return [None if t is None else t.to(dev()) for t in ts]


DENSE = [(1, 1, 128), (1, 16, 256), (2, 3, 128), (15, 17, 384), (16, 128, 2048), (17, 130, 256), (33, 200, 640),
         (64, 576, 512), (65, 64, 1024), (100, 4096, 128), (127, 257, 256), (128, 256, 384), (129, 255, 128),
         (255, 300, 512), (256, 512, 256), (300, 129, 1152), (513, 640, 256), (1000, 264, 384), (1, 4096, 2048),
         (40, 1000, 2048), (700, 1031, 256), (2, 20000, 128), (243, 4315, 256), (324, 2712, 256), (300, 4096, 2304),
         (770, 4741, 128), (1358, 1030, 384), (194, 4424, 128), (1500, 2001, 2304), (2177, 2737, 128),
         (1100, 5003, 1280), (3905, 3217, 128), (2300, 4100, 2304), (254, 4287, 640), (36, 4187, 1536)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_gemm_fp8(M, N, K):
    for make in (exact_operands, random_operands):
        rng = np.random.default_rng(M * 7 + N * 3 + K)
        a, w, sa, sw, av, wv = make(rng, M, 1, N, K, True)
        ref = av @ wv[0].T
        ad, wd, sad, swd = put(a, w[0], sa, sw[0])
        out = torch.full((M + 1, N), 5.0, dtype=torch.bfloat16, device=dev())
        ops.moe_gemm_fp8(ad, sad, wd, swd, out=out[:M])
        got = bf16_to_f64(out)
        assert (got[M] == 5.0).all(), "wrote behind the last row"
        if make is exact_operands:
            np.testing.assert_array_equal(got[:M], O.round_bf16(ref))
        else:
            excess = np.abs(got[:M] - ref) / tolerance(av, wv[0], ref, True)
            log(f"gemm_fp8 {M}x{N}x{K}: {excess.max():.3f} of the tolerance")
            assert excess.max() <= 1.0
        again = ops.moe_gemm_fp8(ad.view(torch.float8_e4m3fn), sad, wd, swd)
        assert same_bits(again, out[:M].contiguous()), "a second call differs"


def sizes_to_offsets(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


GROUPED = [  # group sizes, rows before the first and behind the last group, N, K
    ([1], 0, 0, 16, 128), ([0, 0, 3], 0, 2, 40, 128), ([5, 0, 1, 0, 0, 18], 2, 3, 130, 256),
    ([16, 17, 15, 33], 0, 0, 64, 384), ([64, 1, 0, 65, 129], 1, 0, 257, 256), ([0] * 8, 3, 4, 32, 128),
    ([2, 1] * 40 + [0] * 20, 0, 1, 96, 512), ([300, 0, 7], 0, 0, 512, 256), ([0, 511, 1], 0, 9, 384, 640),
    ([1] * 130, 0, 0, 256, 2048), ([40, 60, 3, 0, 128, 256, 255, 70], 5, 6, 320, 256),
    ([128] * 6, 0, 0, 1000, 384), ([600, 500], 0, 0, 1536, 512),
    ([0] * 700 + [3, 1] * 150 + [0] * 23 + [90], 0, 0, 40, 128),   # the most groups there can be
]


@pytest.mark.parametrize("sizes,head,tail,N,K", GROUPED)
@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_gemm(sizes, head, tail, N, K, fp8):
    rows, E = head + sum(sizes) + tail, len(sizes)
    off = sizes_to_offsets(sizes, head)
    for make in (exact_operands, random_operands):
        rng = np.random.default_rng(rows * 5 + E * 3 + N)
        a, w, sa, sw, av, wv = make(rng, rows, E, N, K, fp8)
        ref = O.grouped_product(av, wv, off)
        ad, wd, sad, swd = put(a, w, sa, sw)
        offd = torch.from_numpy(off).to(dev())
        out = torch.full((rows, N), 5.0, dtype=torch.bfloat16, device=dev())
        ops.moe_grouped_gemm(ad, wd, offd, sad, swd, out=out)
        got = bf16_to_f64(out)
        outside = np.isnan(ref[:, 0])
        assert (got[outside] == 5.0).all(), "wrote outside the groups"
        inside = ~outside
        if make is exact_operands:
            np.testing.assert_array_equal(got[inside], O.round_bf16(ref[inside]))
        else:
            for e in range(E):
                lo, hi = off[e], off[e + 1]
                if hi > lo:
                    tol = tolerance(av[lo:hi], wv[e], ref[lo:hi], fp8)
                    assert (np.abs(got[lo:hi] - ref[lo:hi]) <= tol).all(), (e, lo, hi)
        second = out.clone()
        ops.moe_grouped_gemm(ad, wd, offd, sad, swd, out=second)
        assert same_bits(second, out)


# rows in groups of uneven sizes (some empty), N, K: the larger tiles, and weights too many for the last-level cache
TILES = [(1083, 2, 103, 384), (4202, 2, 79, 128), (5939, 16, 87, 256), (5683, 3, 137, 256), (955, 40, 390, 256),
         (748, 40, 474, 1280), (59, 16, 1341, 384), (1358, 40, 783, 128), (5449, 3, 129, 384), (3747, 40, 1156, 128),
         (4763, 5, 2601, 128), (4815, 40, 1288, 640), (2995, 40, 391, 2304), (5247, 40, 150, 256),
         (852, 40, 398, 512), (40, 32, 4096, 1024), (700, 32, 4096, 1024), (1020, 16, 916, 1152),
         (6000, 30, 1300, 2304), (2500, 6, 2601, 2304)]


@pytest.mark.parametrize("rows,E,N,K", TILES)
@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_gemm_tiles(rows, E, N, K, fp8):
    rng = np.random.default_rng(rows + E)
    load = rng.exponential(size=E) ** 2
    off = sizes_to_offsets(rng.multinomial(rows, load / load.sum()))
    a, w, sa, sw, av, wv = exact_operands(rng, rows, E, N, K, fp8)
    ref = O.grouped_product(av, wv, off)
    ad, wd, sad, swd = put(a, w, sa, sw)
    buf = torch.full((rows + 2, N), 5.0, dtype=torch.bfloat16, device=dev())
    # an output that starts inside a buffer where its rows are whole 16-byte pieces
    out = buf[1: rows + 1] if (2 * N) % 16 == 0 else buf[:rows]
    ops.moe_grouped_gemm(ad, wd, torch.from_numpy(off).to(dev()), sad, swd, out=out)
    np.testing.assert_array_equal(bf16_to_f64(out), O.round_bf16(ref))
    assert (buf[rows + 1:] == 5.0).all() and (out.data_ptr() == buf.data_ptr() or (buf[0] == 5.0).all())


@pytest.mark.parametrize("K", [64, 192, 320])
def test_grouped_bf16_odd_steps(K):
    """K in whole 64-element steps that are no multiple of 128."""
    rng = np.random.default_rng(K)
    sizes = [3, 0, 40, 17]
    off = sizes_to_offsets(sizes)
    a, w, _, _, av, wv = exact_operands(rng, sum(sizes), len(sizes), 72, K, False)
    out = ops.moe_grouped_gemm(*put(a, w, torch.from_numpy(off)))
    np.testing.assert_array_equal(bf16_to_f64(out), O.round_bf16(O.grouped_product(av, wv, off)))


@pytest.mark.parametrize("K", [64, 192, 448])
def test_grouped_bf16_large_tiles_odd_steps(K):
    """One, three and seven stages of the largest tile; last blocks of every width class."""
    rng = np.random.default_rng(K)
    sizes = [2048 + 65, 1024 + 129, 0, 1, 768 + 64, 512 + 128]
    off = sizes_to_offsets(sizes)
    a, w, _, _, av, wv = exact_operands(rng, sum(sizes), len(sizes), 2601, K, False)
    out = ops.moe_grouped_gemm(*put(a, w, torch.from_numpy(off)))
    np.testing.assert_array_equal(bf16_to_f64(out), O.round_bf16(O.grouped_product(av, wv, off)))


@pytest.mark.parametrize("rows,N,K,fp8", [(3, 40, 2 ** 20, True), (300, 260, 2 ** 16, True), (20, 40, 2 ** 18, False),
                                          (520, 300, 2 ** 15, False)])
def test_long_sums(rows, N, K, fp8):
    """K up to the limit, one group (fp8: the dense product).  bf16 sums take
    one addition per 32 products, so K / 32 stands in place of K / 128."""
    rng = np.random.default_rng(K + rows)
    a, w, sa, sw, av, wv = random_operands(rng, rows, 1, N, K, fp8)
    ad, wd, sad, swd = put(a, w, sa, sw)
    if fp8:
        out = ops.moe_gemm_fp8(ad, sad, wd[0], swd[0])
    else:
        out = ops.moe_grouped_gemm(ad, wd, torch.tensor([0, rows], dtype=torch.int32, device=dev()))
    ref = av @ wv[0].T
    tol = tolerance(av, wv[0], ref, fp8) + 2.0 ** -24 * (K / 32 - K / 128) * (np.abs(av) @ np.abs(wv[0]).T)
    assert (np.abs(bf16_to_f64(out) - ref) <= tol).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("off", [[-5, 3, 7, 400], [10, 4, 90, 60], [0, 1000, 1000, 2000], [120, 120, 120, 120]])
def test_grouped_bad_offsets_stay_in_bounds(off, fp8):
    """A table that is not ascending or leaves [0, rows] is held to the rows:
    nothing outside the output is touched (guard rows on both sides)."""
    rows, E, N, K = 100, 3, 200, 256
    rng = np.random.default_rng(5)
    a, w, sa, sw, *_ = random_operands(rng, rows, E, N, K, fp8)
    ad, wd, sad, swd = put(a, w, sa, sw)
    buf = torch.full((rows + 256, N), 5.0, dtype=torch.bfloat16, device=dev())
    ops.moe_grouped_gemm(ad, wd, torch.tensor(off, dtype=torch.int32, device=dev()), sad, swd,
                         out=buf[128: 128 + rows])
    torch.cuda.synchronize()
    assert (buf[:128] == 5.0).all() and (buf[128 + rows:] == 5.0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_rows_do_not_depend_on_their_neighbours(fp8):
    """A NaN or an infinity in one row stays in that row."""
    rng = np.random.default_rng(9)
    sizes = [70, 3, 20]
    rows, N, K = sum(sizes), 136, 256
    a, w, sa, sw, *_ = random_operands(rng, rows, 3, N, K, fp8)
    ad, wd, sad, swd = put(a, w, sa, sw)
    off = torch.from_numpy(sizes_to_offsets(sizes)).to(dev())
    clean = ops.moe_grouped_gemm(ad, wd, off, sad, swd)
    bad = ad.clone()
    if fp8:
        bad[69] = 0x7f                     # E4M3's NaN, in the last row of a group
    else:
        bad[69], bad[71, 5] = float("nan"), float("inf")
    got = ops.moe_grouped_gemm(bad, wd, off, sad, swd)
    keep = torch.ones(rows, dtype=torch.bool, device=dev())
    keep[[69, 71]] = False
    assert torch.equal(got[keep].view(torch.int16), clean[keep].view(torch.int16))
    assert got[69].isnan().all()


def test_beyond_32_bits():
    """Buffers past 2^32 elements: the last rows of large inputs, weights and
    outputs, with everything in front of them zero (or not looked at)."""
    d = dev()
    last = 3
    g = torch.Generator().manual_seed(32)
    # rows of x, h, codes and outputs past 2^32 elements
    rows, cols = 2 ** 32 // 8192 + 1029, 8192
    tail = rng_bf16(g, last, cols)
    w = rng_bf16(g, cols)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=d)
    x[-last:] = tail.to(d)
    y, _, codes, scales = ops.moe_rmsnorm(x, w.to(d), 1e-6, quant="fp8", y=x)     # in place, to save memory
    yo, _ = O.rmsnorm(bf16_to_f64(tail), None, bf16_to_f64(w), 1e-6)
    np.testing.assert_array_equal(bf16_to_f64(y[-last:]), yo)
    check_codes("fp8", y[-last:].contiguous(), codes[-last:], scales[-last:])
    assert not y[:-last].any()
    a, c2, s2 = ops.moe_silu_mul(x, quant="mxfp8", with_y=True)
    ao = O.silu_mul(yo)
    np.testing.assert_array_equal(bf16_to_f64(a[-last:]), ao)
    check_codes("mxfp8", a[-last:].contiguous(), c2[-last:], s2[-last:])
    del y, a, c2, s2
    # the codes as rows of a product: a past 2^32 bytes
    rng = np.random.default_rng(33)
    _, wq, _, sw, _, wv = exact_operands(rng, 1, 2, 40, 2304, True)
    wq, sw, wv = wq[:, :, :256].contiguous(), sw[:, :, :2].contiguous(), wv[:, :, :256]
    big = codes.view(-1, 256)                     # more rows of fewer columns
    n = big.shape[0]
    scale = torch.ones(n, 2, dtype=torch.float32, device=d)
    off = torch.tensor([5, n - 70, n], dtype=torch.int32, device=d)
    av = O.act_values(big[-70:].cpu().numpy(), np.ones((70, 2)))
    ref = av @ wv[1].T
    wqd, swd = put(wq, sw)
    out = ops.moe_grouped_gemm(big, wqd, off, scale, swd)
    assert (np.abs(bf16_to_f64(out[-70:]) - ref) <= tolerance(av, wv[1], ref, True)).all()
    out = ops.moe_gemm_fp8(big, scale, wqd[1].contiguous(), swd[1].contiguous())
    assert (np.abs(bf16_to_f64(out[-70:]) - ref) <= tolerance(av, wv[1], ref, True)).all()
    del x, codes, scales, big, scale, out
    # outputs past 2^32 elements, and weights past 2^32 bytes
    rows, N, K = 2 ** 32 // 4096 + 517, 4096, 128
    ab = torch.zeros(rows, K, dtype=torch.bfloat16, device=d)
    tail, wide = rng_bf16(g, 300, K), rng_bf16(g, 1, N, K)
    ab[-300:] = tail.to(d)
    out = ops.moe_grouped_gemm(ab, wide.to(d), torch.tensor([0, rows], dtype=torch.int32, device=d))
    av, wv = bf16_to_f64(tail), bf16_to_f64(wide)
    ref = av @ wv[0].T
    assert (np.abs(bf16_to_f64(out[-300:]) - ref) <= tolerance(av, wv[0], ref, False)).all()
    del out, ab
    E, N, K = 300, 4096, 2048
    wl = torch.zeros(E, N, K, dtype=torch.bfloat16, device=d)
    one = rng_bf16(g, N, K)
    wl[-1] = one.to(d)
    at = rng_bf16(g, 20, K)
    sizes = [0] * (E - 2) + [4, 16]
    out = ops.moe_grouped_gemm(at.to(d), wl, torch.from_numpy(sizes_to_offsets(sizes)).to(d))
    av, wv = bf16_to_f64(at[4:]), bf16_to_f64(one)
    ref = av @ wv.T
    assert (np.abs(bf16_to_f64(out[4:]) - ref) <= tolerance(av, wv, ref, False)).all()
    assert not out[:4].any()


def test_silu_mul_beyond_one_launch():
    """More than 2^31 pieces of 8 outputs, which take a second launch: rows on
    both sides of its border."""
    d = dev()
    rows, cols, last = 2 ** 21 + 3, 8192, 8
    tail = rng_bf16(torch.Generator().manual_seed(31), last, 2 * cols)
    h = torch.empty(rows, 2 * cols, dtype=torch.bfloat16, device=d)
    h[-last:] = tail.to(d)
    _, codes, scales = ops.moe_silu_mul(h, quant="fp8")
    y = torch.from_numpy(O.silu_mul(bf16_to_f64(tail)).astype(np.float32)).bfloat16().to(d)
    check_codes("fp8", y, codes[-last:], scales[-last:])


@pytest.mark.parametrize("cols", [8, 24, 40, 104, 1000, 2816, 65544])
def test_silu_mul_row_of_every_piece(cols):
    """Every 8-column piece reads its own row: gate 1, up the row's number."""
    rows = 300
    h = torch.ones(rows, 2 * cols, dtype=torch.bfloat16)
    h[:, cols:] = torch.arange(rows, dtype=torch.float32).bfloat16()[:, None] % 256
    y = ops.moe_silu_mul(h.to(dev()))[0]
    np.testing.assert_array_equal(bf16_to_f64(y), O.silu_mul(bf16_to_f64(h)))


# ------------------------------------------------- together, as a user would ---

def test_shared_expert_chain():
    """Norm + quantise, gate/up product, gated multiply + quantise, down
    product: a shared expert, each step against the definition applied to the
    step's own input."""
    T, H, I = 37, 512, 256
    rng = np.random.default_rng(21)
    g = torch.Generator().manual_seed(21)
    x, r = rng_bf16(g, T, H), rng_bf16(g, T, H, scale=2.0)
    w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16()
    _, w13, _, s13, _, w13v = random_operands(rng, 1, 1, 2 * I, H, True)
    _, w2, _, s2, _, w2v = random_operands(rng, 1, 1, H, I, True)
    xd, rd, wd, w13d, s13d, w2d, s2d = put(x, r, w, w13[0], s13[0], w2[0], s2[0])
    _, res, codes, scales = ops.moe_rmsnorm(xd, wd, residual=rd, quant="fp8")
    h = ops.moe_gemm_fp8(codes, scales, w13d, s13d)
    _, c2, sc2 = ops.moe_silu_mul(h, quant="fp8")
    out = ops.moe_gemm_fp8(c2, sc2, w2d, s2d)

    yo, ro = O.rmsnorm(bf16_to_f64(x), bf16_to_f64(r), bf16_to_f64(w), 1e-6)
    np.testing.assert_array_equal(bf16_to_f64(res), ro)
    co, so, yv = O.quant_act(yo)
    np.testing.assert_array_equal(codes.cpu().numpy(), co)
    ref = yv @ w13v[0].T
    assert (np.abs(bf16_to_f64(h) - ref) <= tolerance(yv, w13v[0], ref, True)).all()
    co, so, av = O.quant_act(O.silu_mul(bf16_to_f64(h)))
    np.testing.assert_array_equal(c2.cpu().numpy(), co)
    ref = av @ w2v[0].T
    assert (np.abs(bf16_to_f64(out) - ref) <= tolerance(av, w2v[0], ref, True)).all()


@pytest.mark.parametrize("wdtype", ["bf16", "fp8"])
def test_expert_parallel_chain_matches_the_fused_layer(wdtype):
    """Rows sorted by expert through grouped products and the gated multiply,
    weighted and summed per token, against moe_forward on the same layer."""
    from dataclasses import replace
    from gpu_util import TAU, layer_for, routing, bits_to_bf16
    from moe_layer_amd.workloads import CONFIGS, Workload
    cfg = replace(CONFIGS["tiny"], wdtype=wdtype)
    layer, (ids, tw, _) = layer_for(cfg), routing(cfg)
    layer.ensure(range(cfg.E))
    d = dev()
    x = bits_to_bf16(Workload(cfg).x_bf16_bits()).to(d)
    ids_t = torch.from_numpy(ids.astype(np.int32)).to(d)
    tw_t = torch.from_numpy(tw.astype(np.float32)).to(d)
    ref, _ = ops.moe_forward(x, layer.w13, layer.w2, ids_t, tw_t, layer.s13, layer.s2)

    flat = ids_t.flatten().long()
    order = torch.argsort(flat, stable=True)
    off = torch.zeros(cfg.E + 1, dtype=torch.int32, device=d)
    off[1:] = torch.bincount(flat, minlength=cfg.E).cumsum(0)
    rows = x[order // cfg.topk].contiguous()
    if wdtype == "fp8":
        c, s = ops.moe_quant_act(rows)
        h = ops.moe_grouped_gemm(c, layer.w13, off, s, layer.s13)
        _, c, s = ops.moe_silu_mul(h, quant="fp8")
        y = ops.moe_grouped_gemm(c, layer.w2, off, s, layer.s2)
    else:
        h = ops.moe_grouped_gemm(rows, layer.w13, off)
        a, _, _ = ops.moe_silu_mul(h)
        y = ops.moe_grouped_gemm(a, layer.w2, off)
    out = torch.zeros(cfg.T, cfg.H, device=d)
    out.index_add_(0, order // cfg.topk, y.float() * tw_t.flatten()[order, None])
    o = ref.double()
    # both are within tau of the layer's definition
    err = (out.double() - o).abs().max() / o.square().mean().sqrt()
    log(f"expert-parallel chain {wdtype}: {float(err):.2e} of the layer's RMS")
    assert float(err) <= 2 * TAU[wdtype]


def chain(st):
    """The run of the four operators on one set of buffers."""
    ops.moe_rmsnorm(st["x"], st["w"], residual=st["r"], quant="fp8", residual_out=st["res"], codes=st["c"],
                    scales=st["s"])
    ops.moe_gemm_fp8(st["c"], st["s"], st["w13"], st["s13"], out=st["h"])
    ops.moe_silu_mul(st["h"], quant="fp8", codes=st["c2"], scales=st["s2"])
    ops.moe_grouped_gemm(st["c2"], st["w2"], st["off"], st["s2"], st["sw2"], out=st["out"])


def chain_state(seed, T=70, H=384, I=256, E=5):
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    _, w13, _, s13, *_ = random_operands(rng, 1, 1, 2 * I, H, True)
    _, w2, _, sw2, *_ = random_operands(rng, 1, E, H, I, True)
    sizes = rng.multinomial(T, [1 / E] * E)
    d = dev()
    e = lambda *s, t=torch.uint8: torch.zeros(*s, dtype=t, device=d)   # noqa: E731
    x, r, w, w13d, s13d, w2d, sw2d, off = put(rng_bf16(g, T, H), rng_bf16(g, T, H), rng_bf16(g, H), w13[0], s13[0],
                                              w2, sw2, torch.from_numpy(sizes_to_offsets(sizes)))
    return dict(x=x, r=r, w=w, w13=w13d, s13=s13d, w2=w2d, sw2=sw2d, off=off, res=e(T, H, t=torch.bfloat16),
                c=e(T, H), s=e(T, H // 128, t=torch.float32), h=e(T, 2 * I, t=torch.bfloat16), c2=e(T, I),
                s2=e(T, I // 128, t=torch.float32), out=e(T, H, t=torch.bfloat16))


def test_captured_chain_replays():
    """The chain in a captured graph, replayed on new inputs with eager work of
    the same operators between the replays."""
    st, other = chain_state(1), chain_state(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(st)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(st)
    for seed in (1, 3, 4):
        new = chain_state(seed)
        for k in ("x", "r", "off"):
            st[k].copy_(new[k])
        for k in ("w", "w13", "s13", "w2", "sw2"):
            st[k].copy_(new[k])
        st["out"].zero_()
        chain(other)
        graph.replay()
        chain(new)
        torch.cuda.synchronize()
        for k in ("res", "c", "s", "h", "c2", "s2", "out"):
            assert same_bits(st[k], new[k]), (seed, k)


def test_two_streams_at_once():
    """Chains on two streams at the same time, each with its own buffers."""
    states = [chain_state(s, T=200) for s in (5, 6)]
    want = []
    for st in states:
        chain(st)
        want.append(st["out"].clone())
        st["out"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(5):
        for st, s in zip(states, streams):
            with torch.cuda.stream(s):
                chain(st)
    torch.cuda.synchronize()
    for st, w in zip(states, want):
        assert same_bits(st["out"], w)


def test_two_threads_at_once():
    """Chains from two threads, each on a stream of its own (the calls run
    without the interpreter's lock)."""
    states = [chain_state(s, T=64) for s in (7, 8)]
    want = []
    for st in states:
        chain(st)
        want.append(st["out"].clone())
        st["out"].zero_()
    torch.cuda.synchronize()
    failed = []

    def work(st, s):
        try:
            with torch.cuda.stream(s):
                for _ in range(20):
                    chain(st)
        except Exception as e:   # noqa: BLE001 - reported by the test
            failed.append(e)

    threads = [threading.Thread(target=work, args=(st, torch.cuda.Stream())) for st in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for st, w in zip(states, want):
        assert same_bits(st["out"], w)


def test_empty_calls():
    d = dev()
    e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device=d)   # noqa: E731
    assert ops.moe_rmsnorm(e(0, 256), e(256), quant="fp8")[2].shape == (0, 256)
    assert ops.moe_silu_mul(e(0, 512))[0].shape == (0, 256)
    assert ops.moe_gemm_fp8(e(0, 128, t=torch.uint8), e(0, 1, t=torch.float32), e(5, 128, t=torch.uint8),
                            e(1, 1, t=torch.float32)).shape == (0, 5)
    assert ops.moe_grouped_gemm(e(0, 64), e(2, 8, 64), torch.zeros(3, dtype=torch.int32, device=d)).shape == (0, 8)
