"""int8 rows and products on the GPU against their 64-bit definitions
(oracle/sorted_oracle.py).

Comparison rules, fixed before the first run: everything bit for bit.  A code
is one rounding of an exact product, a scale one of a quotient; a product's sum
is exact, and its three fp32 roundings and the one to bf16 are the oracle's.
"""
import threading

import numpy as np
import pytest
import torch

import oracle as O
from moe_layer_amd import ops

from gpu_util import bf16_to_f64, dev, log

pytestmark = pytest.mark.gpu


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# --------------------------------------------------------------------- rows ---

ROWS = [(1, 16), (3, 48), (5, 512), (2, 528), (7, 1024), (4, 1040), (129, 1536), (9, 2048), (6, 2064), (3, 4096),
        (2, 4112), (3, 8192), (2, 8208), (2, 16384), (1, 16400), (2, 32768), (1031, 64),
        (5, 64), (7, 80), (9, 128), (17, 144), (9, 256), (5, 272), (2047, 1008), (2050, 48), (2049, 1008),
        (2051, 1296), (2048, 2032), (2050, 2576), (2053, 3104), (2048, 4112)]


@pytest.mark.parametrize("rows,cols", ROWS)
def test_quant_act_int8(rows, cols):
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.logspace(-6, 6, rows)[:, None]).bfloat16()
    x[0, : cols // 8] *= 20
    codes, scales = ops.moe_quant_act_int8(x.to(dev()))
    c, s = O.quant_int8(bf16_to_f64(x))
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    np.testing.assert_array_equal(scales.cpu().numpy(), s.astype(np.float32))


def test_quant_act_int8_every_largest_magnitude():
    """Rows whose largest value is every finite bf16 magnitude, in a place that
    moves along the row: scale and codes."""
    bits = np.arange(0x7F80, dtype=np.uint16)
    most = torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16)
    n, cols = len(bits), 64
    g = torch.Generator().manual_seed(2)
    x = (torch.rand(n, cols, generator=g) * 2 - 1).mul(most.float()[:, None] * 0.99).bfloat16()
    x[torch.arange(n), torch.arange(n) % cols] = -most
    codes, scales = ops.moe_quant_act_int8(x.to(dev()))
    c, s = O.quant_int8(bf16_to_f64(x))
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    np.testing.assert_array_equal(scales.cpu().numpy(), s.astype(np.float32))


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("limit", [0.0, 2.5, float("inf")])
def test_silu_mul_int8(rows, cols, limit):
    g = torch.Generator().manual_seed(rows + cols)
    h = (torch.randn(rows, 2 * cols, generator=g) * 3).bfloat16()
    codes, scales = ops.moe_silu_mul_int8(h.to(dev()), clamp_limit=limit)
    c, s = O.quant_int8(O.silu_mul(bf16_to_f64(h), limit))
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    np.testing.assert_array_equal(scales.cpu().numpy(), s.astype(np.float32))
    # moe_silu_mul's rows quantised apart
    y, _, _ = ops.moe_silu_mul(h.to(dev()), clamp_limit=limit)
    apart = ops.moe_quant_act_int8(y)
    assert same_bits(apart[0], codes) and same_bits(apart[1], scales)


@pytest.mark.parametrize("rows,cols,gated", [(33000, 1536, True), (13000, 4096, True), (110000, 464, True),
                                             (210000, 480, False), (26000, 4096, False), (4000, 32768, False)])
def test_int8_rows_more_than_the_last_cache_holds(rows, cols, gated):
    """Inputs of 192 MiB and more: the bits that parts of them give."""
    d, g = dev(), torch.Generator(device=dev()).manual_seed(rows)
    x = torch.randn(rows, cols * (2 if gated else 1), generator=g, device=d).bfloat16()
    assert x.nbytes >= 192 << 20
    run = (lambda v: ops.moe_silu_mul_int8(v, clamp_limit=2.0)) if gated else ops.moe_quant_act_int8
    codes, scales = run(x)
    for lo in range(0, rows, rows // 4):
        part = run(x[lo: lo + rows // 4])
        assert same_bits(part[0], codes[lo: lo + rows // 4]) and same_bits(part[1], scales[lo: lo + rows // 4])


@pytest.mark.parametrize("cols", [64, 2048, 8192, 32768])
def test_int8_rows_with_nan_or_infinity(cols):
    """Such a row's scale is NaN, and what a product makes of it; its neighbours
    keep their codes.  Rows of zeros are zeros."""
    d = dev()
    x = torch.randn(6, cols, generator=torch.Generator().manual_seed(cols)).bfloat16()
    x[0] = 0.0
    x[2, cols - 1], x[4, 0] = float("nan"), float("-inf")
    codes, scales = ops.moe_quant_act_int8(x.to(d))
    c, s = O.quant_int8(bf16_to_f64(x[[0, 1, 3, 5]]))
    np.testing.assert_array_equal(codes.cpu().numpy()[[0, 1, 3, 5]], c)
    np.testing.assert_array_equal(scales.cpu().numpy()[[0, 1, 3, 5]], s.astype(np.float32))
    assert scales[[2, 4]].isnan().all()
    w = torch.ones(8, cols, dtype=torch.int8, device=d)
    out = ops.moe_gemm_int8(codes, scales, w, torch.ones(8, device=d))
    assert out[[2, 4]].isnan().all() and not out[[0, 1, 3, 5]].isnan().any() and not out[0].any()
    h = torch.cat([torch.ones_like(x), x], 1)
    _, scales = ops.moe_silu_mul_int8(h.to(d))
    assert scales[[2, 4]].isnan().all() and not scales[[0, 1, 3, 5]].isnan().any()


# ----------------------------------------------------------------- products ---

def operands(rng, rows, E, N, K, extreme=False):
    a = rng.integers(-128, 128, (rows, K), dtype=np.int8)
    w = rng.integers(-128, 128, (E, N, K), dtype=np.int8)
    if extreme:                     # sums of the largest magnitude, of either sign
        a[:], w[:] = -128, -128
        w[:, ::2] = 127
    sa = (rng.random(rows) * np.exp(4 * rng.normal(size=rows))).astype(np.float32)
    sw = (rng.random((E, N)) * 1e-3).astype(np.float32)
    return a, w, sa, sw


def put(*arrays):
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev()) for a in arrays]


DENSE = [(1, 1, 16), (1, 8, 32), (3, 17, 48), (16, 64, 128), (17, 33, 144), (5, 1000, 112), (64, 7168, 2048),
         (33, 576, 7168), (80, 257, 1040), (200, 384, 256), (300, 129, 640), (513, 512, 272), (1000, 130, 4096),
         (1, 4096, 7168), (2049, 1031, 208), (130, 2112, 1552), (4100, 300, 1024), (3000, 2600, 80),
         (2, 24, 32768), (150, 260, 32752), (2304, 2560, 3584)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_gemm_int8(M, N, K):
    rng = np.random.default_rng(M + 3 * N + 7 * K)
    a, w, sa, sw = operands(rng, M, 1, N, K)
    ad, wd, sad, swd = put(a, w[0], sa, sw[0])
    out = torch.full((M + 1, N), 5.0, dtype=torch.bfloat16, device=dev())
    ops.moe_gemm_int8(ad, sad, wd, swd, out=out[:M])
    assert (out[M] == 5.0).all(), "wrote behind the last row"
    np.testing.assert_array_equal(bf16_to_f64(out[:M]), reference(a, sa, w[0], sw[0]))
    assert same_bits(ops.moe_gemm_int8(ad, sad, wd, swd), out[:M].contiguous())


def reference(a, sa, w, sw):
    """O.int8_product, its sum in fp64 (exact: below 2^53) on the GPU where it is large."""
    if a.shape[0] * w.shape[0] * a.shape[1] < 1 << 26:
        return O.int8_product(a, sa, w, sw)
    ad, wd = put(a, w)
    S = (ad.double() @ wd.double().t()).cpu().numpy()
    v = O.fl32(S) * sa.astype(np.float64)[:, None]
    return O.round_bf16(O.fl32(O.fl32(v) * sw.astype(np.float64)[None, :]))


@pytest.mark.parametrize("M,N,K", [(3, 40, 32768), (300, 260, 32768), (300, 260, 32752), (2304, 2560, 4096)])
def test_gemm_int8_largest_sums(M, N, K):
    """Every product +-2^14 or +-127 128: sums up to 2^29."""
    a, w, sa, sw = operands(np.random.default_rng(1), M, 1, N, K, extreme=True)
    ad, wd, sad, swd = put(a, w[0], sa, sw[0])
    S = np.where(np.arange(N) % 2 == 0, -128 * 127, 128 * 128).astype(np.float64) * K
    want = O.round_bf16(O.fl32(O.fl32(O.fl32(S)[None, :] * sa.astype(np.float64)[:, None]) * sw[0].astype(np.float64)))
    np.testing.assert_array_equal(bf16_to_f64(ops.moe_gemm_int8(ad, sad, wd, swd)), want)


@pytest.mark.parametrize("K", [16, 112, 144, 1008, 1040])
def test_gemm_int8_reads_no_neighbour_behind_a_row(K):
    """K that is no whole number of 128-byte steps: what follows the last row of
    each operand, and the next rows' bytes, stay out of the sums."""
    rng = np.random.default_rng(K)
    for M, N in ((1, 5), (40, 70), (200, 130), (600, 700)):
        a, w, sa, sw = operands(rng, M, 1, N, K)
        bufs = []
        for v in (a, w[0]):
            b = torch.full((v.size + 256,), 127, dtype=torch.int8, device=dev())
            b[:v.size] = torch.from_numpy(v.reshape(-1)).to(dev())
            bufs.append(b[:v.size].view(v.shape))
        out = ops.moe_gemm_int8(bufs[0], *put(sa), bufs[1], *put(sw[0]))
        np.testing.assert_array_equal(bf16_to_f64(out), O.int8_product(a, sa, w[0], sw[0]))


def test_gemm_int8_scales_of_every_size():
    """Scales from the smallest subnormal to infinity; a NaN scale of a row or a
    channel stays there."""
    d = dev()
    sa = np.array([2.0 ** -149, 2.0 ** -126, 1e-20, 1.0, 3e38, np.inf, np.nan, 0.0], dtype=np.float32)
    sw = np.array([2.0 ** -140, 1e-30, 1.0, 3e38, np.inf, np.nan, 0.0, -1.0], dtype=np.float32)
    a, w = np.full((8, 64), 3, dtype=np.int8), np.full((8, 64), 5, dtype=np.int8)
    out = ops.moe_gemm_int8(*put(a, sa, w, sw))
    with np.errstate(all="ignore"):
        v = (np.float32(960) * sa)[:, None] * sw[None, :]
    want = torch.from_numpy(v).bfloat16()
    got = out.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    keep = ~want.isnan()
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))
    del d


GROUPED = [  # group sizes, rows before the first and behind the last group, N, K
    ([1], 0, 0, 16, 128), ([0, 0, 3], 0, 2, 40, 112), ([5, 0, 1, 0, 0, 18], 2, 3, 130, 272),
    ([16, 17, 15, 33], 0, 0, 64, 384), ([64, 1, 0, 65, 129], 1, 0, 257, 256), ([0] * 8, 3, 4, 32, 128),
    ([2, 1] * 40 + [0] * 20, 0, 1, 96, 528), ([300, 0, 7], 0, 0, 512, 256), ([0, 511, 1], 0, 9, 384, 656),
    ([1] * 130, 0, 0, 256, 2048), ([40, 60, 3, 0, 128, 256, 255, 70], 5, 6, 320, 256),
    ([128] * 6, 0, 0, 1000, 400), ([600, 500], 0, 0, 1536, 512), ([2048 + 65, 1025, 0, 1, 768 + 64], 0, 0, 2601, 192),
    ([0] * 700 + [3, 1] * 150 + [0] * 23 + [90], 0, 0, 40, 16),   # the most groups there can be
]


@pytest.mark.parametrize("sizes,head,tail,N,K", GROUPED)
def test_grouped_gemm_int8(sizes, head, tail, N, K):
    rows, E = head + sum(sizes) + tail, len(sizes)
    off = np.concatenate([[head], head + np.cumsum(sizes)]).astype(np.int32)
    a, w, sa, sw = operands(np.random.default_rng(rows * 5 + E), rows, E, N, K)
    ad, wd, sad, swd, offd = put(a, w, sa, sw, off)
    out = torch.full((rows, N), 5.0, dtype=torch.bfloat16, device=dev())
    ops.moe_grouped_gemm(ad, wd, offd, sad, swd, out=out)
    want = np.full((rows, N), 5.0)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            want[lo:hi] = reference(a[lo:hi], sa[lo:hi], w[e], sw[e])
    np.testing.assert_array_equal(bf16_to_f64(out), want)
    again = out.clone()
    ops.moe_grouped_gemm(ad, wd, offd, sad, swd, out=again)
    assert same_bits(again, out)


@pytest.mark.parametrize("E", [1, 3, 4, 5, 63, 64, 65, 255, 256, 257, 260, 1000, 1024])
@pytest.mark.parametrize("N,K,per", [(40, 64, 2), (300, 144, 40)])
def test_grouped_gemm_int8_numbers_of_groups(E, N, K, per):
    """Groups of 0 to 2 per rows, empty ones first, in between and last, in small and
    large tiles, for every number of groups at which the search for a block changes."""
    rng, d, g = np.random.default_rng(E + K), dev(), torch.Generator(device=dev()).manual_seed(E)
    sizes = rng.integers(0, 2 * per + 1, E) * (rng.random(E) < 0.7)
    sizes[E // 2] += 1
    sizes[-1] = 0 if E > 1 else 3
    off = np.concatenate([[3], 3 + np.cumsum(sizes)]).astype(np.int32)
    rows = int(off[-1]) + 5
    a = torch.randint(-128, 128, (rows, K), generator=g, device=d, dtype=torch.int8)
    w = torch.randint(-128, 128, (E, N, K), generator=g, device=d, dtype=torch.int8)
    sa, sw = torch.rand(rows, generator=g, device=d), torch.rand(E, N, generator=g, device=d)
    out = torch.full((rows, N), 5.0, dtype=torch.bfloat16, device=d)
    ops.moe_grouped_gemm(a, w, torch.from_numpy(off).to(d), sa, sw, out=out)
    assert (out[:3] == 5.0).all() and (out[rows - 5:] == 5.0).all()
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            S = (a[lo:hi].double() @ w[e].double().t()).float()
            assert torch.equal(out[lo:hi], ((S * sa[lo:hi, None]) * sw[e]).bfloat16()), e


@pytest.mark.parametrize("off", [[-5, 3, 7, 400], [10, 4, 90, 60], [0, 1000, 1000, 2000], [120, 120, 120, 120]])
def test_grouped_int8_bad_offsets_stay_in_bounds(off):
    rows, E, N, K = 100, 3, 200, 240
    ad, wd, sad, swd = put(*operands(np.random.default_rng(5), rows, E, N, K))
    buf = torch.full((rows + 256, N), 5.0, dtype=torch.bfloat16, device=dev())
    ops.moe_grouped_gemm(ad, wd, torch.tensor(off, dtype=torch.int32, device=dev()), sad, swd,
                         out=buf[128: 128 + rows])
    torch.cuda.synchronize()
    assert (buf[:128] == 5.0).all() and (buf[128 + rows:] == 5.0).all()


def test_beyond_32_bits():
    """Rows, codes and outputs past 2^32 elements and weights past 2^32 bytes."""
    d, last, cols = dev(), 3, 8192
    rows = 2 ** 32 // cols + 1029
    g = torch.Generator().manual_seed(32)
    tail = torch.randn(last, cols, generator=g).bfloat16()
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=d)
    x[-last:] = tail.to(d)
    codes, scales = ops.moe_quant_act_int8(x)
    c, s = O.quant_int8(bf16_to_f64(tail))
    np.testing.assert_array_equal(codes[-last:].cpu().numpy(), c)
    np.testing.assert_array_equal(scales[-last:].cpu().numpy(), s.astype(np.float32))
    assert not codes[:-last].any()
    h = x.view(rows // 1, cols)
    half, hs = ops.moe_silu_mul_int8(h)
    c2, s2 = O.quant_int8(O.silu_mul(bf16_to_f64(tail)))
    np.testing.assert_array_equal(half[-last:].cpu().numpy(), c2)
    np.testing.assert_array_equal(hs[-last:].cpu().numpy(), s2.astype(np.float32))
    del x, h, half
    # the codes as rows of a product: a past 2^32 bytes
    big = codes.view(-1, 256)
    n = big.shape[0]
    rng = np.random.default_rng(3)
    _, w, _, sw = operands(rng, 1, 2, 40, 256)
    wd, swd = put(w, sw)
    one = torch.ones(n, device=d)
    off = torch.tensor([5, n - 70, n], dtype=torch.int32, device=d)
    at = big[-70:].cpu().numpy()
    out = ops.moe_grouped_gemm(big, wd, off, one, swd)
    np.testing.assert_array_equal(bf16_to_f64(out[-70:]), O.int8_product(at, np.ones(70), w[1], sw[1]))
    out = ops.moe_gemm_int8(big, one, wd[1].contiguous(), swd[1].contiguous())
    np.testing.assert_array_equal(bf16_to_f64(out[-70:]), O.int8_product(at, np.ones(70), w[1], sw[1]))
    del codes, big, one, out
    # outputs past 2^32 elements, and weights past 2^32 bytes
    rows, N, K = 2 ** 32 // 4096 + 517, 4096, 64
    a = torch.zeros(rows, K, dtype=torch.int8, device=d)
    t, w, _, sw = operands(rng, 300, 1, N, K)
    a[-300:] = torch.from_numpy(t).to(d)
    out = ops.moe_gemm_int8(a, torch.ones(rows, device=d), *put(w[0], sw[0]))
    np.testing.assert_array_equal(bf16_to_f64(out[-300:]), reference(t, np.ones(300, np.float32), w[0], sw[0]))
    del out, a
    E, N, K = 600, 4096, 2048
    wl = torch.zeros(E, N, K, dtype=torch.int8, device=d)
    t, w, sa, _ = operands(rng, 20, 1, N, K)
    wl[-1] = torch.from_numpy(w[0]).to(d)
    sw = np.ones((E, N), dtype=np.float32)
    off = torch.tensor([0] * (E - 1) + [4, 20], dtype=torch.int32, device=d)
    out = ops.moe_grouped_gemm(*put(t), wl, off, *put(sa, sw))
    np.testing.assert_array_equal(bf16_to_f64(out[4:]), reference(t[4:], sa[4:], w[0], sw[0]))
    assert not out[:4].any()


# ------------------------------------------------- together, as a user would ---

def int8_weights(rng, E, N, K):
    """Expert weights as int8 with a scale per output channel, and their values."""
    w = rng.normal(size=(E, N, K)) / np.sqrt(K)
    s = (np.abs(w).max(-1) / 127).astype(np.float32)
    q = np.rint(w / s[..., None]).clip(-127, 127).astype(np.int8)
    return q, s


def layer_state(seed, T=70, H=384, I=208, E=6, k=3, away=False):
    rng = np.random.default_rng(seed)
    w13, s13 = int8_weights(rng, E, 2 * I, H)
    w2, s2 = int8_weights(rng, E, H, I)
    ids = np.stack([rng.permutation(E + (2 if away else 0))[:k] for _ in range(T)]).astype(np.int32)
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32))
    st = dict(zip(("w13", "s13", "w2", "s2", "ids"), put(w13, s13, w2, s2, ids)))
    d = dev()
    st |= dict(x=x.to(d), w=w.to(d), E=E, host=(x, ids, w, w13, s13, w2, s2))
    R = T * k
    st |= dict(rows=torch.zeros(R, H, dtype=torch.int8, device=d), rs=torch.zeros(R, device=d),
               off=torch.zeros(E + 1, dtype=torch.int32, device=d), inv=torch.zeros(T, k, dtype=torch.int32, device=d),
               h=torch.zeros(R, 2 * I, dtype=torch.bfloat16, device=d), c2=torch.zeros(R, I, dtype=torch.int8, device=d),
               cs=torch.zeros(R, device=d), y=torch.zeros(R, H, dtype=torch.bfloat16, device=d),
               out=torch.zeros(T, H, dtype=torch.bfloat16, device=d),
               scratch=torch.zeros(max(ops.moe_sort_scratch_bytes(T, k, E), 4), dtype=torch.uint8, device=d))
    return st


def layer(st):
    """An int8 expert layer from the operators, on one set of buffers."""
    ops.moe_sort_rows(st["x"], st["ids"], st["E"], quant="int8", rows=st["rows"], scales=st["rs"], offsets=st["off"],
                      inv=st["inv"], scratch=st["scratch"])
    ops.moe_grouped_gemm(st["rows"], st["w13"], st["off"], st["rs"], st["s13"], out=st["h"])
    ops.moe_silu_mul_int8(st["h"], codes=st["c2"], scales=st["cs"])
    ops.moe_grouped_gemm(st["c2"], st["w2"], st["off"], st["cs"], st["s2"], out=st["y"])
    ops.moe_combine_rows(st["y"], st["inv"], st["w"], out=st["out"])


OUTPUTS = ("rows", "rs", "off", "inv", "h", "c2", "cs", "y", "out")


@pytest.mark.parametrize("away", [False, True])
def test_int8_layer(away):
    """Each step against the definition, bit for bit up to the combine."""
    st = layer_state(3, away=away)
    layer(st)
    x, ids, w, w13, s13, w2, s2 = st["host"]
    off, inv, token = O.sort_slots(ids, st["E"])
    n = int(off[-1])
    c, s = O.quant_int8(bf16_to_f64(x))
    np.testing.assert_array_equal(st["rows"].cpu().numpy()[:n], c[token])
    h = O.int8_grouped_product(c[token], s[token], w13, s13, off)
    np.testing.assert_array_equal(bf16_to_f64(st["h"])[:n], h)
    c2, cs = O.quant_int8(O.silu_mul(h))
    np.testing.assert_array_equal(st["c2"].cpu().numpy()[:n], c2)
    y = O.int8_grouped_product(c2, cs, w2, s2, off)
    np.testing.assert_array_equal(bf16_to_f64(st["y"])[:n], y)
    ref, size = O.combine_rows(y, inv, w.numpy())
    tol = (2.0 ** -8 * np.abs(ref) + 2.0 ** -24 * (ids.shape[1] + 1) * size) * (1 + 2.0 ** -8)
    assert (np.abs(bf16_to_f64(st["out"]) - ref) <= tol).all()


@pytest.mark.parametrize("T", [40, 1500])
def test_captured_layer_replays(T):
    """The layer in a captured graph, replayed on new inputs with eager work of
    the same operators between the replays."""
    st, other = layer_state(1, T=T), layer_state(2, T=T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(st)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(st)
    for seed in (1, 3, 4):
        new = layer_state(seed, T=T)
        for name in ("x", "ids", "w", "w13", "s13", "w2", "s2"):
            st[name].copy_(new[name])
        st["out"].zero_()
        layer(other)
        graph.replay()
        layer(new)
        torch.cuda.synchronize()
        for name in OUTPUTS:
            assert same_bits(st[name], new[name]), (seed, name)


def test_two_threads_at_once():
    """Layers from two threads, each on a stream of its own with its own buffers."""
    states = [layer_state(s, T=800) for s in (7, 8)]
    want = []
    for st in states:
        layer(st)
        want.append([st[name].clone() for name in OUTPUTS])
        for name in OUTPUTS:
            st[name].zero_()
    torch.cuda.synchronize()
    failed = []

    def work(st, s):
        try:
            with torch.cuda.stream(s):
                for _ in range(20):
                    layer(st)
        except Exception as e:   # noqa: BLE001 - reported by the test
            failed.append(e)

    threads = [threading.Thread(target=work, args=(st, torch.cuda.Stream())) for st in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for st, kept in zip(states, want):
        for name, v in zip(OUTPUTS, kept):
            assert same_bits(st[name], v), name


def test_bf16_layer_and_its_gradient():
    """Sort, grouped bf16 products and combine forward, and the gradients of x and
    of the router's weights back through them (the products' own gradient with
    the transposed weights), against 64-bit arithmetic on the same roundings.

    Each bf16 product is off by 2^-8 of its value and 2^-24 (K / 32 + 16) of its
    sum of magnitudes; the combine by its rule; a gradient of x takes both."""
    rng, d = np.random.default_rng(11), dev()
    T, k, E, H, N = 90, 2, 5, 128, 192
    ids = routing_ids(rng, T, k, E)
    x, w = torch.from_numpy(rng.normal(size=(T, H))).bfloat16(), rng.random((T, k)).astype(np.float32)
    W = torch.from_numpy(rng.normal(size=(E, N, H)) / np.sqrt(H)).bfloat16()
    grad = torch.from_numpy(rng.normal(size=(T, N))).bfloat16()
    xd, idd, wd, Wd, gd = x.to(d), torch.from_numpy(ids).to(d), torch.from_numpy(w).to(d), W.to(d), grad.to(d)
    rows, _, off, inv = ops.moe_sort_rows(xd, idd, E)
    y = ops.moe_grouped_gemm(rows, Wd, off)
    out = ops.moe_combine_rows(y, inv, wd)
    g_y, g_w = ops.moe_combine_rows_bwd(gd, inv, rows=y, weights=wd)
    g_rows = ops.moe_grouped_gemm(g_y, Wd.transpose(1, 2).contiguous(), off)
    g_x = ops.moe_combine_rows(g_rows, inv)

    x64, W64, g64 = bf16_to_f64(x), bf16_to_f64(W), bf16_to_f64(grad)
    half, tiny = 2.0 ** -8 * 1.01, 2.0 ** -24 * 64
    for t in range(T):
        o, o_tol, gx, gx_tol = 0.0, 0.0, 0.0, 0.0
        for j in range(k):
            e = ids[t, j]
            yj = W64[e] @ x64[t]
            y_tol = half * np.abs(yj) + tiny * (np.abs(W64[e]) @ np.abs(x64[t]))
            o, o_tol = o + w[t, j] * yj, o_tol + w[t, j] * y_tol + tiny * w[t, j] * np.abs(yj)
            want_w = np.sum(g64[t] * yj)
            assert abs(float(g_w[t, j]) - want_w) <= np.sum(np.abs(g64[t]) * (y_tol + 2.0 ** -24 * N * np.abs(yj)) * 1.01)
            gy = w[t, j] * g64[t]
            gr = W64[e].T @ gy
            mag = np.abs(W64[e]).T @ np.abs(gy)
            gx, gx_tol = gx + gr, gx_tol + half * mag + half * np.abs(gr) + half * half * mag + tiny * mag
        assert (np.abs(bf16_to_f64(out[t]) - o) <= half * np.abs(o) + (1 + half) * o_tol).all()
        assert (np.abs(bf16_to_f64(g_x[t]) - gx) <= half * np.abs(gx) + (1 + half) * gx_tol).all()


def routing_ids(rng, T, k, E):
    return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)


def test_bf16_chain_matches_the_fused_layer():
    """Sorted rows through grouped products, the gated multiply and the combine
    against moe_forward on the same layer; both are within tau of its definition."""
    from gpu_util import TAU, bits_to_bf16, layer_for, routing
    from moe_layer_amd.workloads import CONFIGS, Workload
    cfg = CONFIGS["tiny"]
    lay, (ids, tw, _) = layer_for(cfg), routing(cfg)
    lay.ensure(range(cfg.E))
    d = dev()
    x = bits_to_bf16(Workload(cfg).x_bf16_bits()).to(d)
    ids_t, tw_t = torch.from_numpy(ids.astype(np.int32)).to(d), torch.from_numpy(tw.astype(np.float32)).to(d)
    ref, _ = ops.moe_forward(x, lay.w13, lay.w2, ids_t, tw_t)
    rows, _, off, inv = ops.moe_sort_rows(x, ids_t, cfg.E)
    a, _, _ = ops.moe_silu_mul(ops.moe_grouped_gemm(rows, lay.w13, off))
    out = ops.moe_combine_rows(ops.moe_grouped_gemm(a, lay.w2, off), inv, tw_t)
    o = ref.double()
    err = float((out.double() - o).abs().max() / o.square().mean().sqrt())
    log(f"sorted chain: {err:.2e} of the layer's RMS")
    assert err <= 2 * TAU["bf16"]


def test_empty_calls():
    d = dev()
    e = lambda *s, t=torch.int8: torch.empty(*s, dtype=t, device=d)   # noqa: E731
    f = torch.float32
    assert ops.moe_quant_act_int8(e(0, 64, t=torch.bfloat16))[0].shape == (0, 64)
    assert ops.moe_silu_mul_int8(e(0, 64, t=torch.bfloat16))[0].shape == (0, 32)
    assert ops.moe_gemm_int8(e(0, 64), e(0, t=f), e(5, 64), e(5, t=f)).shape == (0, 5)
    off = torch.zeros(3, dtype=torch.int32, device=d)
    assert ops.moe_grouped_gemm(e(0, 64), e(2, 8, 64), off, e(0, t=f), e(2, 8, t=f)).shape == (0, 8)
