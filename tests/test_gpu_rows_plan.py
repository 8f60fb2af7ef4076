"""Every kernel of the dense and grouped products, bit for bit: operands whose
partial sums are exact fp32 values in every order (|a| |w| <= 105, or 21 where K
is above 2304, and scales of four neighbouring powers of two on either side: at
most 2^24 of the smallest unit), against 64-bit products on the same device."""
import numpy as np
import pytest
import torch

from moe_layer_amd import ops

from gpu_util import dev
from rows_plan_cases import KERNELS, planned
from test_gpu_rows import sizes_to_offsets

pytestmark = pytest.mark.gpu


def values(codes, scales, span):
    """fp64 values of codes [n, K] with scales [ceil(n / span), K / 128]."""
    v = codes.double()
    if scales is None:
        return v
    return v * scales.double().repeat_interleave(128, 1).repeat_interleave(span, 0)[: v.shape[0]]


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_kernel(kernel):
    fp8 = kernel[0]
    rows, E, N, K = KERNELS[kernel]
    assert planned(ops, fp8, rows, E, N, K) == kernel
    ma, mw = (7, 15) if K <= 2304 else (3, 7)
    assert ma * mw * K * 64 < 2 ** 24
    d, groups, nb = dev(), max(E, 1), -(-N // 128)
    g = torch.Generator(device=d).manual_seed(rows + N + K)

    def whole(most, *shape):
        v = torch.randint(-most, most + 1, shape, generator=g, device=d, dtype=torch.int8)
        return v.float().to(torch.float8_e4m3fn) if fp8 else v.bfloat16()

    def pow2(lo, hi, *shape):
        return torch.exp2(torch.randint(lo, hi + 1, shape, generator=g, device=d).float()) if fp8 else None

    a, w = whole(ma, rows, K), whole(mw, groups, N, K)
    sa, sw = pow2(-2, 1, rows, K // 128), pow2(-1, 2, groups, nb, K // 128)
    if E == 0:
        off = np.array([0, rows])
        call = lambda out: ops.moe_gemm_fp8(a, sa, w[0], sw[0], out=out)   # noqa: E731
    else:
        rng = np.random.default_rng(rows)
        load = rng.exponential(size=E) ** 2
        off = sizes_to_offsets(rng.multinomial(rows, load / load.sum()))
        offd = torch.from_numpy(off).to(d)
        call = lambda out: ops.moe_grouped_gemm(a, w, offd, sa, sw, out=out)   # noqa: E731
    buf = torch.full((rows + 1, N), 5.0, dtype=torch.bfloat16, device=d)
    call(buf[:rows])
    assert (buf[rows] == 5.0).all(), "wrote behind the last row"
    for e in range(groups):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            ref = values(a[lo:hi], None if sa is None else sa[lo:hi], 1) @ \
                values(w[e], None if sw is None else sw[e], 128).t().contiguous()
            assert torch.equal(buf[lo:hi], ref.float().bfloat16()), (e, lo, hi)   # (the sums are exact in fp32)
    again = torch.full((rows + 1, N), 7.0, dtype=torch.bfloat16, device=d)
    call(again[:rows])
    assert torch.equal(again[:rows], buf[:rows]), "a second call differs"
