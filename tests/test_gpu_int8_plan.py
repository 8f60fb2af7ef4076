"""Every int8 kernel on the GPU, bit for bit: full-range codes, groups of uneven
sizes, rows outside of every group, operands that end where their buffers end."""
import numpy as np
import pytest
import torch

import oracle as O
from moe_layer_amd import ops

from gpu_util import dev
from int8_plan_cases import KERNELS, planned

pytestmark = pytest.mark.gpu


def exact(a, sa, w, sw):
    """bf16(fl32(fl32(S) sa) sw) with S summed exactly (fp64 on the GPU)."""
    S = (a.double() @ w.double().t()).float()
    return ((S * sa[:, None]) * sw).bfloat16()


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_kernel(kernel):
    rows, E, N, K = KERNELS[kernel]
    assert planned(ops, rows, E, N, K) == kernel
    d, g = dev(), torch.Generator(device=dev()).manual_seed(rows + N)
    a = torch.randint(-128, 128, (rows, K), generator=g, device=d, dtype=torch.int8)
    w = torch.randint(-128, 128, (max(E, 1), N, K), generator=g, device=d, dtype=torch.int8)
    sa, sw = torch.rand(rows, generator=g, device=d), torch.rand(max(E, 1), N, generator=g, device=d)
    buf = torch.full((rows + 2, N), 5.0, dtype=torch.bfloat16, device=d)
    # an output that starts inside a buffer where its rows are whole 16-byte pieces
    inside = (2 * N) % 16 == 0
    out = buf[1: rows + 1] if inside else buf[:rows]
    if E == 0:
        ops.moe_gemm_int8(a, sa, w[0], sw[0], out=out)
        assert torch.equal(out, exact(a, sa, w[0], sw[0]))
    else:
        rng = np.random.default_rng(E)
        load = rng.exponential(size=E) ** 2
        sizes = rng.multinomial(rows - rows // 10, load / load.sum())
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + rows // 20
        ops.moe_grouped_gemm(a, w, torch.from_numpy(off).to(d), sa, sw, out=out)
        assert (out[: off[0]] == 5.0).all() and (out[off[-1]:] == 5.0).all()
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            if hi > lo:
                assert torch.equal(out[lo:hi], exact(a[lo:hi], sa[lo:hi], w[e], sw[e])), (e, lo, hi)
    assert (buf[rows + 1:] == 5.0).all() and (not inside or (buf[0] == 5.0).all())


def test_definition_is_the_oracles():
    """exact() here against the NumPy definition."""
    d, g = dev(), torch.Generator(device=dev()).manual_seed(1)
    a = torch.randint(-128, 128, (40, 208), generator=g, device=d, dtype=torch.int8)
    w = torch.randint(-128, 128, (30, 208), generator=g, device=d, dtype=torch.int8)
    sa, sw = torch.rand(40, generator=g, device=d), torch.rand(30, generator=g, device=d)
    want = O.int8_product(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy())
    np.testing.assert_array_equal(exact(a, sa, w, sw).double().cpu().numpy(), want)


@pytest.mark.parametrize("blocks", [[256], [64], [65, 128, 129, 255], [1, 63, 64, 127, 192, 193, 257, 384]])
@pytest.mark.parametrize("K", [16, 128, 144, 256, 272, 384, 400, 1024])
def test_last_blocks_of_every_width(blocks, K):
    """The large tiles at one to eight stages, whole and in part, and last blocks of
    every width class, with weight rows that end inside a tile."""
    E, N = 8, 2601
    sizes = [(768 if K > 128 else 2048) + b for b in (blocks * 8)[:E]]
    rows = sum(sizes)
    d, g = dev(), torch.Generator(device=dev()).manual_seed(K)
    a = torch.randint(-128, 128, (rows, K), generator=g, device=d, dtype=torch.int8)
    w = torch.randint(-128, 128, (E, N, K), generator=g, device=d, dtype=torch.int8)
    sa, sw = torch.rand(rows, generator=g, device=d), torch.rand(E, N, generator=g, device=d)
    off = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int32, device=d)
    out = ops.moe_grouped_gemm(a, w, off, sa, sw)
    lo = 0
    for e, n in enumerate(sizes):
        assert torch.equal(out[lo: lo + n], exact(a[lo: lo + n], sa[lo: lo + n], w[e], sw[e])), e
        lo += n
