"""Outputs of the large product tiles wherever they start: rows that are whole
lines are stored past the caches' replacement, others are not, with the same bits
and nothing beside them written."""
import pytest
import torch

from moe_layer_amd import ops

from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("rows,N,K", [(3000, 2048, 512), (3000, 2056, 512), (2900, 2051, 512)])
def test_outputs_on_and_off_a_line(kind, rows, N, K):
    d, g = dev(), torch.Generator().manual_seed(N)
    offsets = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device=d)
    if kind == "bf16":
        a, w = torch.randn(rows, K, generator=g).bfloat16().to(d), torch.randn(2, N, K, generator=g).bfloat16().to(d)
        sa = sw = None
    elif kind == "fp8":
        a = torch.randint(0, 112, (rows, K), generator=g, dtype=torch.uint8).to(d)
        w = torch.randint(0, 112, (2, N, K), generator=g, dtype=torch.uint8).to(d)
        sa, sw = torch.rand(rows, K // 128, generator=g).to(d), torch.rand(2, -(-N // 128), K // 128, generator=g).to(d)
    else:
        a = torch.randint(-128, 128, (rows, K), generator=g, dtype=torch.int8).to(d)
        w = torch.randint(-128, 128, (2, N, K), generator=g, dtype=torch.int8).to(d)
        sa, sw = torch.rand(rows, generator=g).to(d), torch.rand(2, N, generator=g).to(d)
    wdtype = {"bf16": ops.MOE_WDTYPE_BF16, "fp8": ops.MOE_WDTYPE_FP8_E4M3, "int8": ops.MOE_WDTYPE_INT8}[kind]
    assert ops.moe_gemm_plan(rows, N, K, E=2, wdtype=wdtype)["block_cols"] == 256
    got = []
    for off in (0, 8, 32):                                 # 0, 16 and 64 bytes behind a line's start
        buf = torch.full((64 + rows * N + 64,), 5.0, dtype=torch.bfloat16, device=d)
        lead = -(buf.data_ptr() // 2) % 64 + off
        out = buf[lead: lead + rows * N].view(rows, N)
        got.append(ops.moe_grouped_gemm(a, w, offsets, sa, sw, out=out).clone())
        assert (buf[:lead] == 5.0).all() and (buf[lead + rows * N:] == 5.0).all()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    if kind == "int8":                                     # exact sums: the same bits from another tile and other stores
        few = ops.moe_gemm_int8(a[:7].contiguous(), sa[:7].contiguous(), w[0], sw[0])
        assert torch.equal(few, got[0][:7])
