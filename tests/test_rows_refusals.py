"""What the operators around the layer refuse, on the host: every call here
fails validation (or has no rows) before any device work."""
import ctypes as C

import pytest
import torch

from moe_layer_amd import ops

FAKE = 0x7f0000000000
GAP = 1 << 36                      # between fake buffers
OK, BAD, NOT = ops.MOE_OK, ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED


def P(i):
    return C.c_void_p(FAKE + i * GAP)


def norm(**kw):
    a = dict(x=P(0), residual=P(1), weight=P(2), eps=1e-6, rows=4, cols=256, quant=1, residual_out=P(3), y=P(4),
             codes=P(5), scales=P(6)) | kw
    return ops.lib().moe_rmsnorm(a["x"], a["residual"], a["weight"], a["eps"], a["rows"], a["cols"], a["quant"],
                                 a["residual_out"], a["y"], a["codes"], a["scales"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(cols=-128), BAD), (dict(quant=3), BAD), (dict(quant=-1), BAD),
    (dict(eps=-1e-6), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(cols=264), NOT), (dict(cols=264, quant=2), NOT), (dict(cols=260, quant=0, codes=None, scales=None), NOT),
    (dict(cols=32768 + 128), NOT),
    (dict(x=None), BAD), (dict(weight=None), BAD), (dict(codes=None), BAD), (dict(scales=None), BAD),
    (dict(quant=0), BAD),                                           # codes without a format
    (dict(quant=0, codes=None, scales=None, y=None, residual_out=None), BAD),   # no output
    (dict(residual=None), BAD),                                     # residual_out without a residual
    (dict(x=C.c_void_p(FAKE + 8)), BAD), (dict(y=C.c_void_p(FAKE + 4 * GAP + 2)), BAD),
    (dict(scales=C.c_void_p(FAKE + 6 * GAP + 2)), BAD),
    (dict(y=P(3)), BAD),                                            # two outputs in one place
    (dict(y=C.c_void_p(FAKE + 16)), BAD),                           # over a part of x
    (dict(codes=P(0)), BAD), (dict(scales=P(2)), BAD), (dict(residual_out=P(2)), BAD),
    (dict(rows=0, x=None, weight=None), OK),
])
def test_rmsnorm(kw, status):
    assert norm(**kw) == status


def act(**kw):
    a = dict(h=P(0), rows=4, cols=256, limit=0.0, quant=1, y=P(1), codes=P(2), scales=P(3)) | kw
    return ops.lib().moe_silu_mul(a["h"], a["rows"], a["cols"], a["limit"], a["quant"], a["y"], a["codes"],
                                  a["scales"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(quant=5), BAD), (dict(limit=-1.0), BAD),
    (dict(limit=float("nan")), BAD), (dict(cols=192), NOT), (dict(cols=48, quant=2), NOT),
    (dict(cols=12, quant=0, codes=None, scales=None), NOT), (dict(cols=(1 << 20) + 128), NOT),
    (dict(h=None), BAD), (dict(quant=0, y=None, codes=None, scales=None), BAD), (dict(codes=None), BAD),
    (dict(h=C.c_void_p(FAKE + 4)), BAD), (dict(y=P(0)), BAD), (dict(codes=C.c_void_p(FAKE + 2048)), BAD),
    (dict(rows=0, h=None), OK),
])
def test_silu_mul(kw, status):
    assert act(**kw) == status


def dense(**kw):
    a = dict(a=P(0), sa=P(1), w=P(2), sw=P(3), M=4, N=256, K=256, out=P(4)) | kw
    return ops.lib().moe_gemm_fp8(a["a"], a["sa"], a["w"], a["sw"], a["M"], a["N"], a["K"], a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=192), NOT), (dict(K=(1 << 20) + 128), NOT),
    (dict(M=(1 << 30) + 1), NOT), (dict(N=(1 << 30) + 1), NOT),
    (dict(a=None), BAD), (dict(sa=None), BAD), (dict(w=None), BAD), (dict(sw=None), BAD), (dict(out=None), BAD),
    (dict(a=C.c_void_p(FAKE + 8)), BAD), (dict(sa=C.c_void_p(FAKE + GAP + 2)), BAD), (dict(out=P(0)), BAD),
    (dict(out=P(2)), BAD), (dict(M=0, a=None, out=None), OK),
])
def test_gemm_fp8(kw, status):
    assert dense(**kw) == status


def grouped(**kw):
    a = dict(a=P(0), sa=P(1), w=P(2), sw=P(3), off=P(4), rows=4, E=3, N=256, K=256, wd=1, out=P(5)) | kw
    return ops.lib().moe_grouped_gemm(a["a"], a["sa"], a["w"], a["sw"], a["off"], a["rows"], a["E"], a["N"], a["K"],
                                      a["wd"], a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(E=0), BAD), (dict(E=1025), BAD), (dict(N=0), BAD), (dict(K=0), BAD),
    (dict(wd=2), NOT), (dict(wd=3), BAD), (dict(K=192), NOT), (dict(K=96, wd=0, sa=None, sw=None), NOT),
    (dict(rows=(1 << 30) + 1), NOT), (dict(N=(1 << 30) + 1), NOT), (dict(K=1 << 21), NOT),
    (dict(a=None), BAD), (dict(off=None), BAD), (dict(sa=None), BAD), (dict(wd=0), BAD),   # scales with bf16
    (dict(off=C.c_void_p(FAKE + 4 * GAP + 2)), BAD), (dict(out=P(2)), BAD), (dict(out=P(4)), BAD),
    (dict(rows=0, a=None, off=None), OK),
])
def test_grouped_gemm(kw, status):
    assert grouped(**kw) == status


def test_binding_checks():
    """The binding refuses wrong types, shapes, layouts and combinations
    before it calls the library."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)   # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)      # noqa: E731
    f32 = torch.zeros
    for call in (
            lambda: ops.moe_rmsnorm(f32(2, 256), bf(256)),
            lambda: ops.moe_rmsnorm(bf(2, 256), bf(128)),
            lambda: ops.moe_rmsnorm(bf(256, 2).t(), bf(256)),
            lambda: ops.moe_rmsnorm(bf(2, 256), bf(256), quant="fp4"),
            lambda: ops.moe_rmsnorm(bf(2, 256), bf(256), residual=bf(1, 256)),
            lambda: ops.moe_rmsnorm(bf(2, 256), bf(256), residual_out=bf(2, 256)),
            lambda: ops.moe_rmsnorm(bf(2, 256), bf(256), codes=u8(2, 256)),
            lambda: ops.moe_rmsnorm(bf(2, 256), bf(256), quant="mxfp8", scales=f32(2, 2)),
            lambda: ops.moe_rmsnorm(bf(2, 256), bf(256), y=bf(2, 256), with_y=False),
            lambda: ops.moe_silu_mul(bf(2, 255)),
            lambda: ops.moe_silu_mul(bf(2, 256), quant="fp8", codes=u8(2, 256)),
            lambda: ops.moe_gemm_fp8(bf(2, 256), f32(2, 2), u8(8, 256), f32(1, 2)),
            lambda: ops.moe_gemm_fp8(u8(2, 256), f32(2, 1), u8(8, 256), f32(1, 2)),
            lambda: ops.moe_gemm_fp8(u8(2, 256), f32(2, 2), u8(8, 128), f32(1, 2)),
            lambda: ops.moe_gemm_fp8(u8(2, 256), f32(2, 2), u8(130, 256), f32(1, 2)),
            lambda: ops.moe_gemm_fp8(u8(2, 256), f32(2, 2), u8(8, 256), f32(1, 2), out=bf(8, 2)),
            lambda: ops.moe_grouped_gemm(bf(2, 64), bf(3, 8, 64), torch.zeros(4, dtype=torch.int64)),
            lambda: ops.moe_grouped_gemm(bf(2, 64), bf(3, 8, 64), torch.zeros(3, dtype=torch.int32)),
            lambda: ops.moe_grouped_gemm(bf(2, 64), u8(3, 8, 64), torch.zeros(4, dtype=torch.int32)),
            lambda: ops.moe_grouped_gemm(u8(2, 128), u8(3, 8, 128), torch.zeros(4, dtype=torch.int32)),
            lambda: ops.moe_grouped_gemm(bf(2, 64), bf(3, 8, 64), torch.zeros(4, dtype=torch.int32), f32(2, 1)),
            lambda: ops.moe_rmsnorm(None, bf(256)),
            lambda: ops.moe_gemm_fp8([[1.0]], f32(2, 2), u8(8, 256), f32(1, 2)),
            lambda: ops.moe_gemm_fp8(u8(2, 256), None, u8(8, 256), f32(1, 2)),
            # right but for the device
            lambda: ops.moe_rmsnorm(bf(2, 256), bf(256)),
            lambda: ops.moe_silu_mul(bf(2, 256), quant="fp8"),
            lambda: ops.moe_gemm_fp8(u8(2, 256), f32(2, 2), u8(8, 256), f32(1, 2)),
            lambda: ops.moe_grouped_gemm(bf(2, 64), bf(3, 8, 64), torch.zeros(4, dtype=torch.int32)),
    ):
        with pytest.raises(AssertionError):
            call()
