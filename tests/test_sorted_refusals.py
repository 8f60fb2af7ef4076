"""What the operators that sort a batch by expert, bring it back and run it in
8-bit integers refuse, on the host: every call here fails validation (or has
nothing to do) before any device work."""
import ctypes as C

import pytest
import torch

from moe_layer_amd import ops

from test_rows_refusals import BAD, FAKE, GAP, NOT, OK, P

WS = ops.MOE_ERR_WORKSPACE
BF16, FP8, MX, INT8 = ops.MOE_WDTYPE_BF16, ops.MOE_WDTYPE_FP8_E4M3, ops.MOE_WDTYPE_MXFP8, ops.MOE_WDTYPE_INT8


def sort(**kw):
    a = dict(x=P(0), xs=None, ids=P(1), T=4, topk=2, E=8, cols=256, xt=BF16, rt=BF16, rows=P(2), rs=None, off=P(3),
             inv=P(4), scratch=None, room=0) | kw
    return ops.lib().moe_sort_rows(a["x"], a["xs"], a["ids"], a["T"], a["topk"], a["E"], a["cols"], a["xt"], a["rt"],
                                   a["rows"], a["rs"], a["off"], a["inv"], a["scratch"], a["room"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(topk=0), BAD), (dict(topk=65), BAD), (dict(E=0), BAD), (dict(E=1025), BAD),
    (dict(cols=0), BAD), (dict(cols=-8), BAD), (dict(cols=4), NOT), (dict(cols=(1 << 20) + 8), NOT),
    (dict(xt=MX), NOT), (dict(rt=MX), NOT), (dict(xt=3), BAD), (dict(rt=7), BAD), (dict(xt=-1), BAD),
    (dict(xt=FP8, xs=P(5)), BAD), (dict(xt=INT8, xs=P(5), rt=FP8, rs=P(6)), BAD),     # codes to another format
    (dict(rt=FP8, rs=P(6), cols=192), NOT), (dict(rt=INT8, rs=P(6), cols=264), NOT),
    (dict(rt=INT8, rs=P(6), cols=32768 + 16), NOT),
    (dict(T=(1 << 30) // 2 + 1), NOT), (dict(T=2 ** 31 - 1, topk=64), NOT),
    (dict(x=None), BAD), (dict(ids=None), BAD), (dict(rows=None), BAD), (dict(off=None), BAD), (dict(inv=None), BAD),
    (dict(rt=FP8), BAD), (dict(rt=INT8), BAD), (dict(rs=P(6)), BAD), (dict(xs=P(5)), BAD),
    (dict(xt=FP8, rt=FP8, rs=P(6)), BAD), (dict(xt=INT8, rt=INT8, xs=P(5)), BAD),
    (dict(x=C.c_void_p(FAKE + 8)), BAD), (dict(rows=C.c_void_p(FAKE + 2 * GAP + 8)), BAD),
    (dict(inv=C.c_void_p(FAKE + 4 * GAP + 2)), BAD), (dict(off=C.c_void_p(FAKE + 3 * GAP + 1)), BAD),
    (dict(rt=INT8, rs=C.c_void_p(FAKE + 6 * GAP + 2)), BAD),
    (dict(rows=P(0)), BAD), (dict(rows=C.c_void_p(FAKE + 4 * 512 - 16)), BAD), (dict(inv=P(1)), BAD),
    (dict(off=P(4)), BAD), (dict(rt=INT8, rs=P(3)), BAD), (dict(rows=P(4)), BAD),
    (dict(T=30000), WS), (dict(T=30000, scratch=P(7), room=59 * 8 * 4 - 1), WS),
    (dict(T=30000, scratch=C.c_void_p(FAKE + 7 * GAP + 2), room=1 << 20), WS),
    (dict(T=30000, scratch=P(0), room=1 << 20), BAD), (dict(T=30000, scratch=P(4), room=1 << 20), BAD),
])
def test_sort_rows(kw, status):
    assert sort(**kw) == status


def test_sort_scratch_bytes():
    L = ops.lib()
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 65, 8), (4, 2, 0), (4, 2, 1025)):
        assert L.moe_sort_scratch_bytes(*bad) == BAD
    assert L.moe_sort_scratch_bytes(2 ** 30, 2, 8) == NOT
    assert L.moe_sort_scratch_bytes(0, 8, 64) == 0 and L.moe_sort_scratch_bytes(1, 64, 1024) == 0
    sizes = [L.moe_sort_scratch_bytes(T, 8, 256) for T in (1, 64, 1024, 8192, 10 ** 6, 2 ** 27)]
    assert sizes == sorted(sizes) and max(sizes) <= 256 * 256 * 4
    with pytest.raises(ops.MoeError):
        ops.moe_sort_scratch_bytes(4, 65, 8)


def combine(**kw):
    a = dict(rows=P(0), inv=P(1), w=P(2), T=4, topk=2, cols=256, num=8, out=P(3)) | kw
    return ops.lib().moe_combine_rows(a["rows"], a["inv"], a["w"], a["T"], a["topk"], a["cols"], a["num"], a["out"], None)


def combine_bwd(**kw):
    a = dict(g=P(0), rows=P(1), inv=P(2), w=P(3), T=4, topk=2, cols=256, num=8, gr=P(4), gw=P(5)) | kw
    return ops.lib().moe_combine_rows_bwd(a["g"], a["rows"], a["inv"], a["w"], a["T"], a["topk"], a["cols"], a["num"],
                                          a["gr"], a["gw"], None)


SIZES = [(dict(T=-1), BAD), (dict(topk=0), BAD), (dict(topk=65), BAD), (dict(cols=0), BAD), (dict(num=-1), BAD),
         (dict(cols=12), NOT), (dict(cols=(1 << 20) + 8), NOT), (dict(num=(1 << 30) + 1), NOT),
         (dict(T=1 << 30), NOT), (dict(rows=None), BAD), (dict(inv=None), BAD),
         (dict(rows=C.c_void_p(FAKE + 8)), BAD), (dict(inv=C.c_void_p(FAKE + 2)), BAD),
         (dict(w=C.c_void_p(FAKE + 2)), BAD)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(out=None), BAD), (dict(out=P(0)), BAD), (dict(out=P(1)), BAD), (dict(out=P(2)), BAD),
    (dict(out=C.c_void_p(FAKE + 3 * GAP + 2)), BAD), (dict(out=C.c_void_p(FAKE + 8 * 512 - 16)), BAD),
    (dict(T=0, rows=None, inv=None, out=None), OK),
])
def test_combine_rows(kw, status):
    assert combine(**kw) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(g=None), BAD), (dict(gr=None), BAD), (dict(gw=None), BAD),      # rows without grad_weights
    (dict(gr=P(0)), BAD), (dict(gr=P(1)), BAD), (dict(gr=P(5)), BAD), (dict(gw=P(3)), BAD), (dict(gw=P(2)), BAD),
    (dict(gr=C.c_void_p(FAKE + 4 * GAP + 2)), BAD), (dict(gw=C.c_void_p(FAKE + 5 * GAP + 1)), BAD),
    (dict(T=0, g=None, inv=None, gr=None), OK),
])
def test_combine_rows_bwd(kw, status):
    assert combine_bwd(**kw) == status


def quant(**kw):
    a = dict(x=P(0), rows=4, cols=256, codes=P(1), scales=P(2)) | kw
    return ops.lib().moe_quant_act_int8(a["x"], a["rows"], a["cols"], a["codes"], a["scales"], None)


def act(**kw):
    a = dict(x=P(0), rows=4, cols=256, limit=0.0, codes=P(1), scales=P(2)) | kw
    return ops.lib().moe_silu_mul_int8(a["x"], a["rows"], a["cols"], a["limit"], a["codes"], a["scales"], None)


INT8_ROWS = [(dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(cols=24), NOT), (dict(cols=32768 + 16), NOT),
             (dict(x=None), BAD), (dict(codes=None), BAD), (dict(scales=None), BAD),
             (dict(x=C.c_void_p(FAKE + 8)), BAD), (dict(codes=C.c_void_p(FAKE + GAP + 8)), BAD),
             (dict(scales=C.c_void_p(FAKE + 2 * GAP + 2)), BAD), (dict(codes=P(0)), BAD), (dict(scales=P(1)), BAD),
             (dict(codes=C.c_void_p(FAKE + 4 * 512 - 16)), BAD), (dict(rows=0, x=None, codes=None, scales=None), OK)]


@pytest.mark.parametrize("kw,status", INT8_ROWS)
def test_quant_act_int8(kw, status):
    assert quant(**kw) == status


@pytest.mark.parametrize("kw,status", INT8_ROWS + [
    (dict(limit=-1.0), BAD), (dict(limit=float("nan")), BAD), (dict(codes=C.c_void_p(FAKE + 4 * 1024 - 16)), BAD)])
def test_silu_mul_int8(kw, status):
    assert act(**kw) == status


def dense(**kw):
    a = dict(a=P(0), sa=P(1), w=P(2), sw=P(3), M=4, N=256, K=256, out=P(4)) | kw
    return ops.lib().moe_gemm_int8(a["a"], a["sa"], a["w"], a["sw"], a["M"], a["N"], a["K"], a["out"], None)


def grouped(**kw):
    a = dict(a=P(0), sa=P(1), w=P(2), sw=P(3), off=P(4), rows=4, E=3, N=256, K=256, out=P(5)) | kw
    return ops.lib().moe_grouped_gemm(a["a"], a["sa"], a["w"], a["sw"], a["off"], a["rows"], a["E"], a["N"], a["K"],
                                      INT8, a["out"], None)


PRODUCTS = [(dict(N=0), BAD), (dict(K=0), BAD), (dict(K=24), NOT), (dict(K=32768 + 16), NOT),
            (dict(N=(1 << 30) + 1), NOT), (dict(a=None), BAD), (dict(sa=None), BAD), (dict(w=None), BAD),
            (dict(sw=None), BAD), (dict(out=None), BAD), (dict(a=C.c_void_p(FAKE + 8)), BAD),
            (dict(sw=C.c_void_p(FAKE + 3 * GAP + 2)), BAD), (dict(out=P(0)), BAD), (dict(out=P(1)), BAD),
            (dict(out=P(3)), BAD)]


@pytest.mark.parametrize("kw,status", PRODUCTS + [(dict(M=-1), BAD), (dict(M=(1 << 30) + 1), NOT),
                                                  (dict(M=0, a=None, out=None), OK)])
def test_gemm_int8(kw, status):
    assert dense(**kw) == status


@pytest.mark.parametrize("kw,status", PRODUCTS + [
    (dict(rows=-1), BAD), (dict(E=0), BAD), (dict(E=1025), BAD), (dict(off=None), BAD), (dict(out=P(4)), BAD),
    # the weights' scales of all experts, [E, N]
    (dict(out=C.c_void_p(FAKE + 3 * GAP + 4 * 3 * 256 - 16)), BAD), (dict(rows=0, a=None, off=None), OK)])
def test_grouped_gemm_int8(kw, status):
    assert grouped(**kw) == status


@pytest.mark.parametrize("rows,E,N,K,status", [
    (1, 0, 8, 16, OK), (1, 3, 8, 16, OK), (1, 0, 8, 32768, OK), (1, 0, 8, 24, NOT), (1, 0, 8, 32784, NOT),
    (0, 0, 8, 16, BAD), (1, 1025, 8, 16, BAD)])
def test_gemm_plan_int8(rows, E, N, K, status):
    assert ops.lib().moe_gemm_plan(rows, E, N, K, INT8, C.byref(ops.GemmPlanInfo())) == status


def test_binding_checks():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)   # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)      # noqa: E731
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8)       # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)     # noqa: E731
    f32 = torch.zeros
    for call in (
            lambda: ops.moe_sort_rows(bf(4, 64), i32(3, 2), 8),
            lambda: ops.moe_sort_rows(bf(4, 64), torch.zeros(4, 2, dtype=torch.int64), 8),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(8), 8),
            lambda: ops.moe_sort_rows(f32(4, 64), i32(4, 2), 8),
            lambda: ops.moe_sort_rows(bf(64, 4).t(), i32(4, 2), 8),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 0),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8, x_scale=f32(4)),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8, quant="mxfp8"),
            lambda: ops.moe_sort_rows(i8(4, 64), i32(4, 2), 8),
            lambda: ops.moe_sort_rows(i8(4, 64), i32(4, 2), 8, x_scale=f32(4, 1)),
            lambda: ops.moe_sort_rows(i8(4, 64), i32(4, 2), 8, x_scale=f32(4), quant="int8"),
            lambda: ops.moe_sort_rows(u8(4, 128), i32(4, 2), 8, x_scale=f32(4)),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8, rows=bf(4, 64)),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8, quant="int8", rows=u8(8, 64)),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8, scales=f32(8)),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8, offsets=i32(8)),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8, inv=i32(8)),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8, scratch=i32(8)),
            lambda: ops.moe_sort_rows(None, i32(4, 2), 8),
            lambda: ops.moe_combine_rows(f32(8, 64), i32(4, 2)),
            lambda: ops.moe_combine_rows(bf(8, 64), i32(4, 2), bf(4, 2)),
            lambda: ops.moe_combine_rows(bf(8, 64), i32(4, 2), f32(2, 4)),
            lambda: ops.moe_combine_rows(bf(8, 64), i32(4, 2), out=bf(8, 64)),
            lambda: ops.moe_combine_rows(bf(8, 64), torch.zeros(4, 2, dtype=torch.int64)),
            lambda: ops.moe_combine_rows_bwd(bf(4, 64), i32(3, 2)),
            lambda: ops.moe_combine_rows_bwd(bf(4, 64), i32(4, 2), rows=bf(8, 32)),
            lambda: ops.moe_combine_rows_bwd(bf(4, 64), i32(4, 2), rows=bf(8, 64), grad_rows=bf(9, 64)),
            lambda: ops.moe_combine_rows_bwd(bf(4, 64), i32(4, 2), grad_weights=f32(4, 2)),
            lambda: ops.moe_combine_rows_bwd(bf(4, 64), i32(4, 2), grad_rows=f32(8, 64)),
            lambda: ops.moe_quant_act_int8(f32(2, 64)),
            lambda: ops.moe_quant_act_int8(bf(2, 64), codes=u8(2, 64)),
            lambda: ops.moe_quant_act_int8(bf(2, 64), scales=f32(2, 1)),
            lambda: ops.moe_silu_mul_int8(bf(2, 63)),
            lambda: ops.moe_silu_mul_int8(bf(2, 64), codes=i8(2, 64)),
            lambda: ops.moe_gemm_int8(u8(2, 64), f32(2), i8(8, 64), f32(8)),
            lambda: ops.moe_gemm_int8(i8(2, 64), f32(2, 1), i8(8, 64), f32(8)),
            lambda: ops.moe_gemm_int8(i8(2, 64), f32(2), i8(8, 32), f32(8)),
            lambda: ops.moe_gemm_int8(i8(2, 64), f32(2), i8(8, 64), f32(2)),
            lambda: ops.moe_grouped_gemm(i8(2, 64), i8(3, 8, 64), i32(4)),
            lambda: ops.moe_grouped_gemm(i8(2, 64), bf(3, 8, 64), i32(4), f32(2), f32(3, 8)),
            lambda: ops.moe_grouped_gemm(i8(2, 64), i8(3, 8, 64), i32(4), f32(2), f32(8)),
            # right but for the device
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8),
            lambda: ops.moe_sort_rows(bf(4, 64), i32(4, 2), 8, quant="int8"),
            lambda: ops.moe_combine_rows(bf(8, 64), i32(4, 2), f32(4, 2)),
            lambda: ops.moe_combine_rows_bwd(bf(4, 64), i32(4, 2), rows=bf(8, 64)),
            lambda: ops.moe_quant_act_int8(bf(2, 64)),
            lambda: ops.moe_silu_mul_int8(bf(2, 64)),
            lambda: ops.moe_gemm_int8(i8(2, 64), f32(2), i8(8, 64), f32(8)),
            lambda: ops.moe_grouped_gemm(i8(2, 64), i8(3, 8, 64), i32(4), f32(2), f32(3, 8)),
    ):
        with pytest.raises(AssertionError):
            call()
