"""The contract of the operators around the layer on the host, where it is
easily lost: every call here is refused before any device work."""
import ctypes as C
import os
import subprocess
import sys

import pytest

from moe_layer_amd import ops

from test_rows_refusals import BAD, FAKE, GAP, P, norm


@pytest.mark.parametrize("kw", [dict(y=P(2)), dict(residual_out=P(2)), dict(y=C.c_void_p(FAKE + 2 * GAP + 16))])
def test_rmsnorm_one_row_is_not_written_over_the_weight(kw):
    """One row is as long as the weight, which is no row that an output may replace."""
    assert norm(rows=1, **kw) == BAD
    assert norm(rows=1, cols=128, quant=0, codes=None, scales=None, **kw) == BAD


def test_refusals_do_not_depend_on_assert_statements():
    """The same exceptions from an interpreter that skips assert statements."""
    code = """
import torch
from moe_layer_amd import ops
bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
for call in (lambda: ops.moe_rmsnorm(None, bf(256)),
             lambda: ops.moe_rmsnorm(bf(2, 256), bf(256), quant="fp4"),
             lambda: ops.moe_silu_mul([1.0]),
             lambda: ops.moe_gemm_fp8(None, None, None, None),
             lambda: ops.moe_grouped_gemm(None, None, None),
             lambda: ops.moe_silu_mul(bf(2, 256), quant=1)):
    try:
        call()
    except AssertionError:
        continue
    raise SystemExit("not refused")
print("all refused")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(ops.__file__)))
    r = subprocess.run([sys.executable, "-O", "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all refused" in r.stdout, r.stderr[-2000:]


def test_ops_import_on_a_torch_without_gpu_support():
    """Such a torch has no current GPU or stream to ask for: importing the
    package's operators, and what needs neither, works."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    delattr(torch._C, name)
from moe_layer_amd import ops
print(ops.lib().moe_status_string(0).decode())
try:
    ops.moe_silu_mul(torch.zeros(2, 256, dtype=torch.bfloat16))
except AssertionError as e:
    print("refused:", e)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(ops.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused:" in r.stdout, r.stderr[-2000:]
