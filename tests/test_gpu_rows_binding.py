"""The binding of the operators around the layer: errors of the caller's own
objects come through."""
import pytest
import torch

from moe_layer_amd import ops

from gpu_util import dev

pytestmark = pytest.mark.gpu


class Undecided:
    def __bool__(self):
        raise ValueError("neither")


def test_with_y_without_a_truth_value():
    d = dev()
    x = torch.ones(2, 256, dtype=torch.bfloat16, device=d)
    w = torch.ones(256, dtype=torch.bfloat16, device=d)
    for call in (lambda: ops.moe_rmsnorm(x, w, quant="fp8", with_y=Undecided()),
                 lambda: ops.moe_silu_mul(x, quant="mxfp8", with_y=Undecided())):
        with pytest.raises(ValueError, match="neither"):
            call()
    with pytest.raises(RuntimeError):                  # a tensor of two values has no truth value either
        ops.moe_rmsnorm(x, w, quant="fp8", with_y=torch.tensor([True, False]))
    assert ops.moe_rmsnorm(x, w, quant="fp8")[0] is None
