"""The contract of the operators around the layer on the host, where it is
easily lost: every call here is refused before any device work."""
import ctypes as C

import pytest

from moe_layer_amd import ops

from test_rows_refusals import BAD, FAKE, GAP, P, norm


@pytest.mark.parametrize("kw", [dict(y=P(2)), dict(residual_out=P(2)), dict(y=C.c_void_p(FAKE + 2 * GAP + 16))])
def test_rmsnorm_one_row_is_not_written_over_the_weight(kw):
    """One row is as long as the weight, which is no row that an output may replace."""
    assert norm(rows=1, **kw) == BAD
    assert norm(rows=1, cols=128, quant=0, codes=None, scales=None, **kw) == BAD
