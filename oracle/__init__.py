"""fp64 CPU oracle of the fused MoE layer and the operators around it (test
infrastructure only).

Only the tests, the package smoke check and the benchmark's CPU-baseline leg
may import this package; the product path never does.
"""
from . import moe_oracle as _layer, rows_oracle as _rows
from .moe_oracle import *  # noqa: F401,F403
from .rows_oracle import *  # noqa: F401,F403

__all__ = [*_layer.__all__, *_rows.__all__]
