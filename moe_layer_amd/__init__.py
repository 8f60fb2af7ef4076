"""moe_layer_amd: a fused Mixture-of-Experts layer for AMD MI355X (gfx950).

The layer (router softmax + top-k, token-to-expert alignment, grouped gate/up
GEMM with a fused SiLU-mul (+fp8 re-quant) epilogue, grouped down GEMM and the
router-weighted combine) runs in hand-written HIP kernels behind the C ABI of
``libmoe_mi355x.so`` (declared in ``include/moe.h``).  So do the operators
around it: the quantising residual-add + RMSNorm, the quantising SiLU-gated
multiply, the dense block-scaled fp8 product, the dense int8 product and the
ragged products grouped by expert, tokens' rows sorted by expert and combined
again (with the gradients), and rows quantised to int8.  ``moe_layer_amd.ops``
is the thin Python binding with the same entry-point names; importing this
package does not load the library.
"""

__all__ = ["ops", "workloads"]
