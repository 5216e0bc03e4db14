"""MI355X-native MoE expert layer: routing, sentinel-aware offsets, permute,
grouped GEMMs with fused SiLU*up, and combine (and the layer's backward), its
products on 4-bit weights at decode sizes, and the norm and dropout around it,
as hand-written HIP for gfx950 behind the C ABI in ``include/moe.h``.

``ops`` holds torch-tensor wrappers (argument marshalling only); ``_lib``
loads ``libmoe.so``; ``build`` compiles it.
"""

from ._lib import MoeKernels, load  # noqa: F401
from .ops import (  # noqa: F401
    Gradients,
    NormGradients,
    NormStats,
    backward,
    backward_workspace_bytes,
    build_offsets,
    build_offsets_noalloc,
    dropout_add,
    dropout_add_backward,
    dropout_counters,
    forward,
    forward_fourbit,
    forward_fourbit_workspace_bytes,
    forward_workspace_bytes,
    grouped_gemm,
    grouped_gemm_gather,
    grouped_gemm_tile_shape,
    grouped_matvec_fourbit,
    layer_norm,
    layer_norm_backward,
    layer_norm_backward_workspace_bytes,
    permute,
    quantize_fourbit,
    quantize_rows,
    route_topk,
    unpermute_combine,
    unpermute_combine_dropout,
)
