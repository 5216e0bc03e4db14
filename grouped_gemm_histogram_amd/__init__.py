"""MI355X-native MoE expert layer: routing, sentinel-aware offsets, permute,
grouped GEMMs with fused SiLU*up, and combine (and the layer's backward), its
products on 4-bit weights at decode sizes and on 8-bit integers at any, its form
for up to 16 tokens in two kernels, the norm and dropout around it, and the
AdamW step after its backward, as hand-written HIP for gfx950 behind the C ABI
in ``include/moe.h``.

``ops`` holds torch-tensor wrappers (argument marshalling only); ``_lib``
loads ``libmoe.so``; ``build`` compiles it.
"""

from ._lib import MoeKernels, load  # noqa: F401
from .ops import (  # noqa: F401
    AdamWState,
    Gradients,
    NormGradients,
    NormStats,
    adamw_counters,
    adamw_init,
    adamw_schedule,
    adamw_starts,
    adamw_step,
    backward,
    backward_workspace_bytes,
    build_offsets,
    build_offsets_noalloc,
    dropout_add,
    dropout_add_backward,
    dropout_counters,
    forward,
    forward_decode,
    forward_decode_workspace_bytes,
    forward_eightbit,
    forward_eightbit_workspace_bytes,
    forward_fourbit,
    forward_fourbit_workspace_bytes,
    forward_workspace_bytes,
    grouped_gemm,
    grouped_gemm_eightbit,
    grouped_gemm_gather,
    grouped_gemm_tile_shape,
    grouped_matvec_fourbit,
    layer_norm,
    layer_norm_backward,
    layer_norm_backward_workspace_bytes,
    permute,
    quantize_fourbit,
    quantize_rows,
    quantize_rows_eightbit,
    route_topk,
    unpermute_combine,
    unpermute_combine_dropout,
)
