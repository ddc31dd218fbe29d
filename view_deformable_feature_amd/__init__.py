"""Sparse4D-style deformable aggregation for AMD Instinct MI355X (gfx950).

The computation lives in ``libdeformagg.so`` (HIP kernels behind a C ABI,
declared in ``include/*.h``); ``api``, ``pack``, ``dcn``, ``norm``, ``int8``,
``rope`` and ``attention`` bind it to PyTorch tensors.
``workloads`` draws seeded synthetic inputs.
"""
from .api import (DeformableAggregationFunction, da_backward, da_backward_accumulate,  # noqa: F401
                  da_backward_atomic, da_forward, deformable_aggregation, forward_workspace_size,
                  workspace_size)

from .pack import (PackLevelsFunction, da_pack_levels, da_unpack_levels,  # noqa: F401
                   feature_maps_format, pack_layout, pack_levels)

from .dcn import (DCNFunction, dcn_backward, dcn_forward, dcn_forward_projected,  # noqa: F401
                  dcn_out_size, dcn_workspace_size, deformable_conv)

from .norm import (GroupNormActFunction, gn_backward, gn_backward_workspace_size,  # noqa: F401
                   gn_forward, gn_workspace_size, group_norm_act)

from .int8 import (i8_linear, i8_linear_workspace_size, i8_matmul,  # noqa: F401
                   i8_matmul_workspace_size, i8_norm_linear, i8_norm_linear_workspace_size,
                   i8_quantize_rows)

from .rope import (NormRotaryFunction, RotaryFunction, norm_rotary, rope_forward,  # noqa: F401
                     rope_frequencies, rope_norm_backward, rope_norm_backward_workspace_size,
                     rope_norm_forward, rotary)

from .attention import (CrossAttentionFunction, attn_backward,  # noqa: F401
                        attn_backward_workspace_size, attn_forward, attn_workspace_size,
                        cross_attention)

__version__ = "1.2.0"
