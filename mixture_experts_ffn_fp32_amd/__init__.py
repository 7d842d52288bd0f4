"""MI355X-native DeepSeekMoE layer (forward and backward): gfx950 HIP kernels behind a C ABI.

The library (libmoe.so, built by ``python -m mixture_experts_ffn_fp32_amd.build``)
does all of the layer's work; this package only marshals arguments to it.
"""
from .moe import (MoEError, STAGE_NAMES, backward_workspace_size, balance_loss,  # noqa: F401
                  balance_loss_backward, balance_stats, combine, dequantize_rows, dispatch,
                  expert_ffn, grouped_matmul, grouped_matmul_backward, grouped_matmul_quantized,
                  grouped_matmul_quantized_dx, layer_backward, layer_forward,
                  layer_forward_static, layer_norm, layer_norm_backward, load_library,
                  orthogonalize, quantize_blocks, quantize_rows, rms_norm, rms_norm_backward,
                  rms_norm_quantized, route, timing_enable, timing_read, workspace_size)
