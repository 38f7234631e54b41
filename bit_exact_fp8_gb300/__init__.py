"""bit_exact_fp8_gb300 -- the FP8 scaled GEMM of a reference tensor-core platform
(the mmaemu "hopper" and "ada" presets), computed bit for bit by hand-written
sm_103a CUDA kernels on a GB300.

    from bit_exact_fp8_gb300 import scaled_mm
    y = scaled_mm(x, w.t(), scale_x, scale_w, out_dtype=torch.bfloat16, use_fast_accum=True)

The C ABI is include/emu_fp8.h (libemufp8.so, built by ``build.build()``);
``_lib`` binds it through ctypes, ``api`` adds the torch-facing call and ``ops`` the
operators around an 8-bit product: ``rms_norm_quant`` makes its operand from the residual
stream, ``int8_scaled_mm`` is the product of the other 8-bit type, ``token_logprobs`` reads
the logits of a model's last product.  ``block_quant``, ``block_scaled_mm``,
``grouped_block_scaled_mm`` and ``swiglu_quant`` are 8-bit layers with a scale for each block of
128, dense and by expert, with their gradients.
"""
from .api import (EmuCudaError, EmuError, ReferenceRejectsError, UnsupportedFeatureError,
                  accumulate, preset_params, scaled_mm, scaled_mm_host, staging_bytes,
                  tile_for, workspace_bytes)
from .ops import (BlockQuant, RmsNormQuant, SwigluQuant, TokenLogprobs, block_mm_workspace_bytes, block_quant,
                  block_scaled_mm, block_wgrad_workspace_bytes, grouped_block_scaled_mm,
                  grouped_block_scaled_wgrad, int8_scaled_mm, int8_workspace_bytes, rms_norm_backward,
                  rms_norm_quant, swiglu_backward, swiglu_quant, token_logprobs, token_logprobs_backward)

__all__ = ["scaled_mm", "scaled_mm_host", "accumulate", "preset_params", "workspace_bytes",
           "staging_bytes", "tile_for", "EmuError", "ReferenceRejectsError", "UnsupportedFeatureError",
           "EmuCudaError", "rms_norm_quant", "rms_norm_backward", "RmsNormQuant", "int8_scaled_mm",
           "int8_workspace_bytes", "token_logprobs", "token_logprobs_backward", "TokenLogprobs", "block_quant",
           "BlockQuant", "block_scaled_mm", "block_mm_workspace_bytes", "grouped_block_scaled_mm",
           "grouped_block_scaled_wgrad", "block_wgrad_workspace_bytes", "swiglu_quant", "swiglu_backward",
           "SwigluQuant"]
