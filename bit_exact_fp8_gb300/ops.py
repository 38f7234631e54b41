"""torch-facing operators around an 8-bit product: RMS norm with the residual's addition
and an 8-bit output (``rms_norm_quant``), the product of 8-bit integers
(``int8_scaled_mm``), and the log probabilities of given tokens (``token_logprobs``),
with the gradients that training needs.  They follow ``scaled_mm``: PyTorch provides
device memory and the stream, the work runs in libemufp8's CUDA kernels on the current
stream, and there is no CPU path.  They take no part in autograd: a training step calls
the ``_backward`` functions itself, and an input or output that requires grad under grad mode,
or carries a forward-mode tangent, is refused.  Writing into a tensor that was given
counts as a write in place.  No call reads back the device status: a kernel whose bounded
wait gave up leaves outputs unwritten and sets ``_lib.emu_ops_device_status``, which is the
caller's to check where it synchronises.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from .api import EmuCudaError, UnsupportedFeatureError

#: the most alternatives that ``token_logprobs`` returns for a row
MAX_TOP_K = 32


class RmsNormQuant(NamedTuple):
    q: torch.Tensor                        # [T, H], 8 bits
    scale: torch.Tensor                    # [T] fp32, or the one-element scale that was given
    residual: Optional[torch.Tensor]       # [T, H] x + residual in x's dtype; x itself without a residual
    rstd: torch.Tensor                     # [T] fp32


class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor                  # [T] fp32
    entropy: torch.Tensor                  # [T] fp32
    lse: torch.Tensor                      # [T] fp32
    stats: torch.Tensor                    # [T, 3] fp32, for the gradient
    top_logprobs: torch.Tensor             # [T, top_k] fp32
    top_ids: torch.Tensor                  # [T, top_k] int64


_ext = None


def _calls():
    """The extension that checks arguments, allocates and calls libemufp8 (raises OSError if
    it has not been built)."""
    global _ext
    if _ext is None:
        ext = _lib.load_ops()
        ext.set_errors(UnsupportedFeatureError, EmuCudaError)
        _ext = ext
    return _ext


def rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
                   eps: float = 1e-6, out_dtype: torch.dtype = torch.float8_e4m3fn,
                   scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   residual_out: Optional[torch.Tensor] = None) -> RmsNormQuant:
    """RMS norm of the rows of ``x + residual`` with an 8-bit output.

    x, residual [T, H] fp32, bf16 or fp16 (rows contiguous, any row stride); weight [H] of
    x's dtype or fp32.  ``h = x + residual`` in fp32; ``y = h / sqrt(mean(h^2) + eps) *
    weight``; ``q = y / scale`` rounded to nearest even and saturated to out_dtype
    (float8_e4m3fn, float8_e5m2 or int8).  ``scale`` is a one-element fp32 tensor (what
    ``scaled_mm`` takes as scale_a); without it each row has its own, ``max|y| / qmax``
    but at least 2^-126: with int8 codes what ``int8_scaled_mm`` takes as scale_a.  FP8 codes
    with a scale for each row are for products outside this package (``scaled_mm`` takes one
    scale for all rows).  The returned
    ``residual`` is h rounded to x's dtype, in ``residual_out`` if given (it may be
    ``residual`` or ``x``: updated in place); ``rstd`` is for ``rms_norm_backward``.

    A row holding NaN or Inf, or whose sum of squares passes fp32's range (values of about
    1e18 and more), has NaN for its rstd and its own scale, and codes of NaN (int8: 0)."""
    return RmsNormQuant._make(_calls().rms_norm_quant(x, weight, residual, eps, out_dtype, scale, out,
                                                       residual_out))


def rms_norm_backward(grad_y: torch.Tensor, hidden: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                      grad_residual: Optional[torch.Tensor] = None, *,
                      workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradients of ``rms_norm_quant``, straight through its 8-bit rounding: (grad_x [T, H]
    of hidden's dtype, which is the gradient of x and of residual alike; grad_weight [H]
    fp32).  ``hidden`` is the returned ``residual``, ``grad_y`` the gradient of the
    normalised output and ``grad_residual`` the one that reaches ``residual`` directly."""
    return _calls().rms_norm_backward(grad_y, hidden, rstd, weight, grad_residual, workspace)


def int8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Device workspace bytes ``int8_scaled_mm`` needs for these sizes."""
    return int(_lib.load().emu_int8_workspace_bytes(M, N, K))


def int8_scaled_mm(mat1: torch.Tensor, mat2: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor, *,
                   out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``(mat1 @ mat2) * scale_a * scale_b`` of 8-bit integers, the sums exact in 32 bits.

    mat1 [M, K] with contiguous rows, mat2 [K, N] with contiguous columns (``w.t()`` of a
    row-major [N, K] weight); any M, N and K up to 131071, any row stride.  scale_a holds
    M values (one for each token) or one, scale_b N (one for each channel) or one, fp32.
    Returns [M, N] in out_dtype (fp32, bf16 or fp16)."""
    return _calls().int8_scaled_mm(mat1, mat2, scale_a, scale_b, out_dtype, out, workspace)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, top_k: int = 0,
                   ignore_index: int = -100) -> TokenLogprobs:
    """Log probabilities of ``tokens`` [T] (int64) under ``logits`` [T, V] (fp32, bf16 or
    fp16, rows contiguous), with each row's entropy, log-sum-exp, ``stats`` and ``top_k`` (0 to 32)
    largest log probabilities with their ids, in falling order, equal ones by lower id.

    A token equal to ignore_index has logprob 0; any other token outside [0, V) has NaN.
    -inf logits have probability 0.  A row of nothing but -inf has entropy 0 and -inf
    otherwise; a row holding NaN or +inf has NaN, and ids of -1 (an ignored token's logprob
    is 0 there too)."""
    return TokenLogprobs._make(_calls().token_logprobs(logits, tokens, top_k, ignore_index))


def token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, stats: torch.Tensor,
                            grad_logprob: Optional[torch.Tensor], grad_entropy: Optional[torch.Tensor] = None, *,
                            ignore_index: int = -100, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of ``token_logprobs``' logprob and entropy by the logits, of their dtype;
    ``stats`` is what it returned.  Rows of tokens outside [0, V) that are not ignored get NaN,
    whatever else holds of them; rows of nothing but -inf zeros.  ``out`` may be the logits themselves: the gradient then
    takes their place."""
    return _calls().token_logprobs_backward(logits, tokens, stats, grad_logprob, grad_entropy, ignore_index, out)
