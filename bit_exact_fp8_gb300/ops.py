"""torch-facing operators around an 8-bit product: RMS norm with the residual's addition
and an 8-bit output (``rms_norm_quant``), the product of 8-bit integers
(``int8_scaled_mm``), and the log probabilities of given tokens (``token_logprobs``),
with the gradients that training needs; and 8-bit layers with a scale for each block of 128
codes: quantisation (``block_quant``), the FP8 product, dense and by expert
(``block_scaled_mm``, ``grouped_block_scaled_mm``), and SwiGLU between two of them
(``swiglu_quant``).  They follow ``scaled_mm``: PyTorch provides
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


class BlockQuant(NamedTuple):
    q: torch.Tensor                        # [T, H] FP8
    scale: torch.Tensor                    # fp32, one for each block


class SwigluQuant(NamedTuple):
    q: torch.Tensor                        # [T, H] FP8
    scale: torch.Tensor                    # fp32, one for each block
    checkpoint: Optional[torch.Tensor]     # [T, 2 H] E4M3: the inputs, for the gradient
    checkpoint_scale: Optional[torch.Tensor]   # [T, 2 ceil(H / 128)] fp32


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


def block_quant(x: torch.Tensor, *, block: Tuple[int, int] = (1, 128),
                out_dtype: torch.dtype = torch.float8_e4m3fn, out: Optional[torch.Tensor] = None) -> BlockQuant:
    """``x`` [T, H] (fp32, bf16 or fp16, rows contiguous, any row stride) as FP8 codes
    (float8_e4m3fn or float8_e5m2) with an fp32 scale for each block, ``max|x| / qmax`` but at
    least 2^-126.  The codes are those of ``x / scale`` in fp32.

    block (1, 128): for products over H, scales [T, ceil(H / 128)].  (128, 1): for products over T (a
    weight's gradient), scales [ceil(T / 128), H].  (128, 128): for both, scales [ceil(T / 128),
    ceil(H / 128)]: a weight, or activations that the forward product reads and the backward
    pass reads again.  A block holding NaN or Inf has NaN for its scale and codes."""
    return BlockQuant._make(_calls().block_quant(x, block, out_dtype, out))


def block_mm_workspace_bytes(mat1: torch.Tensor, mat2: torch.Tensor) -> int:
    """Device workspace bytes ``block_scaled_mm`` (mat2 [K, N]) or ``grouped_block_scaled_mm``
    (mat2 [E, K, N]) needs for these operands."""
    return _calls().block_mm_workspace_bytes(mat1, mat2)


def block_scaled_mm(mat1: torch.Tensor, mat2: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor, *,
                    out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``mat1 @ mat2`` of FP8 codes (either format on either side) with a scale for each block
    of 128 of K, each block's products summed in fp32 and scaled by ``scale_a * scale_b``.

    mat1 [M, K] and mat2 [K, N], either dimension of each contiguous; scale_a [M, ceil(K / 128)] or
    [ceil(M / 128), ceil(K / 128)], scale_b [ceil(K / 128), N] or [ceil(K / 128), ceil(N / 128)],
    fp32, of any strides.  With activations x and a weight w [N, K] quantised by ``block_quant``:

        y      = block_scaled_mm(x.q, w.q.t(), x.scale, w.scale.t())
        grad_x = block_scaled_mm(g.q, w.q, g.scale, w.scale)            # g: grad_y in (1, 128) or (128, 128)
        grad_w = block_scaled_mm(g.q.t(), x.q, g.scale.t(), x.scale)    # both in (128, 1) or (128, 128)

    Returns [M, N] in out_dtype (fp32, bf16 or fp16)."""
    return _calls().block_scaled_mm(mat1, mat2, scale_a, scale_b, out_dtype, out, workspace)


def grouped_block_scaled_mm(mat1: torch.Tensor, mat2: torch.Tensor, offsets: torch.Tensor, scale_a: torch.Tensor,
                            scale_b: torch.Tensor, *, out_dtype: torch.dtype = torch.bfloat16,
                            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``block_scaled_mm`` by expert: rows offsets[e] to offsets[e + 1] of mat1 [T, K] (rows
    contiguous) times mat2[e], mat2 [E, K, N] with either of its last dimensions contiguous
    (``w.transpose(1, 2)`` of weights [E, N, K]), E up to 1024.

    offsets [E + 1] int32 on the device, rising; read there alone, so no call waits for the router.
    (They are taken within [0, T] and none below the one before it.)  scale_a as for
    ``block_scaled_mm``, scale_b [E, ceil(K / 128), N or ceil(N / 128)].  Returns [T, N]; rows of
    no expert are 0, or as they were in a given ``out``."""
    return _calls().grouped_block_scaled_mm(mat1, mat2, offsets, scale_a, scale_b, out_dtype, out, workspace)


def block_wgrad_workspace_bytes(grad: torch.Tensor, x: torch.Tensor) -> int:
    """Device workspace bytes ``grouped_block_scaled_wgrad`` needs for these operands."""
    return _calls().block_wgrad_workspace_bytes(grad, x)


def grouped_block_scaled_wgrad(grad: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, scale_grad: torch.Tensor,
                               scale_x: torch.Tensor, *, out_dtype: torch.dtype = torch.float32,
                               out: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradients of the experts' weights: ``grad[rows of e].t() @ x[rows of e]`` for each expert,
    [E, N, K] in out_dtype.  grad [T, N] and x [T, K] are the FP8 codes of the outputs' gradients and of
    the inputs (rows contiguous) as ``block_quant`` makes them of all T rows in blocks (128, 1) or
    (128, 128), whatever the groups are; offsets as for ``grouped_block_scaled_mm``.  An expert
    without rows gets zeros."""
    return _calls().grouped_block_scaled_wgrad(grad, x, offsets, scale_grad, scale_x, out_dtype, out, workspace)


def swiglu_quant(gate_up: torch.Tensor, *, block: Tuple[int, int] = (1, 128),
                 out_dtype: torch.dtype = torch.float8_e4m3fn, checkpoint: bool = False,
                 out: Optional[torch.Tensor] = None) -> SwigluQuant:
    """``silu(gate) * up`` as FP8 codes with block scales, (1, 128) or (128, 128), as
    ``block_quant`` would make them of the fp32 values; gate_up [T, 2 H] (fp32, bf16 or fp16) holds
    gate in its first H columns.  With ``checkpoint`` the inputs are kept too, as E4M3 codes with a scale
    for each (1, 128) block of either half: half the bytes of 16-bit ones, for ``swiglu_backward``."""
    return SwigluQuant._make(_calls().swiglu_quant(gate_up, block, out_dtype, checkpoint, out))


def swiglu_backward(grad_y: torch.Tensor, checkpoint: torch.Tensor, checkpoint_scale: torch.Tensor) -> torch.Tensor:
    """Gradient of ``swiglu_quant`` by gate_up, [T, 2 H] of grad_y's dtype, straight through the
    8-bit roundings, at the inputs that the checkpoint holds; grad_y [T, H] is the gradient of its output."""
    return _calls().swiglu_backward(grad_y, checkpoint, checkpoint_scale)
