"""torch-facing operators around an 8-bit product: RMS norm with the residual's addition
and an 8-bit output (``rms_norm_quant``), the product of 8-bit integers
(``int8_scaled_mm``), and the log probabilities of given tokens (``token_logprobs``),
with the gradients that training needs.  They follow ``scaled_mm``: PyTorch provides
device memory and the stream, the work runs in libemufp8's CUDA kernels on the current
stream, and there is no CPU path.  They take no part in autograd: a training step calls
the ``_backward`` functions itself.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from .api import EmuCudaError, UnsupportedFeatureError

_FLOAT = {torch.float32: _lib.EMU_OUT_F32, torch.bfloat16: _lib.EMU_OUT_BF16,
          torch.float16: _lib.EMU_OUT_F16}
_Q = {torch.float8_e4m3fn: _lib.EMU_Q_E4M3FN, torch.float8_e5m2: _lib.EMU_Q_E5M2,
      torch.int8: _lib.EMU_Q_INT8}

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


def _raise(status: int, what: str):
    msg = f"{what}: {_lib.emu_ops_last_error()}"
    if status == _lib.EMU_EUNSUPPORTED:
        raise UnsupportedFeatureError(msg)
    if status == _lib.EMU_ECUDA:
        raise EmuCudaError(msg)
    raise ValueError(msg)


def _rows(name: str, t: torch.Tensor, shape, dtype, dev) -> int:
    """The row stride of a [rows, columns] tensor whose rows are contiguous."""
    if t.shape != shape or t.dtype != dtype or t.device != dev:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if shape[0] <= 1:
        return shape[1]
    if s0 < shape[1]:
        raise ValueError(f"{name}: rows must not overlap (row stride {s0} of {shape[1]} values)")
    return s0


def _vector(name: str, t: torch.Tensor, count: int, dtype, dev) -> int:
    if t.dtype != dtype or t.device != dev or t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{name}: expected {count} contiguous {dtype} on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _first(t: torch.Tensor, name: str) -> torch.device:
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name}: all tensors must be on a CUDA device (there is no CPU path)")
    return t.device


def _no_grad(*tensors):
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise UnsupportedFeatureError("not differentiable by autograd: an input requires grad under "
                                              "grad mode (call the _backward function)")


def _call(fn, dev: torch.device, what: str, *args):
    """One C call on the device's current stream."""
    if dev.index == torch.cuda.current_device():
        st = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    if st != _lib.EMU_OK:
        _raise(st, what)


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
    but at least 2^-126 (what ``int8_scaled_mm`` takes as scale_a).  The returned
    ``residual`` is h rounded to x's dtype, in ``residual_out`` if given (it may be
    ``residual`` or ``x``: updated in place); ``rstd`` is for ``rms_norm_backward``."""
    dev = _first(x, "x")
    _no_grad(x, weight, residual)
    T, H = x.shape
    dt = x.dtype
    if dt not in _FLOAT:
        raise ValueError(f"x: fp32, bf16 or fp16 expected, got {dt}")
    if out_dtype not in _Q:
        raise UnsupportedFeatureError(f"out_dtype {out_dtype} is not supported")
    ldx = _rows("x", x, (T, H), dt, dev)
    wdt = weight.dtype
    if wdt != dt and wdt != torch.float32:
        raise ValueError(f"weight: {dt} or fp32 expected, got {wdt}")
    wp = _vector("weight", weight, H, wdt, dev)
    rp = ldr = op = ldo = 0
    if residual is not None:
        ldr, rp = _rows("residual", residual, (T, H), dt, dev), residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty((T, H), dtype=dt, device=dev)
    if residual_out is not None:
        ldo, op = _rows("residual_out", residual_out, (T, H), dt, dev), residual_out.data_ptr()
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
    elif out.shape != (T, H) or out.dtype != out_dtype or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous [T, H] tensor of out_dtype on the device")
    rstd = torch.empty(T, dtype=torch.float32, device=dev)
    if scale is None:
        scale_out = torch.empty(T, dtype=torch.float32, device=dev)
        sp, so = 0, scale_out.data_ptr()
    else:
        scale_out = scale
        sp, so = _vector("scale", scale, 1, torch.float32, dev), 0
    _call(_lib.load().emu_rms_norm_quant, dev, "rms_norm_quant", x.data_ptr(), ldx, rp, ldr, wp, _FLOAT[wdt],
          _FLOAT[dt], T, H, eps, sp, _Q[out_dtype], out.data_ptr(), so, op, ldo, rstd.data_ptr())
    return RmsNormQuant(out, scale_out, x if residual_out is None else residual_out, rstd)


def rms_norm_backward(grad_y: torch.Tensor, hidden: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                      grad_residual: Optional[torch.Tensor] = None, *,
                      workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradients of ``rms_norm_quant``, straight through its 8-bit rounding: (grad_x [T, H]
    of hidden's dtype, which is the gradient of x and of residual alike; grad_weight [H]
    fp32).  ``hidden`` is the returned ``residual``, ``grad_y`` the gradient of the
    normalised output and ``grad_residual`` the one that reaches ``residual`` directly."""
    dev = _first(hidden, "hidden")
    _no_grad(grad_y, hidden, weight, grad_residual)
    T, H = hidden.shape
    dt = hidden.dtype
    if dt not in _FLOAT:
        raise ValueError(f"hidden: fp32, bf16 or fp16 expected, got {dt}")
    ldh = _rows("hidden", hidden, (T, H), dt, dev)
    ldy = _rows("grad_y", grad_y, (T, H), dt, dev)
    wdt = weight.dtype
    if wdt != dt and wdt != torch.float32:
        raise ValueError(f"weight: {dt} or fp32 expected, got {wdt}")
    wp = _vector("weight", weight, H, wdt, dev)
    rp = _vector("rstd", rstd, T, torch.float32, dev)
    gp = ldg = 0
    if grad_residual is not None:
        ldg, gp = _rows("grad_residual", grad_residual, (T, H), dt, dev), grad_residual.data_ptr()
    L = _lib.load()
    need = L.emu_rms_norm_backward_workspace_bytes(T, H)
    if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    grad_x = torch.empty((T, H), dtype=dt, device=dev)
    grad_weight = torch.empty(H, dtype=torch.float32, device=dev)
    _call(L.emu_rms_norm_backward, dev, "rms_norm_backward", grad_y.data_ptr(), ldy, hidden.data_ptr(), ldh, rp, wp,
          _FLOAT[wdt], gp, ldg, _FLOAT[dt], T, H, grad_x.data_ptr(), grad_weight.data_ptr(),
          workspace.data_ptr() if need > 0 else 0, need)
    return grad_x, grad_weight


def int8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Device workspace bytes ``int8_scaled_mm`` needs for these sizes, whatever the
    operands' alignment."""
    return int(_lib.load().emu_int8_workspace_bytes(M, N, K, 0))


def int8_scaled_mm(mat1: torch.Tensor, mat2: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor, *,
                   out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``(mat1 @ mat2) * scale_a * scale_b`` of 8-bit integers, the sums exact in 32 bits.

    mat1 [M, K] with contiguous rows, mat2 [K, N] with contiguous columns (``w.t()`` of a
    row-major [N, K] weight); any M, N and K up to 131071, any row stride.  scale_a holds
    M values (one for each token) or one, scale_b N (one for each channel) or one, fp32.
    Returns [M, N] in out_dtype (fp32, bf16 or fp16)."""
    dev = _first(mat1, "mat1")
    if mat2.dim() != 2:
        raise ValueError("mat2 must be 2-D")
    M, K = mat1.shape
    K2, N = mat2.shape
    if K != K2:
        raise ValueError(f"shape mismatch: {tuple(mat1.shape)} @ {tuple(mat2.shape)}")
    lda = _rows("mat1", mat1, (M, K), torch.int8, dev)
    ldb = _rows("mat2.t()", mat2.t(), (N, K), torch.int8, dev)
    if out_dtype not in _FLOAT:
        raise UnsupportedFeatureError(f"out_dtype {out_dtype} is not supported")
    na, nb = scale_a.numel(), scale_b.numel()
    if na != 1 and na != M:
        raise ValueError(f"scale_a: one value or {M} expected, got {na}")
    if nb != 1 and nb != N:
        raise ValueError(f"scale_b: one value or {N} expected, got {nb}")
    sa = _vector("scale_a", scale_a, na, torch.float32, dev)
    sb = _vector("scale_b", scale_b, nb, torch.float32, dev)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    elif out.shape != (M, N) or out.dtype != out_dtype or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous [M, N] tensor of out_dtype on the device")
    L = _lib.load()
    pa, pb = mat1.data_ptr(), mat2.data_ptr()
    need = L.emu_int8_workspace_bytes(M, N, K, (K | lda | ldb | pa | pb) % 16 == 0)
    wp = 0
    if need > 0:
        if workspace is None or workspace.numel() * workspace.element_size() < need or workspace.data_ptr() % 256:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        wp = workspace.data_ptr()
    _call(L.emu_int8_scaled_mm, dev, "int8_scaled_mm", pa, lda, pb, ldb, M, N, K, sa, na,
          sb, nb, out.data_ptr(), _FLOAT[out_dtype], wp, need)
    return out


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, top_k: int = 0,
                   ignore_index: int = -100) -> TokenLogprobs:
    """Log probabilities of ``tokens`` [T] (int64) under ``logits`` [T, V] (fp32, bf16 or
    fp16, rows contiguous), with each row's entropy, log-sum-exp, ``stats`` and ``top_k`` (0 to 32)
    largest log probabilities with their ids, in falling order, equal ones by lower id.

    A token equal to ignore_index has logprob 0; any other token outside [0, V) has NaN.
    -inf logits have probability 0.  A row of nothing but -inf has entropy 0 and -inf
    otherwise; a row holding NaN or +inf has NaN, and ids of -1."""
    dev = _first(logits, "logits")
    _no_grad(logits)
    T, V = logits.shape
    if logits.dtype not in _FLOAT:
        raise ValueError(f"logits: fp32, bf16 or fp16 expected, got {logits.dtype}")
    ldx = _rows("logits", logits, (T, V), logits.dtype, dev)
    tp = _vector("tokens", tokens, T, torch.int64, dev)
    if top_k < 0 or top_k > V:
        raise ValueError(f"top_k {top_k} of {V} logits")
    if top_k > MAX_TOP_K:
        raise UnsupportedFeatureError(f"top_k above {MAX_TOP_K} is not supported")
    logprob = torch.empty(T, dtype=torch.float32, device=dev)
    entropy = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    stats = torch.empty((T, 3), dtype=torch.float32, device=dev)
    lead = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    ids = torch.empty((T, top_k), dtype=torch.int64, device=dev)
    _call(_lib.load().emu_token_logprobs, dev, "token_logprobs", logits.data_ptr(), ldx, _FLOAT[logits.dtype], tp, T,
          V, top_k, ignore_index, logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), stats.data_ptr(),
          lead.data_ptr(), ids.data_ptr())
    return TokenLogprobs(logprob, entropy, lse, stats, lead, ids)


def token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, stats: torch.Tensor,
                            grad_logprob: Optional[torch.Tensor], grad_entropy: Optional[torch.Tensor] = None, *,
                            ignore_index: int = -100, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of ``token_logprobs``' logprob and entropy by the logits, of their dtype;
    ``stats`` is what it returned.  ``out`` may be the logits themselves: the gradient then
    takes their place."""
    dev = _first(logits, "logits")
    _no_grad(logits)
    T, V = logits.shape
    dt = logits.dtype
    if dt not in _FLOAT:
        raise ValueError(f"logits: fp32, bf16 or fp16 expected, got {dt}")
    ldx = _rows("logits", logits, (T, V), dt, dev)
    tp = _vector("tokens", tokens, T, torch.int64, dev)
    sp = _vector("stats", stats, 3 * T, torch.float32, dev)
    glp = 0 if grad_logprob is None else _vector("grad_logprob", grad_logprob, T, torch.float32, dev)
    gep = 0 if grad_entropy is None else _vector("grad_entropy", grad_entropy, T, torch.float32, dev)
    if out is None:
        out = torch.empty((T, V), dtype=dt, device=dev)
    ldo = _rows("out", out, (T, V), dt, dev)
    _call(_lib.load().emu_token_logprobs_backward, dev, "token_logprobs_backward", logits.data_ptr(), ldx, _FLOAT[dt],
          tp, T, V, ignore_index, sp, glp, gep, out.data_ptr(), ldo)
    return out
