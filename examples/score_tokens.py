"""Score a sequence under the 8-bit output head of a model, in FP8 (bit for bit as the
reference platform computes it) and in int8, and take one training step's gradients
through it.

    python examples/score_tokens.py [--tokens 64] [--width 1920] [--vocabulary 512]

The last layer's output is added to the residual stream, normalised and quantised in one
kernel (``rms_norm_quant``), multiplied by the head's 8-bit weights (``scaled_mm`` or
``int8_scaled_mm``), and the logits are read once for the tokens' log probabilities, the
rows' entropies and their leading alternatives (``token_logprobs``).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_exact_fp8_gb300 import (int8_scaled_mm, rms_norm_backward, rms_norm_quant, scaled_mm,  # noqa: E402
                                 token_logprobs, token_logprobs_backward)


def quantise_head(weight: torch.Tensor, dtype: torch.dtype):
    """An [V, H] head in 8 bits: FP8 with one scale, or int8 with one for each row of it."""
    if dtype == torch.int8:
        scale = weight.abs().amax(1) / 127.0
        return (weight / scale[:, None]).round().to(torch.int8), scale
    scale = (weight.abs().amax() / 448.0).reshape(1)
    return (weight / scale).to(dtype), scale


def head_logits(x, residual, norm_weight, head, head_scale, act_scale=None, preset="hopper"):
    """(the norm's outputs, bf16 logits) of the last hidden states."""
    if head.dtype == torch.int8:
        n = rms_norm_quant(x, norm_weight, residual, out_dtype=torch.int8)        # a scale for each token
        return n, int8_scaled_mm(n.q, head.t(), n.scale, head_scale)
    n = rms_norm_quant(x, norm_weight, residual, out_dtype=head.dtype, scale=act_scale)
    return n, scaled_mm(n.q, head.t(), n.scale, head_scale, out_dtype=torch.bfloat16, use_fast_accum=True, preset=preset)


def training_gradients(n, logits, scores, tokens, norm_weight, head, head_scale, entropy_bonus=0.01):
    """Gradients of -mean(logprob) - entropy_bonus * mean(entropy) by the residual stream and the
    norm's weight; the head itself is frozen, and the 8-bit roundings pass gradients straight on."""
    T = tokens.numel()
    gl = torch.full((T,), -1.0 / T, device=logits.device)
    ge = torch.full((T,), -entropy_bonus / T, device=logits.device)
    grad_logits = token_logprobs_backward(logits, tokens, scores.stats, gl, ge)
    dequantised = (head.float() * (head_scale[:, None] if head.dtype == torch.int8 else head_scale)).to(torch.bfloat16)
    return rms_norm_backward(grad_logits @ dequantised, n.residual, n.rstd, norm_weight)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--width", type=int, default=1920)
    ap.add_argument("--vocabulary", type=int, default=512)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x, residual = randn(a.tokens, a.width).bfloat16(), (3 * randn(a.tokens, a.width)).bfloat16()
    norm_weight = (1 + 0.1 * randn(a.width)).bfloat16()
    weight = randn(a.vocabulary, a.width) / a.width ** 0.5 * 3
    tokens = torch.randint(0, a.vocabulary, (a.tokens,), generator=g, device="cuda")
    results = {}
    for name, dtype in (("fp8", torch.float8_e4m3fn), ("int8", torch.int8)):
        head, head_scale = quantise_head(weight, dtype)
        act_scale = torch.full((1,), 8.0 / 448.0, device="cuda")
        n, logits = head_logits(x, residual, norm_weight, head, head_scale, act_scale)
        scores = token_logprobs(logits, tokens, top_k=min(5, a.vocabulary))
        grad_x, grad_weight = training_gradients(n, logits, scores, tokens, norm_weight, head, head_scale)
        results[name] = scores
        print(f"{name}: mean log probability {scores.logprob.mean():.4f}, mean entropy {scores.entropy.mean():.4f}, "
              f"token is the likeliest in {(scores.top_ids[:, 0] == tokens).float().mean():.1%} of rows, "
              f"gradient norms {grad_x.float().norm():.4f} and {grad_weight.norm():.4f}")
    off = (results["fp8"].logprob - results["int8"].logprob).abs()
    print(f"fp8 and int8 differ by {off.mean():.4f} a token, at most {off.max():.4f}")
    return results


if __name__ == "__main__":
    main()
