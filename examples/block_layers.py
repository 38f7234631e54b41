"""An 8-bit MLP and a mixture of experts with block scales: one training step's outputs and gradients,
with what the backward pass reads kept in FP8.

    python examples/block_layers.py [--tokens 512] [--width 1920] [--hidden 2560] [--experts 8]

Forward: the input is quantised in squares of 128 x 128 (``block_quant``), so that the same codes serve
the product here and the weight's gradient later; the first product's output goes through
``swiglu_quant``, which keeps its inputs in 8 bits; the second product follows.  Backward: the
outputs' gradients are quantised in squares too, the inputs' gradients come from the weights'
codes as they lie, and ``swiglu_backward`` reads the 8-bit checkpoint.
"""
from __future__ import annotations

import argparse
import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_exact_fp8_gb300 import (block_quant, block_scaled_mm, grouped_block_scaled_mm,  # noqa: E402
                                 grouped_block_scaled_wgrad, swiglu_backward, swiglu_quant)

SQUARES = (128, 128)


class Kept(NamedTuple):
    x: object            # BlockQuant of the input
    act: object          # SwigluQuant


def quantise_weight(w: torch.Tensor):
    """(codes, scales) of [N, K] or, expert by expert, of [E, N, K] weights."""
    if w.dim() == 2:
        return tuple(block_quant(w, block=SQUARES))
    parts = [block_quant(e, block=SQUARES) for e in w]
    return torch.stack([p.q.view(torch.uint8) for p in parts]).view(parts[0].q.dtype), torch.stack([p.scale for p in parts])


def mlp(x, w1, w2):
    """x [T, D]; w1, w2 (codes, scales) of [2 H, D] and [D, H].  (output, what the backward pass needs)"""
    xq = block_quant(x, block=SQUARES)
    gate_up = block_scaled_mm(xq.q, w1[0].t(), xq.scale, w1[1].t())
    act = swiglu_quant(gate_up, block=SQUARES, checkpoint=True)
    return block_scaled_mm(act.q, w2[0].t(), act.scale, w2[1].t()), Kept(xq, act)


def mlp_backward(grad, kept, w1, w2):
    """(grad_x, grad_w1, grad_w2), the weights' in fp32."""
    g = block_quant(grad, block=SQUARES, out_dtype=torch.float8_e5m2)
    grad_w2 = block_scaled_mm(g.q.t(), kept.act.q, g.scale.t(), kept.act.scale, out_dtype=torch.float32)
    grad_y = block_scaled_mm(g.q, w2[0], g.scale, w2[1])
    grad_gu = swiglu_backward(grad_y, kept.act.checkpoint, kept.act.checkpoint_scale)
    h = block_quant(grad_gu, block=SQUARES, out_dtype=torch.float8_e5m2)
    grad_w1 = block_scaled_mm(h.q.t(), kept.x.q, h.scale.t(), kept.x.scale, out_dtype=torch.float32)
    return block_scaled_mm(h.q, w1[0], h.scale, w1[1]), grad_w1, grad_w2


def experts(x, offsets, w1, w2):
    """The same for rows sorted by expert; w1, w2 of [E, 2 H, D] and [E, D, H]."""
    xq = block_quant(x, block=SQUARES)
    gate_up = grouped_block_scaled_mm(xq.q, w1[0].transpose(1, 2), offsets, xq.scale, w1[1].transpose(1, 2))
    act = swiglu_quant(gate_up, block=SQUARES, checkpoint=True)
    return grouped_block_scaled_mm(act.q, w2[0].transpose(1, 2), offsets, act.scale, w2[1].transpose(1, 2)), Kept(xq, act)


def experts_backward(grad, kept, offsets, w1, w2):
    g = block_quant(grad, block=SQUARES, out_dtype=torch.float8_e5m2)
    grad_w2 = grouped_block_scaled_wgrad(g.q, kept.act.q, offsets, g.scale, kept.act.scale)
    grad_y = grouped_block_scaled_mm(g.q, w2[0], offsets, g.scale, w2[1])
    grad_gu = swiglu_backward(grad_y, kept.act.checkpoint, kept.act.checkpoint_scale)
    h = block_quant(grad_gu, block=SQUARES, out_dtype=torch.float8_e5m2)
    grad_w1 = grouped_block_scaled_wgrad(h.q, kept.x.q, offsets, h.scale, kept.x.scale)
    return grouped_block_scaled_mm(h.q, w1[0], offsets, h.scale, w1[1]), grad_w1, grad_w2


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1920)
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--experts", type=int, default=8)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    x, grad = randn(a.tokens, a.width).bfloat16(), (randn(a.tokens, a.width) / a.tokens).bfloat16()
    w1, w2 = randn(2 * a.hidden, a.width) / a.width ** 0.5, randn(a.width, a.hidden) / a.hidden ** 0.5
    q1, q2 = quantise_weight(w1), quantise_weight(w2)
    y, kept = mlp(x, q1, q2)
    grads = mlp_backward(grad, kept, q1, q2)
    results = {"mlp": (y, *grads)}

    choice = torch.randint(0, a.experts, (a.tokens,), generator=gen, device="cuda")
    order = choice.argsort(stable=True)
    counts = torch.bincount(choice, minlength=a.experts)
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)      # stays on the device
    e1 = quantise_weight(w1 + 0.5 * randn(a.experts, *w1.shape) / a.width ** 0.5)
    e2 = quantise_weight(w2 + 0.5 * randn(a.experts, *w2.shape) / a.hidden ** 0.5)
    y, kept = experts(x[order], offsets, e1, e2)
    results["experts"] = (y, *experts_backward(grad[order], kept, offsets, e1, e2))
    for name, values in results.items():
        print(f"{name}: " + ", ".join(f"{n} {v.float().norm():.4f}" for n, v in zip(("output", "grad_x", "grad_w1", "grad_w2"), values)))
    return results


if __name__ == "__main__":
    main()
