"""The operators with block scales as a layer uses them together: an MLP and a mixture of experts, forward and
backward, against the same steps in 64 bits on the codes that each step was given; captured in a graph;
beside autograd."""
import importlib.util
import os

import pytest
import torch
import torch.autograd.forward_ad as fwd

from block_helpers import COLUMNS, DEV, ROWS, SQUARES, blocks, check_codes, check_product, gen, half_step, operand, value

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


@pytest.fixture(scope="module")
def layers(fw):
    spec = importlib.util.spec_from_file_location("block_layers", os.path.join(ROOT, "examples", "block_layers.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def weights(layers, g, *shape):
    return layers.quantise_weight(torch.randn(*shape, generator=g, device=DEV) / shape[-1] ** 0.5)


def silu_grad(gate, up, gy):
    s = torch.sigmoid(gate)
    return torch.cat([gy * up * s * (1 + gate * (1 - s)), gy * gate * s], 1)


@pytest.mark.parametrize("T,D,H", [(1, 256, 128), (37, 200, 333), (130, 384, 512), (700, 640, 768)])
def test_mlp(fw, layers, T, D, H):
    g = gen(T)
    x = torch.randn(T, D, generator=g, device=DEV).bfloat16()
    grad = (torch.randn(T, D, generator=g, device=DEV) / T).bfloat16()
    w1, w2 = weights(layers, g, 2 * H, D), weights(layers, g, D, H)
    v1, v2 = value(*w1, SQUARES), value(*w2, SQUARES)
    y, kept = layers.mlp(x, w1, w2)
    check_codes(kept.x.q, kept.x.scale, x.double(), SQUARES, "e4m3")
    act = value(kept.act.q, kept.act.scale, SQUARES)
    check_product(y, act, v2.t(), "output")
    n = blocks(H)
    gate = value(kept.act.checkpoint[:, :H], kept.act.checkpoint_scale[:, :n], ROWS)
    up = value(kept.act.checkpoint[:, H:], kept.act.checkpoint_scale[:, n:], ROWS)
    # the checkpoint holds the first product's output within half a step of E4M3 (2^-4) of it, or of its block's smallest step
    # (a code's 2^-10 times the scale), and that output was rounded to bf16
    first = value(kept.x.q, kept.x.scale, SQUARES) @ v1.t()
    smallest = torch.cat([s.double().repeat_interleave(128, 1)[:, :H] for s in (kept.act.checkpoint_scale[:, :n], kept.act.checkpoint_scale[:, n:])], 1)
    mag = value(kept.x.q, kept.x.scale, SQUARES).abs() @ v1.t().abs()
    off = (torch.cat([gate, up], 1) - first).abs()
    assert bool((off <= first.abs() * (2.0 ** -4 + 2.0 ** -7) + 2.0 ** -10 * smallest + 2.0 ** -18 * mag).all())
    grad_x, grad_w1, grad_w2 = layers.mlp_backward(grad, kept, w1, w2)
    q = fw.block_quant(grad, block=SQUARES, out_dtype=torch.float8_e5m2)
    gq = value(q.q, q.scale, SQUARES)
    check_product(grad_w2, gq.t(), act, "grad_w2")
    grad_y = fw.block_scaled_mm(q.q, w2[0], q.scale, w2[1])
    check_product(grad_y, gq, v2, "grad_y")
    gu = fw.swiglu_backward(grad_y, kept.act.checkpoint, kept.act.checkpoint_scale)
    want = silu_grad(gate, up, grad_y.double())
    assert bool(((gu.double() - want).abs() <= 2 * half_step(torch.bfloat16) * want.abs() + 2.0 ** -16 * want.abs().max()).all())
    h = fw.block_quant(gu, block=SQUARES, out_dtype=torch.float8_e5m2)
    check_product(grad_x, value(h.q, h.scale, SQUARES), v1, "grad_x")
    check_product(grad_w1, value(h.q, h.scale, SQUARES).t(), value(kept.x.q, kept.x.scale, SQUARES), "grad_w1")


@pytest.mark.parametrize("sizes,D,H", [([3, 0, 1], 256, 128), ([40, 0, 90, 130], 200, 260), ([300, 513, 0, 7], 384, 512)])
def test_experts(fw, layers, sizes, D, H):
    """Each expert's rows as the MLP of its weights alone would have them, up to the squares of 128 tokens that they share."""
    T, E = sum(sizes), len(sizes)
    g = gen(T)
    x = torch.randn(T, D, generator=g, device=DEV).bfloat16()
    grad = (torch.randn(T, D, generator=g, device=DEV) / T).bfloat16()
    w1, w2 = weights(layers, g, E, 2 * H, D), weights(layers, g, E, D, H)
    offsets = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    y, kept = layers.experts(x, offsets, w1, w2)
    grad_x, grad_w1, grad_w2 = layers.experts_backward(grad, kept, offsets, w1, w2)
    q = fw.block_quant(grad, block=SQUARES, out_dtype=torch.float8_e5m2)
    grad_y = fw.grouped_block_scaled_mm(q.q, w2[0], offsets, q.scale, w2[1])
    h = fw.block_quant(fw.swiglu_backward(grad_y, kept.act.checkpoint, kept.act.checkpoint_scale), block=SQUARES, out_dtype=torch.float8_e5m2)
    act, xs = value(kept.act.q, kept.act.scale, SQUARES), value(kept.x.q, kept.x.scale, SQUARES)
    gq, hq = value(q.q, q.scale, SQUARES), value(h.q, h.scale, SQUARES)
    ends = offsets.tolist()
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        v1, v2 = value(w1[0][e], w1[1][e], SQUARES), value(w2[0][e], w2[1][e], SQUARES)
        check_product(y[r], act[r], v2.t(), f"output {e}")
        check_product(grad_y[r], gq[r], v2, f"grad_y {e}")
        check_product(grad_x[r], hq[r], v1, f"grad_x {e}")
        check_product(grad_w1[e], hq[r].t(), xs[r], f"grad_w1 {e}")
        check_product(grad_w2[e], gq[r].t(), act[r], f"grad_w2 {e}")


def test_the_gradients_are_the_formulas(fw, layers):
    """The whole step against autograd in 64 bits through the dequantised weights: what the 8-bit roundings leave.  Each value
    passes a few roundings of at most 2^-3 (E5M2) or 2^-4 (E4M3) of its size, independent of one another, so that a
    gradient of many terms is within a fraction of that in the 2-norm: a wrong factor, sign or transpose is not."""
    g = gen(3)
    T, D, H = 256, 256, 384
    x = torch.randn(T, D, generator=g, device=DEV).bfloat16()
    grad = torch.randn(T, D, generator=g, device=DEV).bfloat16()
    w1, w2 = weights(layers, g, 2 * H, D), weights(layers, g, D, H)
    y, kept = layers.mlp(x, w1, w2)
    got = layers.mlp_backward(grad, kept, w1, w2)
    leaves = [t.requires_grad_() for t in (x.double(), value(*w1, SQUARES), value(*w2, SQUARES))]
    gate, up = (leaves[0] @ leaves[1].t()).chunk(2, 1)
    out = (torch.nn.functional.silu(gate) * up) @ leaves[2].t()
    want = torch.autograd.grad(out, leaves, grad.double())
    for a, b in zip((y, *got), (out.detach(), *want)):
        assert float((a.double() - b).norm() / b.norm()) < 2.0 ** -3


def test_a_step_in_a_graph(fw, layers):
    """Captured once and replayed on other inputs and another routing, beside an eager step of the same tensors on another stream."""
    g = gen(5)
    T, D, H, E = 300, 256, 256, 4
    w1, w2 = weights(layers, g, E, 2 * H, D), weights(layers, g, E, D, H)
    xs = [torch.randn(T, D, generator=g, device=DEV).bfloat16() for _ in range(2)]
    offs = [torch.tensor(o, dtype=torch.int32, device=DEV) for o in ([0, 100, 100, 250, 300], [0, 10, 200, 299, 299])]
    grad = torch.randn(T, D, generator=g, device=DEV).bfloat16()

    def step(x, off):
        y, kept = layers.experts(x, off, w1, w2)
        return (y, *layers.experts_backward(grad, kept, off, w1, w2))

    want = [step(x, o) for x, o in zip(xs, offs)]
    x, off = xs[0].clone(), offs[0].clone()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(x, off)
        graphs.append((graph, out))
    side = torch.cuda.Stream()
    for i in (1, 0):
        x.copy_(xs[i])
        off.copy_(offs[i])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            eager = step(xs[i], offs[i])
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for outs in [eager] + [o for _, o in graphs]:
            for a, b in zip(outs, want[i]):
                assert torch.equal(a, b)


def test_same_results_from_run_to_run(fw):
    g = gen(9)
    a, sa = operand(g, (2000, 1000), ROWS)
    w, sw = operand(g, (3000, 1000), SQUARES)
    ref = fw.block_scaled_mm(a, w.t(), sa, sw.t())
    for _ in range(5):
        assert torch.equal(ref, fw.block_scaled_mm(a, w.t(), sa, sw.t()))


def test_example(layers, capsys):
    results = layers.main(["--tokens", "96", "--width", "256", "--hidden", "200", "--experts", "3"])
    assert set(results) == {"mlp", "experts"}
    for values in results.values():
        assert all(bool(torch.isfinite(v).all()) for v in values)
    assert "grad_w2" in capsys.readouterr().out


# ------------------------------------------------------------------------------- beside autograd
def calls(fw):
    f = lambda *s: torch.randn(*s, device=DEV)               # noqa: E731
    q = f(4, 256).to(torch.float8_e4m3fn)
    w = f(8, 256).to(torch.float8_e4m3fn)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    kept = fw.swiglu_quant(f(4, 512), checkpoint=True)
    return [(lambda x: fw.block_quant(x), dict(x=f(4, 256))),
            (lambda gate_up: fw.swiglu_quant(gate_up), dict(gate_up=f(4, 512))),
            (lambda grad_y, scale: fw.swiglu_backward(grad_y, kept.checkpoint, scale), dict(grad_y=f(4, 256), scale=kept.checkpoint_scale)),
            (lambda scale_a, scale_b, out: fw.block_scaled_mm(q, w.t(), scale_a, scale_b, out_dtype=torch.float32, out=out),
             dict(scale_a=f(4, 2), scale_b=f(2, 8), out=f(4, 8))),
            (lambda scale_a, scale_b, out: fw.grouped_block_scaled_mm(q, w.t()[None].expand(1, 256, 8), off[1:], scale_a, scale_b,
                                                                      out_dtype=torch.float32, out=out),
             dict(scale_a=f(4, 2), scale_b=f(1, 2, 8), out=f(4, 8))),
            (lambda scale_grad, scale_x, out: fw.grouped_block_scaled_wgrad(q, q, off, scale_grad, scale_x, out=out),
             dict(scale_grad=f(1, 256), scale_x=f(1, 2), out=f(2, 256, 256)))]


def test_inputs_that_require_grad_or_carry_tangents_are_refused(fw):
    for call, args in calls(fw):
        call(**args)
        for name in args:
            some = dict(args, **{name: args[name].clone().requires_grad_()})
            with pytest.raises(fw.UnsupportedFeatureError, match="requires grad"):
                call(**some)
            with torch.no_grad():
                call(**some)
            with fwd.dual_level():
                dual = fwd.make_dual(args[name], torch.ones_like(args[name]))
                with pytest.raises(fw.UnsupportedFeatureError, match="tangent"):
                    call(**dict(args, **{name: dual}))


def test_writes_in_place_are_known(fw):
    x, out = torch.randn(4, 256, device=DEV), torch.empty(4, 256, device=DEV).to(torch.float8_e4m3fn)
    r = fw.block_quant(x, out=out)
    s = fw.swiglu_quant(torch.randn(4, 512, device=DEV), out=out)
    assert s.q is out and r.q is out and out._version == 2 and x._version == 0
    y = torch.empty(4, 4, device=DEV)
    fw.block_scaled_mm(out, out.t(), s.scale, s.scale.t(), out_dtype=torch.float32, out=y)
    assert y._version == 1
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    z = torch.empty(1, 256, 256, device=DEV)
    c = fw.block_quant(x, block=COLUMNS)
    fw.grouped_block_scaled_wgrad(c.q, c.q, off, c.scale, c.scale, out=z)
    fw.grouped_block_scaled_mm(out, out.t()[None], off, s.scale, s.scale.t()[None], out_dtype=torch.float32, out=y)
    assert z._version == 1 and y._version == 2
