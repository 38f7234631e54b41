"""Quantisation in blocks and SwiGLU from and to 8 bits, against the formulas in 64 bits; the gradient
against differences too."""
import itertools

import pytest
import torch

from block_helpers import (COLUMNS, DEV, DT, QT, ROWS, SQUARES, blocks, check_codes, gen, half_step, operand, value)

pytestmark = pytest.mark.gpu
BLOCKS = {"rows": ROWS, "columns": COLUMNS, "squares": SQUARES}


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


def values(g, T, H, dt):
    x = torch.randn(T, H, generator=g, device=DEV) * torch.exp(2 * torch.randn(T, 1, generator=g, device=DEV))
    return x.to(dt)


SIZES = [(1, 1), (1, 128), (1, 1920), (3, 129), (5, 100), (17, 1111), (64, 640), (127, 127), (128, 128), (130, 257), (129, 1030), (300, 512), (1000, 72),
         (2049, 8)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("block", BLOCKS)
def test_quant(fw, T, H, block):
    for (dt, fmt), seed in zip(itertools.product(DT, QT), range(9)):
        x = values(gen(seed), T, H, DT[dt])
        r = fw.block_quant(x, block=BLOCKS[block], out_dtype=QT[fmt])
        assert r.q.dtype == QT[fmt] and r.q.shape == x.shape and r.scale.dtype == torch.float32
        check_codes(r.q, r.scale, x.double(), BLOCKS[block], fmt, what=f"{T} x {H} {block} {dt} {fmt}")


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("pad,skip", [(8, 8), (16, 0), (3, 1)])
def test_quant_strides(fw, block, dt, pad, skip):
    """Rows of a wider tensor, and an output that starts at any byte; the same codes as from a copy."""
    for T, H in ((1, 256), (40, 264), (200, 131)):
        wide = values(gen(T), T, H + pad, DT[dt])
        x = wide[:, skip:skip + H]
        want = fw.block_quant(x.contiguous(), block=BLOCKS[block])
        buf = torch.zeros(T * H + 16, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        out = buf[skip:skip + T * H].view(T, H)
        got = fw.block_quant(x, block=BLOCKS[block], out=out)
        assert got.q is out and torch.equal(out.view(torch.uint8), want.q.view(torch.uint8)) and torch.equal(got.scale, want.scale)
        rest = torch.cat([buf[:skip], buf[skip + T * H:]])
        assert not bool(rest.view(torch.uint8).any())


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("fmt", QT)
def test_quant_extremes(fw, block, fmt):
    """All zeros, the smallest and the largest values, NaN and infinities, each in blocks of their own."""
    br, bc = BLOCKS[block]
    T, H = 3 * br, 5 * bc
    x = torch.randn(T, H, generator=gen(0), device=DEV)
    at = lambda i, j: (slice(i * br, (i + 1) * br), slice(j * bc, (j + 1) * bc))       # noqa: E731
    x[at(0, 0)] = 0.0
    x[at(0, 1)] *= 1e-44
    x[at(0, 2)] = x[at(0, 2)].sign() * 3.4e38
    x[at(0, 3)] *= 1e-37
    x[at(1, 1)][-1, -1] = float("nan")
    x[at(1, 2)][0, 0] = float("inf")
    x[at(1, 4)][-1, 0] = float("-inf")
    r = fw.block_quant(x, block=BLOCKS[block], out_dtype=QT[fmt])
    odd = torch.zeros(3, 5, dtype=torch.bool, device=DEV)
    odd[1, 1] = odd[1, 2] = odd[1, 4] = True
    assert torch.equal(r.scale.isnan(), odd)
    wide = odd.repeat_interleave(br, 0).repeat_interleave(bc, 1)
    assert torch.equal(r.q.float().isnan(), wide)
    y, s = x.double().masked_fill(wide, 1.0), r.scale.masked_fill(odd, 1.0 / {"e4m3": 448.0, "e5m2": 57344.0}[fmt])
    q = torch.where(wide, {"e4m3": 448.0, "e5m2": 57344.0}[fmt], r.q.double())
    check_codes(q, s, y, BLOCKS[block], fmt)
    assert not bool(r.q[at(0, 0)].float().any()) and float(r.scale[0, 0]) == 2.0 ** -126


@pytest.mark.parametrize("block", BLOCKS)
def test_quant_empty_and_single(fw, block):
    for T, H in ((0, 5), (5, 0), (0, 0)):
        r = fw.block_quant(torch.empty(T, H, device=DEV), block=BLOCKS[block])
        assert r.q.shape == (T, H)
        assert r.scale.shape == (blocks(T, BLOCKS[block][0]), blocks(H, BLOCKS[block][1]))


def test_quant_past_32_bits(fw):
    T, H = 70000, 32768                                      # 2.29e9 values
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=gen(0))
    for block in (ROWS, SQUARES, COLUMNS):
        r = fw.block_quant(x, block=block)
        for rows in (slice(0, 128), slice(65536, 65664), slice(69888, T)):
            s = slice(rows.start // block[0], blocks(rows.stop, block[0]))
            check_codes(r.q[rows], r.scale[s], x[rows].double(), block, "e4m3")
        del r


@pytest.mark.parametrize("block", BLOCKS)
def test_quant_same_on_a_side_stream_and_in_a_graph(fw, block):
    x = values(gen(0), 300, 1000, torch.bfloat16)
    want = fw.block_quant(x, block=BLOCKS[block])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = fw.block_quant(x, block=BLOCKS[block])
    s.synchronize()
    assert torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8)) and torch.equal(got.scale, want.scale)
    y = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fw.block_quant(y, block=BLOCKS[block])
    y.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8)) and torch.equal(got.scale, want.scale)


# ------------------------------------------------------------------------------- SwiGLU
def gates(g, T, H, dt):
    x = torch.randn(T, 2 * H, generator=g, device=DEV) * torch.exp(torch.randn(T, 1, generator=g, device=DEV))
    return x.clamp(-40, 40).to(dt)


def silu_off(g):
    """How far g / (1 + e^-g) is off, relative: the fast exponential's 2 + 1.173 |g| units of 2^-23, the fast division's 2,
    and five roundings of 2^-24."""
    return (2 + 1.173 * g.abs() + 2 + 2.5) * 2.0 ** -23


@pytest.mark.parametrize("T,H", [(1, 1), (1, 1920), (3, 129), (5, 100), (17, 1111), (64, 640), (128, 128), (130, 257), (300, 512)])
@pytest.mark.parametrize("block", ["rows", "squares"])
@pytest.mark.parametrize("dt", DT)
def test_swiglu(fw, T, H, block, dt):
    x = gates(gen(T + H), T, H, DT[dt])
    for fmt in QT:
        r = fw.swiglu_quant(x, block=BLOCKS[block], out_dtype=QT[fmt], checkpoint=True)
        gate, up = x.double().chunk(2, 1)
        off = silu_off(gate).max()                           # of the values and, as the maximum, of the scales
        check_codes(r.q, r.scale, gate * torch.sigmoid(gate) * up, BLOCKS[block], fmt, off=off, what="y")
        n = blocks(H)
        assert r.checkpoint.shape == (T, 2 * H) and r.checkpoint_scale.shape == (T, 2 * n)
        for half, k, v in ((r.checkpoint[:, :H], r.checkpoint_scale[:, :n], gate), (r.checkpoint[:, H:], r.checkpoint_scale[:, n:], up)):
            check_codes(half, k, v, ROWS, "e4m3", what="checkpoint")
        bare = fw.swiglu_quant(x, block=BLOCKS[block], out_dtype=QT[fmt])
        assert bare.checkpoint is None and bare.checkpoint_scale is None
        assert torch.equal(bare.q.view(torch.uint8), r.q.view(torch.uint8)) and torch.equal(bare.scale, r.scale)


@pytest.mark.parametrize("block", ["rows", "squares"])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("pad,skip", [(8, 8), (3, 1)])
def test_swiglu_strides(fw, block, dt, pad, skip):
    for T, H in ((1, 256), (40, 264), (200, 131)):
        x = gates(gen(T), T, H + pad, DT[dt])[:, skip:skip + 2 * H]
        want = fw.swiglu_quant(x.contiguous(), block=BLOCKS[block], checkpoint=True)
        got = fw.swiglu_quant(x, block=BLOCKS[block], checkpoint=True)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("block", ["rows", "squares"])
def test_swiglu_extremes(fw, block):
    """Gates far out on both sides, and a NaN that stays in its blocks."""
    T, H = 256, 384
    x = torch.randn(T, 2 * H, generator=gen(0), device=DEV)
    x[:, :128] = -200.0
    x[0, 128:256] = 88.0
    x[130, H + 300] = float("nan")
    r = fw.swiglu_quant(x, block=BLOCKS[block], checkpoint=True)
    assert not bool(r.q[:, :128].float().any())              # e^-200 is nothing
    gate, up = x[0, 128:256].double(), x[0, H + 128:H + 256].double()
    if block == "rows":
        check_codes(r.q[:1, 128:256], r.scale[:1, 1:2], (gate * up)[None], ROWS, "e4m3", off=float(silu_off(gate).max()))
        want = torch.zeros(T, 3, dtype=torch.bool, device=DEV)
        want[130, 2] = True
    else:
        want = torch.zeros(2, 3, dtype=torch.bool, device=DEV)
        want[1, 2] = True
    assert torch.equal(r.scale.isnan(), want)
    kept = torch.zeros(T, 6, dtype=torch.bool, device=DEV)
    kept[130, 5] = True
    assert torch.equal(r.checkpoint_scale.isnan(), kept)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 1920), (3, 129), (17, 1111), (64, 640), (130, 257), (300, 512)])
@pytest.mark.parametrize("dt", DT)
def test_swiglu_backward(fw, T, H, dt):
    g = gen(T)
    kept, _ = operand(g, (T, 2 * H), ROWS)
    n = blocks(H)
    scale = torch.exp(2 * torch.rand(T, 2 * n, generator=g, device=DEV)) / 200
    gy = torch.randn(T, H, generator=g, device=DEV).to(DT[dt])
    got = fw.swiglu_backward(gy, kept, scale)
    gate, up = value(kept[:, :H], scale[:, :n], ROWS), value(kept[:, H:], scale[:, n:], ROWS)
    y, s = gy.double(), torch.sigmoid(gate)
    want = torch.cat([y * up * s * (1 + gate * (1 - s)), y * gate * s], 1)
    # s (1 + g (1 - s)) changes by at most (1 + |g|) times what s is off, and rounds five times by 2^-24 of at most (1 + |g|) s;
    # 1 - s itself is off by s' error and 2^-25, times |g| s
    tol = torch.cat([(y * up).abs() * (1 + gate.abs()) * s * (silu_off(gate) + 5 * 2.0 ** -24), (y * gate).abs() * s * silu_off(gate)], 1)
    # the product of a code and its scale rounds gate and up by 2^-24: relative in up, and in gate (1 + |g|) of the derivative's size
    tol = tol + 2.0 ** -23 * (1 + torch.cat([gate, gate], 1).abs()) * torch.cat([(y * up).abs() * (1 + gate.abs()) * s, (y * gate).abs() * s + y.abs() * s], 1)
    tol = tol + half_step(got.dtype) * (want.abs() + tol) + (2.0 ** -25 if dt == "f16" else 0.0)
    assert got.dtype == DT[dt] and bool(((got.double() - want).abs() <= tol).all())


def test_swiglu_backward_against_differences(fw):
    """(f(x + h) - f(x - h)) / 2h in 64 bits around the inputs that the checkpoint holds: within h^2 f''' / 6 < 1e-7."""
    x = gates(gen(7), 9, 200, torch.float32).clamp(-8, 8)
    r = fw.swiglu_quant(x, checkpoint=True)
    gy = torch.randn(9, 200, generator=gen(8), device=DEV)
    got = fw.swiglu_backward(gy, r.checkpoint, r.checkpoint_scale).double()
    gate, up = value(r.checkpoint[:, :200], r.checkpoint_scale[:, :2], ROWS), value(r.checkpoint[:, 200:], r.checkpoint_scale[:, 2:], ROWS)
    f, h = lambda a, b: a * torch.sigmoid(a) * b, 1e-4       # noqa: E731
    want = torch.cat([gy * (f(gate + h, up) - f(gate - h, up)), gy * (f(gate, up + h) - f(gate, up - h))], 1) / (2 * h)
    torch.testing.assert_close(got, want, rtol=1e-5, atol=1e-5)


def test_swiglu_backward_strides_and_extremes(fw):
    gy = torch.randn(40, 300, generator=gen(0), device=DEV).bfloat16()
    x = gates(gen(1), 40, 264, torch.bfloat16)
    x[3, :264] = -300.0
    x[4, :264] = 300.0
    r = fw.swiglu_quant(x, checkpoint=True)
    for skip in (0, 8, 1):
        part = gy[:, skip:skip + 264]
        got = fw.swiglu_backward(part, r.checkpoint, r.checkpoint_scale)
        assert torch.equal(got, fw.swiglu_backward(part.contiguous(), r.checkpoint, r.checkpoint_scale))
        assert not bool(got[3].any())                        # far below, nothing passes
        up = value(r.checkpoint[4:5, 264:], r.checkpoint_scale[4:5, 3:], ROWS)
        torch.testing.assert_close(got[4:5, :264].double(), part[4:5].double() * up, rtol=2.0 ** -8 + 2.0 ** -20, atol=0)
    assert fw.swiglu_backward(gy[:0, :264], r.checkpoint[:0], r.checkpoint_scale[:0]).shape == (0, 528)


def test_refusals(fw):
    x = torch.randn(4, 256, device=DEV)
    f, s, b = fw.block_quant, fw.swiglu_quant, fw.swiglu_backward
    r = s(x, checkpoint=True)
    gy = torch.randn(4, 128, device=DEV)
    for call in (lambda: f(x.double()), lambda: f(x[0]), lambda: f(x.cpu()), lambda: f(x.t()), lambda: f(x[:1].expand(4, 256)),
                 lambda: f(x, out=torch.empty(4, 256, device=DEV)), lambda: f(x, out=r.q), lambda: s(x[:, :255]), lambda: s(x.int()),
                 lambda: s(x, out=torch.empty(4, 256, device=DEV).to(QT["e4m3"])), lambda: b(gy, r.checkpoint[:, :128], r.checkpoint_scale),
                 lambda: b(gy, r.checkpoint, r.checkpoint_scale[:, :1]), lambda: b(gy, r.checkpoint.float(), r.checkpoint_scale),
                 lambda: b(gy[:3], r.checkpoint, r.checkpoint_scale), lambda: b(gy.cpu(), r.checkpoint, r.checkpoint_scale)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(x, block=(1, 64)), lambda: f(x, out_dtype=torch.int8), lambda: s(x, block=COLUMNS), lambda: s(x, out_dtype=torch.bfloat16)):
        with pytest.raises(fw.UnsupportedFeatureError):
            call()
    for call in (lambda: f(x, block=128), lambda: f(None), lambda: f(x, block=(1.0, 128)), lambda: f(x, out_dtype="e4m3")):
        with pytest.raises(TypeError):
            call()
