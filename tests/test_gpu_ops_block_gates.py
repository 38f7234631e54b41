"""SwiGLU's forward and backward pass at gates far below zero, against the formulas in 64 bits: there
1 / (1 + e^-g) comes to the end of fp32's range while the product with a large value is an ordinary number."""
import pytest
import torch

from block_helpers import DEV, QT, ROWS, SQUARES, blocks, check_codes, gen, spread
from test_gpu_ops_block_quant import silu_off

pytestmark = pytest.mark.gpu

#: what sigmoid's values below fp32's normal range may be off beside their relative error: a step, 2^-149, each of
#: the exponential and the division, and half of one of the product with a gate of 40 at least
SMALLEST = 2.0 ** -147


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


def gates(rows=257):
    """A row for each gate from -40 to -104, and a few above."""
    return torch.cat([torch.linspace(-40, -104, rows), torch.tensor([-87.3, -87.4, -88.0, -88.72, -88.73, -20.0, 0.0, 20.0, 88.0, 104.0])]).to(DEV)


@pytest.mark.parametrize("size", [1.0, 1e30])
@pytest.mark.parametrize("fmt", QT)
@pytest.mark.parametrize("H", [128, 200])
def test_swiglu_far_below_zero(fw, size, fmt, H):
    g = gates()
    T = g.numel()
    up = (torch.rand(T, H, generator=gen(H), device=DEV) + 0.5) * size
    up[:, ::3] *= -1
    x = torch.cat([g[:, None].expand(T, H), up], 1).contiguous()
    r = fw.swiglu_quant(x, block=ROWS, out_dtype=QT[fmt])
    wide = g.double()[:, None]
    y = wide * torch.sigmoid(wide) * up.double()
    for i in range(T):
        off = float(silu_off(wide[i]) + SMALLEST / torch.sigmoid(wide[i]))
        check_codes(r.q[i:i + 1], r.scale[i:i + 1], y[i:i + 1], ROWS, fmt, off=off, what=f"gate {float(g[i])}")
    at = int((g == -88.0).nonzero()[0])
    assert bool((r.q[at].float().abs() >= 16).all())         # 88 e^-88 / 2 is 23 times the smallest scale


def test_swiglu_far_below_zero_in_squares(fw):
    """A square of one gate, its values an ordinary size."""
    for gate in (-60.0, -87.0, -88.5, -90.0):
        up = (torch.rand(128, 128, generator=gen(1), device=DEV) + 0.5) * 1e30
        x = torch.cat([torch.full_like(up, gate), up], 1)
        r = fw.swiglu_quant(x, block=SQUARES)
        g = torch.tensor(gate, dtype=torch.float64, device=DEV)
        check_codes(r.q, r.scale, g * torch.sigmoid(g) * up.double(), SQUARES, "e4m3", off=float(silu_off(g) + SMALLEST / torch.sigmoid(g)))


@pytest.mark.parametrize("size", [1.0, 1e30])
@pytest.mark.parametrize("H", [128, 200])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_swiglu_backward_far_below_zero(fw, size, H, dt):
    g = gates()
    T, n = g.numel(), blocks(H)
    codes = torch.full((T, 2 * H), 448.0, device=DEV)
    codes[:, H:] = (torch.rand(T, H, generator=gen(H), device=DEV) + 0.5) * 200
    scale = torch.empty(T, 2 * n, device=DEV)
    scale[:, :n] = g[:, None] / 448.0
    scale[:, n:] = size / 256
    kept = codes.to(QT["e4m3"])
    gy = (torch.rand(T, H, generator=gen(3), device=DEV) + 0.5).to(dt)
    gy[:, 1::3] *= -1
    got = fw.swiglu_backward(gy, kept, scale)
    held = kept.float() * torch.cat([spread(scale[:, :n], ROWS, (T, H)), spread(scale[:, n:], ROWS, (T, H))], 1)   # in fp32, as stated
    gate, up = held[:, :H].double(), held[:, H:].double()
    y, s = gy.double(), torch.sigmoid(gate)
    want = torch.cat([y * up * s * (1 + gate * (1 - s)), y * gate * s], 1)
    # s, and with it 1 + g (1 - s), as in the tests of ordinary gates, and s' smallest step
    size_g, size_u = (y * up).abs() * (1 + gate.abs()), (y * gate).abs()
    tol = torch.cat([size_g * (s * (silu_off(gate) + 5 * 2.0 ** -24) + SMALLEST), size_u * (s * silu_off(gate) + SMALLEST)], 1)
    tol = tol + torch.finfo(dt).eps / 2 * (want.abs() + tol) + 2.0 ** -150 * (1 if dt == torch.float32 else 2 ** 16)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float(g[bad.nonzero()[0, 0]]))
    far = (g < -87.4) & (g > -88.7)
    assert bool((got[far, H:] != 0).all()) and bool((got[far, :H] != 0).all())


def test_swiglu_backward_far_above_zero(fw):
    """The derivative there is that of g itself, also where the other gradient passes the largest number."""
    kept = torch.full((4, 256), 1.0, device=DEV).to(QT["e4m3"])
    scale = torch.tensor([[1e30, 2.0], [1e38, 2.0], [200.0, 3.0], [89.0, 3.0]], device=DEV)
    gy = torch.full((4, 128), 1e9, device=DEV)
    got = fw.swiglu_backward(gy, kept, scale)
    torch.testing.assert_close(got[:, :128], gy * scale[:, 1:], rtol=2.0 ** -20, atol=0)
    assert bool(got[:2, 128:].isposinf().all()) and bool(got[2:, 128:].isfinite().all())


@pytest.mark.parametrize("T,H", [(300, 640), (77, 333)])
def test_swiglu_backward_of_fp32(fw, T, H):
    """By the exponential itself: the sigmoid within 8 2^-24 (the exponential 4, its sum with 1 one, the inverse 2, the product
    one), s (1 + g (1 - s)) within twice that and one more of (1 + |g|) s, and four products and sums."""
    g = gen(T)
    n = blocks(H)
    kept = (torch.randn(T, 2 * H, generator=g, device=DEV) * 60).clamp(-448, 448).to(QT["e4m3"])
    scale = torch.exp(4 * torch.rand(T, 2 * n, generator=g, device=DEV)) / 100
    gy = torch.randn(T, H, generator=g, device=DEV)
    got = fw.swiglu_backward(gy, kept, scale)
    held = kept.float() * torch.cat([spread(scale[:, :n], ROWS, (T, H)), spread(scale[:, n:], ROWS, (T, H))], 1)
    gate, up = held[:, :H].double(), held[:, H:].double()
    assert float(gate.min()) < -60 and float(gate.max()) > 60
    y, s = gy.double(), torch.sigmoid(gate)
    want = torch.cat([y * up * s * (1 + gate * (1 - s)), y * gate * s], 1)
    tol = torch.cat([(y * up).abs() * (1 + gate.abs()) * (21 * 2.0 ** -24 * s + SMALLEST), (y * gate).abs() * (10 * 2.0 ** -24 * s + SMALLEST)], 1)
    bad = ~((got.double() - want).abs() <= tol + 2.0 ** -149)
    assert not bool(bad.any()), (int(bad.sum()), ((got.double() - want).abs() / tol.clamp_min(1e-300)).max())
