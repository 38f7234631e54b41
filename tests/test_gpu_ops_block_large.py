"""The operators with block scales at sizes where their kernels take several rounds: pairs of CTAs more than one
tile each by expert, the quantisation's kernels several loads a warp, the loops over rows."""
import random

import pytest
import torch

from block_helpers import (COLUMNS, DEV, DT, QT, ROWS, SQUARES, blocks, check_codes, gen, half_step, operand, spread, value)
from test_gpu_ops_block_mm import grouped, wgrad
from test_gpu_ops_block_quant import gates, silu_off, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


def ragged(seed, experts, average):
    """Rows for each expert: some without any, the others up to twice `average`."""
    rng = random.Random(seed)
    return [0 if rng.random() < 0.1 else rng.randrange(1, 2 * average + 1) for _ in range(experts)]


@pytest.mark.parametrize("sizes", [ragged(1, 12, 230), ragged(2, 30, 150), [1500, 0, 5, 900]])
@pytest.mark.parametrize("N,K", [(2048, 1024), (2100, 1111)])
def test_grouped_pairs_large(fw, sizes, N, K):
    """More tiles of 256 x 256 than there are pairs of CTAs."""
    assert sum(-(-s // 256) for s in sizes) * -(-N // 256) > 76
    grouped(fw, sizes, N, K, dt=DT["bf16"], rest=300)
    grouped(fw, sizes, N, K, by_k=False, block=(ROWS, ROWS))


@pytest.mark.parametrize("sizes", [ragged(3, 8, 300), [1000, 0, 77]])
@pytest.mark.parametrize("block", [COLUMNS, SQUARES])
def test_wgrad_large(fw, sizes, block):
    wgrad(fw, sizes, 1000, 1920, block=(block, block))
    wgrad(fw, sizes, 1040, 1300, block=(block, block), dt=DT["bf16"], rest=40)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,H", [(8192, 5760), (8192, 5761), (5000, 8200)])
def test_quant_large(fw, dt, T, H):
    x = values(gen(H), T, H, DT[dt]).clamp(-6e4, 6e4)
    for block, fmt in ((ROWS, "e4m3"), (ROWS, "e5m2"), (COLUMNS, "e4m3"), (SQUARES, "e5m2")):
        r = fw.block_quant(x, block=block, out_dtype=QT[fmt])
        for rows in (slice(0, 256), slice(3968, 4224), slice(T - T % 128 - 128, T)):
            s = slice(rows.start // block[0], blocks(rows.stop, block[0]))
            check_codes(r.q[rows], r.scale[s], x[rows].double(), block, fmt, what=f"{rows} {block} {dt}")
        if block == ROWS:                                    # all of it, bit for bit
            want = (x.float() / spread(r.scale, ROWS, x.shape)).clamp(-448 if fmt == "e4m3" else -57344, 448 if fmt == "e4m3" else 57344)
            assert torch.equal(want.to(QT[fmt]).view(torch.uint8), r.q.view(torch.uint8))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,H", [(8192, 2880), (8192, 2881), (3000, 8200)])
@pytest.mark.parametrize("block", [ROWS, SQUARES])
def test_swiglu_large(fw, dt, T, H, block):
    x = gates(gen(H), T, H, DT[dt])
    r = fw.swiglu_quant(x, block=block, checkpoint=True)
    n = blocks(H)
    for rows in (slice(0, 256), slice(1920, 2176), slice(T - T % 128 - 128, T)):
        gate, up = x[rows].double().chunk(2, 1)
        s = slice(rows.start // block[0], blocks(rows.stop, block[0]))
        check_codes(r.q[rows], r.scale[s], gate * torch.sigmoid(gate) * up, block, "e4m3", off=silu_off(gate).max(), what=f"{rows}")
    for half, k in ((slice(0, H), slice(0, n)), (slice(H, 2 * H), slice(n, 2 * n))):
        scale, v = r.checkpoint_scale[:, k], x[:, half].float()
        top = torch.nn.functional.pad(v.abs(), (0, -H % 128)).view(T, n, 128).amax(2)
        assert torch.equal(scale, (top / torch.full_like(top, 448)).clamp_min(2.0 ** -126))      # (by a number, torch multiplies with its inverse)
        want = (v / spread(scale, ROWS, v.shape)).clamp(-448, 448).to(QT["e4m3"])
        assert torch.equal(want.view(torch.uint8), r.checkpoint[:, half].contiguous().view(torch.uint8))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,H", [(8192, 5760), (8192, 5761), (40000, 264), (40000, 265)])
def test_swiglu_backward_large(fw, dt, T, H):
    g = gen(H)
    kept, _ = operand(g, (T, 2 * H), ROWS)
    n = blocks(H)
    scale = torch.exp(2 * torch.rand(T, 2 * n, generator=g, device=DEV)) / 200
    gy = torch.randn(T, H, generator=g, device=DEV).to(DT[dt])
    got = fw.swiglu_backward(gy, kept, scale)
    for rows in (slice(0, 300), slice(T // 2, T // 2 + 300), slice(T - 300, T)):
        gate, up = value(kept[rows, :H], scale[rows, :n], ROWS), value(kept[rows, H:], scale[rows, n:], ROWS)
        y, s = gy[rows].double(), torch.sigmoid(gate)
        want = torch.cat([y * up * s * (1 + gate * (1 - s)), y * gate * s], 1)
        # as for single rounds: the sigmoid's error, five roundings, and those of the products of codes and scales
        size = torch.cat([(y * up).abs() * (1 + gate.abs()) * s, (y * gate).abs() * s], 1)
        tol = size * torch.cat([silu_off(gate) + 5 * 2.0 ** -24, silu_off(gate)], 1)
        tol = tol + 2.0 ** -23 * (1 + torch.cat([gate, gate], 1).abs()) * torch.cat([size[:, :H], size[:, H:] + y.abs() * s], 1)
        tol = tol + half_step(got.dtype) * (want.abs() + tol) + (2.0 ** -25 if dt == "f16" else 0.0)
        assert bool(((got[rows].double() - want).abs() <= tol).all())
    assert bool(got.isfinite().all())
