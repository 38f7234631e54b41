"""The codes of the quantisation in blocks are those of x / scale in fp32, by the scale that is returned, bit for bit: also
halfway between two codes, where a quotient that is off by a little goes to either side."""
import itertools

import pytest
import torch

from block_helpers import COLUMNS, DEV, DT, QMAX, QT, ROWS, SQUARES, blocks, gen, spread
from test_gpu_ops_block_quant import values

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


def check(q, scale, x, block, fmt, what=""):
    want = (x.float() / spread(scale, block, x.shape)).clamp(-QMAX[fmt], QMAX[fmt]).to(QT[fmt])
    off = q.view(torch.uint8) != want.view(torch.uint8)
    assert not bool(off.any()), f"{what}: {int(off.sum())} of {off.numel()} codes off"


@pytest.mark.parametrize("T,H", [(1, 1920), (37, 1111), (130, 257), (300, 512), (1000, 72), (2049, 1040), (1300, 5760), (1300, 5761)])
@pytest.mark.parametrize("block", BLOCKS)
def test_codes(fw, T, H, block):
    for (dt, fmt), seed in zip(itertools.product(DT, QT), range(9)):
        x = values(gen(seed), T, H, DT[dt])
        r = fw.block_quant(x, block=BLOCKS[block], out_dtype=QT[fmt])
        check(r.q, r.scale, x, BLOCKS[block], fmt, f"{dt} {fmt}")


@pytest.mark.parametrize("dt,bits,exponents", [("bf16", 7, 14), ("f16", 10, 5)])
@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("fmt", QT)
def test_every_pair_of_fractions(fw, dt, bits, exponents, block, fmt):
    """Every fraction of a type below every fraction of a block's largest value, some exponents apart."""
    n = 1 << bits
    f = 1 + torch.arange(n, device=DEV) / n
    top = (2 * f[:, None] * torch.ones(exponents, device=DEV)).reshape(-1, 1, 1)
    rest = f[None, :] * torch.exp2(-torch.arange(exponents, device=DEV, dtype=torch.float32))[:, None]
    rest = torch.nn.functional.pad(rest, (0, -n % 127)).reshape(1, exponents, -1, 127).expand(n, -1, -1, -1).reshape(n * exponents, -1, 127)
    x = torch.cat([top.expand(-1, rest.shape[1], 1), rest], 2)               # [blocks, parts, 128]
    x[:, :, 1::2] *= -1
    x = x.to(DT[dt])
    if block == "squares":
        x = (x if bits == 7 else x[::9])[..., None].expand(-1, -1, -1, 128).contiguous().view(-1, 128)
    else:
        x = x.reshape(-1, 128)
        x = x.t().contiguous() if block == "columns" else x
    r = fw.block_quant(x, block=BLOCKS[block], out_dtype=QT[fmt])
    check(r.q, r.scale, x, BLOCKS[block], fmt)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("fmt", QT)
def test_small_and_large_values(fw, block, fmt):
    """Blocks of every size that fp32 has, down to those whose scale is the smallest and up to infinities (NaN codes), and
    zeros of either sign."""
    br, bc = BLOCKS[block]
    for low in range(-149, 128, 23):
        x = torch.randn(2 * br, 23 * bc, generator=gen(low + 200), device=DEV)
        by = torch.exp2(low + torch.arange(23, device=DEV, dtype=torch.float64)).repeat_interleave(bc)
        x = (x.clamp(-3, 3).double() / 4 * by).float()
        x[:, ::5] *= 0.0
        r = fw.block_quant(x, block=BLOCKS[block], out_dtype=QT[fmt])
        check(r.q, r.scale, x, BLOCKS[block], fmt, f"2^{low}")
        zero = (x == 0) & spread(r.scale, BLOCKS[block], x.shape).isfinite()
        assert torch.equal(r.q.view(torch.uint8)[zero] >> 7, x.signbit()[zero].to(torch.uint8))


@pytest.mark.parametrize("T,H", [(77, 1111), (130, 640)])
@pytest.mark.parametrize("block", ["rows", "squares"])
@pytest.mark.parametrize("dt", DT)
def test_codes_of_the_checkpoint(fw, T, H, block, dt):
    x = values(gen(T), T, 2 * H, DT[dt])
    r = fw.swiglu_quant(x, block=BLOCKS[block], checkpoint=True)
    n = blocks(H)
    for half, s in ((slice(0, H), slice(0, n)), (slice(H, 2 * H), slice(n, 2 * n))):
        check(r.checkpoint[:, half], r.checkpoint_scale[:, s], x[:, half], ROWS, "e4m3")


@pytest.mark.parametrize("block", BLOCKS)
def test_scales_at_any_address(fw, block):
    """The C call with scales that start at any multiple of four bytes: the same codes and scales, and nothing beside them."""
    from bit_exact_fp8_gb300 import _lib
    x = values(gen(0), 300, 512, torch.bfloat16)
    want = fw.block_quant(x, block=BLOCKS[block])
    for off in (0, 1, 3):
        held = torch.full((want.scale.numel() + 8,), -1.0, device=DEV)
        q = torch.empty_like(want.q)
        scale = held[off:off + want.scale.numel()]
        rc = _lib.load().emu_block_quant(x.data_ptr(), 512, _lib.EMU_OUT_BF16, 300, 512, list(BLOCKS).index(block), 0, q.data_ptr(),
                                         scale.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal(q.view(torch.uint8), want.q.view(torch.uint8)) and torch.equal(scale.view_as(want.scale), want.scale)
        assert bool((held[:off] == -1).all()) and bool((held[off + scale.numel():] == -1).all())
