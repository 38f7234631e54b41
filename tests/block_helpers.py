"""What the tests of the operators with block scales share: quantisation on the host's terms, values of
codes in 64 bits, and the bounds that the operators state."""
import torch

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
QT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0}
ROWS, COLUMNS, SQUARES = (1, 128), (128, 1), (128, 128)


def blocks(n, size=128):
    return -(-n // size)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def spread(scale, block, shape):
    """The scale of each value of the last two dimensions."""
    r = torch.arange(shape[-2], device=scale.device) // block[0]
    c = torch.arange(shape[-1], device=scale.device) // block[1]
    return scale[..., r, :][..., c]


def value(codes, scale, block):
    return codes.double() * spread(scale.double(), block, codes.shape)


def operand(g, shape, block, fmt="e4m3", extreme=False):
    """(codes, scales) of one operand: codes of every exponent or near-normal ones, positive scales of a factor of 100."""
    if extreme:
        codes = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8).view(QT[fmt])
        codes = torch.where(codes.float().isfinite(), codes.float(), 1.0).to(QT[fmt])
    else:
        codes = (torch.randn(shape, generator=g, device=DEV) * QMAX[fmt] / 8).clamp(-QMAX[fmt], QMAX[fmt]).to(QT[fmt])
    s = torch.rand(*shape[:-2], blocks(shape[-2], block[0]), blocks(shape[-1], block[1]), generator=g, device=DEV)
    return codes, (0.001 * torch.exp(s * 4.6))


def half_step(dt):
    return torch.finfo(dt).eps / 2


def check_product(got, a, b, what=""):
    """a [M, K] and b [K, N] in 64 bits.  A block's products are within 2^-20 of their magnitudes' sum; the scales'
    product and each step of the fp32 sum over blocks round by 2^-24 of at most that; then the type's rounding
    (fp16: below its normal range by half its smallest step, 2^-25; from halfway between its largest value and
    the power of two above it on, 65520, to infinity)."""
    want, mag = a @ b, a.abs() @ b.abs()
    tol = (2.0 ** -20 + (blocks(a.shape[1]) + 2) * 2.0 ** -24) * mag
    past = want.abs() + tol >= torch.finfo(got.dtype).max * (1 + half_step(got.dtype) / 2)
    tol = tol + half_step(got.dtype) * (want.abs() + tol) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    off = (got.double() - want).abs()
    bad = ~((off <= tol) | (past & (got.double() == want.sign() * torch.inf)))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(off / tol.clamp_min(1e-300)).max():.3g} of the bound"


def code_step(v, fmt):
    """The distance of codes at |v|: 2^(exponent - bits), of the subnormals' at the least."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.frexp(v.abs())[1].double() - 1
    return torch.exp2(e.clamp(min=low) - bits)


def tops(x, block):
    rows, cols = x.shape
    held = torch.zeros(blocks(rows, block[0]) * block[0], blocks(cols, block[1]) * block[1], dtype=torch.float64, device=x.device)
    held[:rows, :cols] = x.abs()
    return held.reshape(blocks(rows, block[0]), block[0], -1, block[1]).amax((1, 3))


def check_codes(q, scale, x, block, fmt, off=0.0, what=""):
    """Codes and scales of x (64 bits): the scale within 2^-23 of max / qmax (its division rounds by 2^-24), a code within
    half a step of x / scale, which was computed within 2^-22 (the quotient qmax / max and a product, 2^-24 each, both
    sides of a step).  `off`: how far the values themselves may be off, relative, each and in the maximum."""
    want = (tops(x, block) / QMAX[fmt]).clamp_min(2.0 ** -126)
    assert scale.shape == want.shape, what
    assert bool(((scale.double() - want).abs() <= (2.0 ** -23 + (off.max() if torch.is_tensor(off) else off)) * want).all()), what
    v = x / spread(want, block, x.shape)
    rel = 2.0 ** -22 + 2 * off
    near = code_step(v * (1 + rel), fmt) / 2 + rel * v.abs()
    bad = ~((q.double() - v).abs() <= near)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} codes off"
