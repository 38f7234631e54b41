"""A row's codes, scale and rstd are the row's own: the same bits whatever kernel the tensors'
alignment leads to, wherever the row stands in its batch and however many rows there are."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


def placed(rows, pad, skip):
    """The rows as a view `skip` elements into rows `pad` longer."""
    T, H = rows.shape
    wide = torch.zeros(T, H + pad, dtype=rows.dtype, device=DEV)
    wide[:, skip:skip + H] = rows
    return wide[:, skip:skip + H]


def layouts(rows):
    """The same rows, lying alike on 16 bytes, alike beside them, and unlike from tensor to tensor."""
    plain, odd, other = (lambda t: t.clone()), (lambda t: placed(t, 8, 3)), (lambda t: placed(t, 5, 1))
    for a, b in ((plain, plain), (odd, odd), (other, other), (plain, odd), (other, plain)):
        yield a(rows[0]), b(rows[1])


def same(a, b, at=slice(None)):
    return (torch.equal(a.q.view(torch.uint8)[at], b.q.view(torch.uint8)) and torch.equal(a.rstd[at], b.rstd)
            and (a.scale.numel() == 1 or torch.equal(a.scale[at], b.scale)))


@pytest.mark.parametrize("q", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("H", [96, 512, 1111, 1920, 5760])
def test_one_arithmetic_in_every_kernel(fw, H, dt, q):
    """Whole numbers, whose squares add up exactly in any order: what is left is the arithmetic after the sum."""
    g = torch.Generator(device=DEV).manual_seed(H)
    x, r = (torch.randint(-40, 41, (400, H), generator=g, device=DEV).to(DT[dt]) for _ in range(2))
    w = (1 + 0.3 * torch.randn(H, generator=g, device=DEV)).to(DT[dt])
    want = fw.rms_norm_quant(x, w, r, out_dtype=q)
    for a, b in layouts((x, r)):
        assert same(fw.rms_norm_quant(a, w, b, out_dtype=q), want)


def codes_step_by_step(x, r, w, q, top, dt):
    """The codes of the formula taken step by step in `dt` (64 bits: the definition's)."""
    h = x.to(dt) + r.to(dt)
    y = h * (1 / torch.sqrt(h.square().mean(-1) + 1e-6))[:, None] * w.to(dt)
    v = y / (y.abs().amax(-1) / top)[:, None]
    if q == torch.int8:
        return v.round()
    bits, low = (3, -6) if q == torch.float8_e4m3fn else (2, -14)
    step = torch.exp2((torch.frexp(v)[1].to(dt) - 1).clamp_min(low) - bits)
    return ((v / step).round() * step).clamp(-top, top)


def test_codes_are_nearer_than_step_by_step(fw):
    """With a scale for each row, y / scale is h w qmax / max|h w|: four roundings to fp32 (two products, the
    largest one's, a quotient) against the six of the formula step by step (y: two, the largest y: two, scale, quotient).
    Codes pass a tie by error in proportion to the root of these, sqrt(4 / 6) = 0.82 as often; 0.9 is asked for."""
    off = {"kernel": 0, "steps": 0}
    for seed in range(4):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x, r = ((torch.randn(4096, 5760, generator=g, device=DEV)).bfloat16() for _ in range(2))
        w = (1 + 0.2 * torch.randn(5760, generator=g, device=DEV)).bfloat16()
        for q, top in ((torch.float8_e4m3fn, 448.0), (torch.float8_e5m2, 57344.0), (torch.int8, 127.0)):
            want = codes_step_by_step(x, r, w, q, top, torch.float64).float()
            off["steps"] += int((codes_step_by_step(x, r, w, q, top, torch.float32) != want).sum())
            off["kernel"] += int((fw.rms_norm_quant(x, w, r, out_dtype=q).q.float() != want).sum())
    assert off["kernel"] <= 0.9 * off["steps"], off


# short rows by vectors and by elements, the ring at each of its sizes (with rows that fill its threads to the last
# column), and rows too long for it
WIDTHS = [33, 91, 255, 256, 512, 640, 700, 768, 1111, 1920, 2047, 2048, 2049, 4096, 4099, 5761, 8192, 16384, 16385, 20481]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("H", WIDTHS)
def test_a_row_is_the_same_wherever_it_stands(fw, H, dt):
    g = torch.Generator(device=DEV).manual_seed(H)
    T = 16
    x, r = (torch.randn(T, H, generator=g, device=DEV).to(DT[dt]) for _ in range(2))
    w = (1 + 0.3 * torch.randn(H, generator=g, device=DEV)).to(DT[dt])
    want = fw.rms_norm_quant(x, w, r, out_dtype=torch.int8)
    for turn in range(1, 9):                                 # every row at other places, eight apart and less
        got = fw.rms_norm_quant(x.roll(turn, 0), w, r.roll(turn, 0), out_dtype=torch.int8)
        assert torch.equal(got.q.roll(-turn, 0), want.q) and torch.equal(got.rstd.roll(-turn, 0), want.rstd)
        assert torch.equal(got.scale.roll(-turn, 0), want.scale) and torch.equal(got.residual.roll(-turn, 0), want.residual)
    for i in range(T):                                       # alone: a view into the batch, and a tensor of its own
        assert same(want, fw.rms_norm_quant(x[i:i + 1], w, r[i:i + 1], out_dtype=torch.int8), slice(i, i + 1))
        assert same(want, fw.rms_norm_quant(x[i:i + 1].clone(), w, r[i:i + 1].clone(), out_dtype=torch.int8), slice(i, i + 1))
    ww = placed(w[None], 3, 1)[0]                            # the weight beside 16 bytes
    for a, b in layouts((x, r)):
        for wt in (w, ww):
            got = fw.rms_norm_quant(a, wt, b, out_dtype=torch.int8)
            assert same(got, want) and torch.equal(got.residual, want.residual)
            got = fw.rms_norm_quant(a[3:4], wt, b[3:4], out_dtype=torch.int8)
            assert same(want, got, slice(3, 4))
    q = torch.empty(T * H + 5, dtype=torch.int8, device=DEV)[5:].view(T, H)      # codes beside 16 bytes
    assert same(fw.rms_norm_quant(x, w, r, out_dtype=torch.int8, out=q), want)
    alone = fw.rms_norm_quant(x, w, out_dtype=torch.float8_e4m3fn)               # without a residual
    for a, _ in layouts((x, r)):
        assert same(fw.rms_norm_quant(a, w, out_dtype=torch.float8_e4m3fn), alone)
    big = x.repeat(60, 1)                                    # many rows
    assert torch.equal(fw.rms_norm_quant(big, w, out_dtype=torch.float8_e4m3fn).q.view(torch.uint8)[-T:], alone.q.view(torch.uint8))


@pytest.mark.parametrize("q", [torch.float8_e4m3fn, torch.float8_e5m2, torch.int8])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H", [64, 91, 255, 700, 1111, 1920, 4096, 20480, 20481])
def test_rows_past_the_range_do_not_look_like_zeros(fw, H, dt, q):
    """Finite values whose squares add up to more than fp32 holds, or rows with an infinity: NaN, not codes of 0."""
    g = torch.Generator(device=DEV).manual_seed(H)
    x = torch.randn(9, H, generator=g, device=DEV).to(DT[dt])
    w = (1 + 0.3 * torch.randn(H, generator=g, device=DEV)).to(DT[dt])
    clean = {s: fw.rms_norm_quant(x, w, out_dtype=q, scale=s) for s in (None, torch.full((1,), 0.03, device=DEV))}
    x[2] *= 1e20
    x[5, H // 2] = 3e19
    x[7, H - 1] = float("inf")
    x[8] *= 1e15                                             # large, but within the range
    for a in (x, placed(x, 8, 3), placed(x, 5, 1)):
        for scale, want in clean.items():
            got = fw.rms_norm_quant(a, w, out_dtype=q, scale=scale)
            codes = got.q.float()
            for i in (2, 5, 7):
                assert bool(got.rstd[i].isnan()) and bool((codes[i] == 0).all() if q == torch.int8 else codes[i].isnan().all())
                assert scale is not None or bool(got.scale[i].isnan())
            for i in (0, 1, 3, 4, 6):
                assert torch.equal(got.q.view(torch.uint8)[i], want.q.view(torch.uint8)[i]) and got.rstd[i] == want.rstd[i]
            assert bool(torch.isfinite(got.rstd[8])) and bool(codes[8].any()) and bool(torch.isfinite(codes[8]).all())
