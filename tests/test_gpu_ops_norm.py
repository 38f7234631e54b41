"""RMS norm with the residual's addition and an 8-bit output, and its gradient, against
their formulas in 64 bits.

Tolerances.  With u = 2^-24, a thread adds at most H / 32 <= 256 squares in turn before a
tree of at most 10 sums (H <= 8192; the longer rows here add at most 64 a thread), all of
one sign, so the sum of squares is within 270 u, rstd within 140 u + 2 u < 1e-5 and the
scale within as much.  A code is the rounding of a value v within 2e-5 of the exact one,
so it is within half a step of the format, at v, and 2e-5 |v| of it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
QT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "int8": torch.int8}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


def half_step(v, q):
    """Half the distance between the format's values around v (64 bits)."""
    if q == "int8":
        return torch.full_like(v, 0.5)
    bits, low = (3, -6) if q == "e4m3" else (2, -14)
    e = (torch.frexp(v)[1].double() - 1).clamp_min(low)
    return torch.exp2(e - bits) / 2


def check_norm(fw, x, w, r, q, scale, eps=1e-6, **kw):
    h = x.double() + (0 if r is None else r.double())
    h32 = x.float() if r is None else x.float() + r.float()
    got = fw.rms_norm_quant(x, w, r, eps=eps, out_dtype=QT[q], scale=scale, **kw)
    torch.cuda.synchronize()
    rstd = 1 / torch.sqrt(h.square().mean(-1) + eps)
    y = h * rstd[:, None] * w.double()
    torch.testing.assert_close(got.rstd.double(), rstd, rtol=1e-5, atol=0)
    assert got.q.dtype == QT[q] and got.q.shape == x.shape
    if r is not None:
        assert torch.equal(got.residual, h32.to(x.dtype))
    if scale is None:
        want = (y.abs().amax(-1) / QMAX[q]).clamp_min(2.0 ** -126)
        torch.testing.assert_close(got.scale.double(), want, rtol=2e-5, atol=0)
        v = y / got.scale.double()[:, None]
    else:
        assert got.scale is scale
        v = y / scale.double()
    top = QMAX[q]
    v = v.clamp(-128 if q == "int8" else -top, top)
    off = (got.q.float().double() - v).abs()
    assert bool((off <= half_step(v, q) + 2e-5 * v.abs() + 1e-12).all()), float((off - half_step(v, q)).max())
    return got


def make(T, H, dt, seed=0, residual=True, wdt=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=DEV).to(dt)
    r = (3 * torch.randn(T, H, generator=g, device=DEV)).to(dt) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g, device=DEV)).to(wdt or dt)
    return x, w, r


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("q", QT)
@pytest.mark.parametrize("T,H", [(1, 1), (1, 1920), (3, 7), (5, 64), (2, 256), (7, 1111), (33, 1024), (2, 2047),
                                 (3, 2056), (2, 4096), (2, 5760), (3, 8192), (2, 9001), (2, 20480)])
def test_sizes(fw, T, H, dt, q):
    x, w, r = make(T, H, DT[dt], seed=H)
    check_norm(fw, x, w, r, q, None)
    check_norm(fw, x, w, None, q, torch.full((1,), 8.0 / QMAX[q], device=DEV))


@pytest.mark.parametrize("T", [0, 1, 2, 3, 4, 5, 1000, 70000])
def test_rows(fw, T):
    x, w, r = make(T, 128, torch.bfloat16)
    check_norm(fw, x, w, r, "int8", None)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_weight_in_fp32(fw, dt):
    for H in (1111, 1920):
        x, w, r = make(6, H, DT[dt], wdt=torch.float32)
        check_norm(fw, x, w, r, "e4m3", None)


@pytest.mark.parametrize("H", [1111, 1920, 20480])
@pytest.mark.parametrize("pad,skip", [(8, 0), (8, 8), (3, 1)])
def test_row_strides_and_alignment(fw, H, pad, skip):
    wide_x, _, wide_r = make(9, H + pad, torch.bfloat16)
    _, w, _ = make(1, H + skip, torch.bfloat16)
    x, r, w = wide_x[:, skip:skip + H], wide_r[:, skip:skip + H], w[skip:]
    out = torch.full((9, H + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    got = check_norm(fw, x, w, r, "e4m3", None, residual_out=out[:, skip:skip + H])
    assert got.residual.data_ptr() == out[:, skip:].data_ptr()
    out[:, skip:skip + H] = 7.0
    assert bool((out == 7.0).all())                        # nothing written beside the rows


@pytest.mark.parametrize("H", [100, 1920, 5761, 20480, 40001])
def test_residual_updated_in_place(fw, H):
    x, w, r = make(5, H, torch.bfloat16)
    want = check_norm(fw, x, w, r, "int8", None)
    for place in (r.clone(), x.clone()):
        a, b = (x, place) if place.data_ptr() != x.data_ptr() and torch.equal(place, r) else (place, r)
        got = fw.rms_norm_quant(a, w, b, out_dtype=torch.int8, residual_out=place)
        assert got.residual is place
        assert torch.equal(place, want.residual) and torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)


def test_zero_and_tiny_rows(fw):
    x = torch.zeros(4, 640, device=DEV)
    x[1] = 1e-30                                           # far below eps: y = 1e-27
    x[2, 5] = 1e-42                                        # a subnormal value alone
    x[3] = 1.0
    w = torch.ones(640, device=DEV)
    got = fw.rms_norm_quant(x, w, out_dtype=torch.int8)
    assert float(got.scale[0]) == 2.0 ** -126 and not bool(got.q[0].any())
    assert float(got.scale[2]) == 2.0 ** -126 and not bool(got.q[2].any())
    assert bool((got.q[1] == 127).all()) and bool((got.q[3] == 127).all())
    torch.testing.assert_close(got.scale[1].item(), 1e-27 / 127, rtol=1e-5, atol=0)


def test_scales_near_the_least(fw):
    """rstd of 1e3 and products h w of 1e-37: y = 1e-34, whose scale 1e-36 is above the least, and rstd / scale
    is past fp32's range."""
    x = torch.full((2, 640), 1e-10, device=DEV)
    x[1, ::2] = -1e-10
    for q in QT:
        check_norm(fw, x, torch.full((640,), 1e-27, device=DEV), None, q, None)


@pytest.mark.parametrize("q", QT)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_values_stay_in_their_row(fw, q, bad):
    for H in (640, 1111, 40000):
        x, w, r = make(5, H, torch.bfloat16)
        clean = fw.rms_norm_quant(x, w, r, out_dtype=QT[q])
        x[3, H // 2] = bad
        got = fw.rms_norm_quant(x, w, r, out_dtype=QT[q])
        assert bool(got.scale[3].isnan())
        keep = [0, 1, 2, 4]
        assert torch.equal(got.q.view(torch.uint8)[keep], clean.q.view(torch.uint8)[keep])
        assert torch.equal(got.scale[keep], clean.scale[keep])


def test_static_scale_saturates(fw):
    x = torch.tensor([[1.0, -1.0, 30.0, -30.0] * 16], device=DEV)
    w = torch.ones(64, device=DEV)
    for q in QT:                                           # 1.41 / 1e-6 is past every format's range, 0.047 / 1e-6 not e5m2's
        got = check_norm(fw, x, w, None, q, torch.full((1,), 1e-6, device=DEV))
        low = -128.0 if q == "int8" else -QMAX[q]
        assert got.q.float()[:, 2::4].unique().item() == QMAX[q] and got.q.float()[:, 3::4].unique().item() == low


def test_other_stream_and_graph(fw):
    x, w, r = make(64, 1920, torch.bfloat16)
    want = fw.rms_norm_quant(x, w, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fw.rms_norm_quant(x, w, r)
    side.synchronize()
    assert torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = fw.rms_norm_quant(x, w, r)
    x.copy_(make(64, 1920, torch.bfloat16, seed=5)[0])
    g.replay()
    torch.cuda.synchronize()
    again = fw.rms_norm_quant(x, w, r)
    assert torch.equal(held.q.view(torch.uint8), again.q.view(torch.uint8)) and torch.equal(held.scale, again.scale)


def test_feeds_the_fp8_product(fw):
    """The static-scale output is scaled_mm's operand: the product is the one of the same codes."""
    import oracle
    x, w, r = make(16, 256, torch.bfloat16)
    scale = torch.full((1,), 1 / 32, device=DEV)
    n = fw.rms_norm_quant(x, w, r, scale=scale)
    wq = torch.randn(64, 256, device=DEV).to(torch.float8_e4m3fn)
    one = torch.ones(1, device=DEV)
    y = fw.scaled_mm(n.q, wq.t(), n.scale, one, out_dtype=torch.float32, use_fast_accum=True)
    want = oracle.scaled_mm(n.q.view(torch.uint8).cpu().numpy(), wq.view(torch.uint8).cpu().numpy(), "e4m3fn",
                            "e4m3fn", 1 / 32, 1.0, "f32", True, 1, "hopper")
    assert (y.view(torch.int32).cpu().numpy().view("uint32") == want).all()


def test_offsets_past_32_bits(fw):
    T, H = 530000, 4096                                    # 2.17e9 values
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    tail, w, _ = make(64, H, torch.bfloat16)
    x[-64:] = tail
    x[:64] = tail
    got = fw.rms_norm_quant(x, w, out_dtype=torch.int8)
    want = fw.rms_norm_quant(tail, w, out_dtype=torch.int8)
    assert torch.equal(got.q[-64:], want.q) and torch.equal(got.q[:64], want.q)
    assert torch.equal(got.scale[-64:], want.scale)


# ----------------------------------------------------------------------------- gradient
def grad_formula(gy, h, rstd, w, gr):
    g = gy * w
    c = (g * h).mean(-1, keepdim=True) * rstd[:, None] ** 2
    gx = rstd[:, None] * (g - h * c)
    return (gx if gr is None else gx + gr), (gy * h * rstd[:, None]).sum(0)


def check_grad(fw, gy, h, rstd, w, gr):
    """Bounds: every fp32 step is within u of its terms' sizes; a row's sum has at most
    H / 256 + 20 roundings in a chain (H <= 40001: 180), a column's at most T / 304 + 60."""
    gx, gw = fw.rms_norm_backward(gy, h, rstd, w, gr)
    torch.cuda.synchronize()
    d = [t.double() if t is not None else None for t in (gy, h, rstd, w, gr)]
    want_x, want_w = grad_formula(*d)
    u = 2.0 ** -24
    g = (d[0] * d[3]).abs()
    size = d[2][:, None] * (g + d[1].abs() * (g * d[1].abs()).mean(-1, keepdim=True) * d[2][:, None] ** 2)
    size = size if gr is None else size + d[4].abs()
    assert gx.dtype == h.dtype and gx.shape == h.shape and gw.dtype == torch.float32
    off = (gx.double() - want_x).abs()
    tiny = 2.0 ** -25 if h.dtype == torch.float16 else 1e-38          # half the smallest subnormal step
    assert bool((off <= 200 * u * size + HALF_ULP[h.dtype] * want_x.abs() * 1.01 + tiny).all())
    size = (d[0] * d[1] * d[2][:, None]).abs().sum(0)
    T = gy.shape[0]
    assert bool(((gw.double() - want_w).abs() <= (T / 304 + 64) * u * size + 1e-38).all())


def make_grad(T, H, dt, seed=0, residual=True, wdt=None):
    h, w, gr = make(T, H, dt, seed, residual, wdt)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    gy = (0.1 * torch.randn(T, H, generator=g, device=DEV)).to(dt)
    rstd = (h.float().square().mean(-1) + 1e-6).rsqrt()
    return gy, h, rstd, w, gr


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,H", [(1, 1), (1, 1920), (3, 7), (5, 64), (301, 1111), (33, 1024), (2, 2047), (700, 2056),
                                 (9, 4096), (320, 5760), (3, 8192), (2, 9001), (2, 20480), (2, 40001), (5000, 33)])
def test_grad_sizes(fw, T, H, dt):
    check_grad(fw, *make_grad(T, H, DT[dt], seed=H))
    check_grad(fw, *make_grad(T, H, DT[dt], seed=H, residual=False))


def test_grad_weight_in_fp32_and_strides(fw):
    for H in (1111, 1920):
        gy, h, rstd, w, gr = make_grad(6, H + 8, torch.bfloat16, wdt=torch.float32)
        check_grad(fw, gy[:, 8:], h[:, 8:], rstd, w[8:].contiguous(), gr[:, 8:])
        check_grad(fw, gy[:, :H], h[:, 1:H + 1], rstd, w[3:H + 3], gr[:, 2:H + 2])


def test_grad_of_no_rows(fw):
    e = torch.empty(0, 64, device=DEV)
    gx, gw = fw.rms_norm_backward(e, e, torch.empty(0, device=DEV), torch.ones(64, device=DEV))
    assert gx.shape == (0, 64) and not bool(gw.any())


def test_grad_is_the_same_every_time(fw):
    a = make_grad(1000, 1920, torch.bfloat16)
    first = fw.rms_norm_backward(*a)
    for _ in range(3):
        again = fw.rms_norm_backward(*a)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_grad_against_differences(fw):
    """Central differences, in 64 bits, of sum(gy * y) + sum(gr * h): their error is about
    step^2 = 1e-8 of the terms, the kernel's 1e-5 of them."""
    gy, h, rstd, w, gr = make_grad(4, 24, torch.float32)
    gx, gw = fw.rms_norm_backward(gy, h, rstd, w, gr)
    gy, h, w, gr = (t.double().cpu() for t in (gy, h, w, gr))

    def loss(hh, ww):
        return (gy * hh / torch.sqrt(hh.square().mean(-1, keepdim=True) + 1e-6) * ww).sum() + (gr * hh).sum()

    d = 1e-4
    for t in range(4):
        for c in range(0, 24, 5):
            e = torch.zeros_like(h)
            e[t, c] = d
            assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - gx[t, c].double().cpu()) < 1e-4
    for c in range(24):
        e = torch.zeros_like(w)
        e[c] = d
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - gw[c].double().cpu()) < 1e-4


def test_refusals(fw):
    x, w, r = make(4, 64, torch.bfloat16)
    bad = [lambda: fw.rms_norm_quant(x.double(), w), lambda: fw.rms_norm_quant(x, w[:-1]),
           lambda: fw.rms_norm_quant(x, w.half()), lambda: fw.rms_norm_quant(x, w, r[:3]),
           lambda: fw.rms_norm_quant(x, w, r.float()), lambda: fw.rms_norm_quant(x.t(), w[:4]),
           lambda: fw.rms_norm_quant(x, w, scale=torch.ones(4, device=DEV)),
           lambda: fw.rms_norm_quant(x, w, scale=torch.ones(1)),
           lambda: fw.rms_norm_quant(x, w, out=torch.empty(4, 64, device=DEV)),
           lambda: fw.rms_norm_quant(x[:1].expand(4, 64), w), lambda: fw.rms_norm_quant(x, w, eps=-1.0),
           lambda: fw.rms_norm_quant(x[1:], w, residual_out=x[:3]),
           lambda: fw.rms_norm_backward(r, x, torch.ones(3, device=DEV), w),
           lambda: fw.rms_norm_backward(r.float(), x, torch.ones(4, device=DEV), w)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fw.UnsupportedFeatureError):
        fw.rms_norm_quant(x, w, out_dtype=torch.uint8)
    with pytest.raises(fw.UnsupportedFeatureError):
        fw.rms_norm_quant(x, w.clone().requires_grad_())


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,H", [(1, 8), (2, 16), (4, 96), (128, 96), (129, 96), (80, 197), (81, 197), (256, 1920), (512, 1920),
                                 (513, 1920), (128, 1921), (400, 1921), (64, 5761), (40, 16384), (17, 16383), (65, 8200)])
def test_grad_of_few_rows(fw, T, H, dt):
    """Columns summed beside the rows, up to as many rows as that takes, and just above."""
    check_grad(fw, *make_grad(T, H, DT[dt], seed=T + H))
    check_grad(fw, *make_grad(T, H, DT[dt], seed=T + H, residual=False, wdt=torch.float32))


def test_grad_rows_do_not_depend_on_how_columns_are_summed(fw):
    for H in (1920, 1921):
        gy, h, rstd, w, gr = make_grad(2000, H, torch.bfloat16)
        all_rows = fw.rms_norm_backward(gy, h, rstd, w, gr)[0]
        assert torch.equal(fw.rms_norm_backward(gy[:64], h[:64], rstd[:64], w, gr[:64])[0], all_rows[:64])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,H", [(300, 96), (3000, 96), (2600, 512), (2500, 255), (2500, 256), (600, 129), (513, 200), (257, 91),
                                 (40, 768), (40, 776), (1100, 384), (1, 255), (9, 33)])
def test_short_rows(fw, T, H, dt):
    """A warp a row, by vectors and by elements, and just longer rows."""
    x, w, r = make(T, H, DT[dt], seed=T + H)
    check_norm(fw, x, w, r, "e4m3", None)
    check_norm(fw, x, w, None, "int8", torch.full((1,), 8.0 / QMAX["int8"], device=DEV))
    check_grad(fw, *make_grad(T, H, DT[dt], seed=T + H))
    check_grad(fw, *make_grad(T, H, DT[dt], seed=T + H, residual=False, wdt=torch.float32))


@pytest.mark.parametrize("skip", [0, 1, 8])
def test_short_rows_of_wider_ones(fw, skip):
    x, w, r = make(700, 272, torch.bfloat16)
    gy, h, rstd, _, gr = make_grad(700, 272, torch.bfloat16)
    for H in (91, 96, 256):
        c = slice(skip, skip + H)
        check_norm(fw, x[:, c], w[:H].contiguous(), r[:, c], "e4m3", None)
        part = h[:, c].float()
        check_grad(fw, gy[:, c], h[:, c], (part.square().mean(-1) + 1e-6).rsqrt(), w[:H].contiguous(), gr[:, c])
