"""Log probabilities of given tokens, entropy, top alternatives and their gradient, against
their definitions in 64 bits.

Tolerances, u = 2^-24: e^t is within 4 u |t| + 4 u of its value, and the weights with |t| > 16
together stay below 2^-7 of a row's sum for V <= 2^17, so z is within about 80 u and log z
within 80 u (absolute); x - lse adds u |lse|.  The entropy's sum of e^t t is within 80 u of
its size.  2e-5 covers each of them for |lse| <= 64, values near 0 taken absolutely.  A
gradient is within 100 u of its largest terms before its rounding to the logits' type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
IGNORE = -100


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


def make(T, V, dt, seed=0, spread=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (spread * torch.randn(T, V, generator=g, device=DEV)).to(dt)
    tok = torch.randint(0, V, (T,), generator=g, device=DEV)
    tok[1::7] = IGNORE
    return x, tok


def definition(x, tok):
    """(logprob, entropy, lse) and every log probability, in 64 bits; the row's largest logit is taken off
    first, so that rows of large equal logits keep their log probabilities."""
    x = x.double()
    empty = torch.isneginf(x).all(-1)
    peak = x.amax(-1).masked_fill(empty, 0.0)
    t = x - peak[:, None]
    logz = t.exp().sum(-1).log()
    lp = t - logz[:, None]
    lp = lp.masked_fill(empty[:, None], -math.inf)
    entropy = torch.special.entr(lp.exp()).sum(-1)
    pad = tok == IGNORE
    at = lp.gather(1, tok.masked_fill(pad, 0)[:, None])[:, 0]
    return at.masked_fill(pad, 0.0), entropy, peak + logz, lp


def check(fw, x, tok, k):
    got = fw.token_logprobs(x, tok, top_k=k)
    torch.cuda.synchronize()
    want = definition(x, tok)
    for a, b in zip(got[:3], want):
        torch.testing.assert_close(a.double(), b, rtol=2e-5, atol=2e-5)
    assert torch.equal(got.stats[:, 0], x.amax(-1).float()) and torch.equal(got.stats[:, 2], got.entropy)
    # equal logits: the lower id first
    v, i = torch.sort(x.float(), dim=-1, descending=True, stable=True)
    assert got.top_ids.dtype == torch.int64 and torch.equal(got.top_ids, i[:, :k])
    lead = want[3].gather(1, i[:, :k])
    torch.testing.assert_close(got.top_logprobs.double(), lead, rtol=2e-5, atol=2e-5)
    return got


SIZES = [(1, 1), (1, 2), (3, 31), (5, 32), (7, 33), (4, 64), (9, 512), (2, 1000), (3, 1024), (2, 1025), (3, 2048),
         (2, 4099), (3, 16384), (2, 32768), (1, 50001), (5, 65536), (1, 131072), (2, 131071), (300, 512), (200, 5001),
         (3, 300001), (1, 1 << 20)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,V", SIZES)
def test_sizes(fw, T, V, dt):
    x, tok = make(T, V, DT[dt], seed=V)
    for k in sorted({0, 1, min(V, 5), min(V, 20), min(V, 32)}):
        check(fw, x, tok, k)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("V", [40, 512, 1500, 5000, 131072])
def test_ties_and_order(fw, V, dt):
    k = 32
    tok = torch.zeros(1, dtype=torch.int64, device=DEV)
    base = torch.zeros(1, V, device=DEV)
    check(fw, base.to(DT[dt]), tok, k)                       # all equal
    signed = base.clone()
    signed[:, ::2] = -0.0                                    # -0 and +0 are equal
    check(fw, signed.to(DT[dt]), tok, k)
    ramp = torch.linspace(-4, 4, V, device=DEV)[None]
    check(fw, ramp.to(DT[dt]), tok, k)                       # rising: every logit is a new largest
    check(fw, ramp.flip(-1).to(DT[dt]), tok, k)
    few = base.clone()
    few[:, V // 2:V // 2 + 3] = 1.0                          # three leaders, then ties from the lowest id on
    check(fw, few.to(DT[dt]), tok, k)
    two = (torch.arange(V, device=DEV) % 2).float()[None]
    check(fw, two.to(DT[dt]), tok, k)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("period", [1, 4, 8, 32, 256, 512, 1024, 2048, 4096, 8192])
def test_leaders_at_one_period(fw, dt, period):
    """The largest logits all at multiples of one distance, as strided work could gather them in one place."""
    V = 131072
    x = torch.randn(2, V, device=DEV)
    x[:, 5 % period::period] += 50.0
    check(fw, x.to(DT[dt]), torch.zeros(2, dtype=torch.int64, device=DEV), 32)


@pytest.mark.parametrize("V", [64, 700, 5000, 131072])
@pytest.mark.parametrize("dt", DT)
def test_masks(fw, V, dt):
    d = DT[dt]
    for low in (-math.inf, torch.finfo(d).min):
        x, tok = make(12, V, d)
        x[0] = low                                           # an empty row, or a uniform one
        x[1, 1:] = low                                       # one logit left
        x[2, :-1] = low
        x[3, 7:] = low                                       # fewer left than alternatives asked for
        x[4, ::2] = low
        tok[1], tok[2], tok[5] = 0, 3, IGNORE
        check(fw, x, tok, 20)
    x, tok = make(6, V, d)
    x[:] = -math.inf
    got = check(fw, x, tok, 5)
    assert got.top_ids.tolist() == [[0, 1, 2, 3, 4]] * 6
    gx = fw.token_logprobs_backward(x, tok, got.stats, torch.ones(6, device=DEV), torch.ones(6, device=DEV))
    assert not bool(gx.any())


@pytest.mark.parametrize("V", [64, 700, 5000, 131072])
@pytest.mark.parametrize("bad", [math.nan, -math.nan, math.inf])
def test_bad_values_stay_in_their_row(fw, V, bad):
    x, tok = make(5, V, torch.float32)
    tok[:] = 2
    tok[4] = IGNORE
    clean = fw.token_logprobs(x, tok, top_k=3)
    x[2, V // 2] = bad
    got = fw.token_logprobs(x, tok, top_k=3)
    for a, b in zip(got, clean):
        keep = [0, 1, 3, 4]
        assert torch.equal(a[keep], b[keep])
    for a in (got.logprob, got.entropy, got.lse):
        assert bool(a[2].isnan())
    assert bool(got.top_logprobs[2].isnan().all()) and got.top_ids[2].tolist() == [-1] * 3


def test_large_and_tiny_logits(fw):
    for spread in (1e-30, 1e4, 1e30):
        x, tok = make(4, 3000, torch.float32, spread=spread)
        got = fw.token_logprobs(x, tok, top_k=4)
        for a, b in zip(got[:3], definition(x, tok)[:3]):
            torch.testing.assert_close(a.double(), b, rtol=2e-5, atol=2e-5)


@pytest.mark.parametrize("V", [512, 50001])
def test_tokens_out_of_range(fw, V):
    x, tok = make(4, V, torch.bfloat16)
    tok[:] = torch.tensor([-1, V, 1 << 40, 0], device=DEV)
    got = fw.token_logprobs(x, tok)
    assert got.logprob.isnan().tolist() == [True, True, True, False]
    gx = fw.token_logprobs_backward(x, tok, got.stats, torch.ones(4, device=DEV))
    assert gx.isnan().all(-1).tolist() == [True, True, True, False] and not bool(gx[3].isnan().any())


@pytest.mark.parametrize("V", [37, 512, 3001, 50000])
@pytest.mark.parametrize("pad,skip", [(8, 0), (8, 8), (5, 3)])
def test_row_strides_and_alignment(fw, V, pad, skip):
    wide, tok = make(9, V + pad, torch.bfloat16)
    tok %= V
    x = wide[:, skip:skip + V]
    got = check(fw, x, tok, 5)
    out = torch.full((9, V + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    check_grad(fw, x, tok, got, out=out[:, skip:skip + V])
    out[:, skip:skip + V] = 7.0
    assert bool((out == 7.0).all())


def check_grad(fw, x, tok, got, entropy=True, **kw):
    T, V = x.shape
    g = torch.Generator(device=DEV).manual_seed(3)
    gl = torch.randn(T, generator=g, device=DEV)
    ge = torch.randn(T, generator=g, device=DEV) if entropy else None
    gx = fw.token_logprobs_backward(x, tok, got.stats, gl, ge, **kw)
    torch.cuda.synchronize()
    _, H, _, lp = definition(x, tok)
    pad = tok == IGNORE
    g64 = gl.double().masked_fill(pad, 0.0)[:, None]
    e64 = ge.double()[:, None] if entropy else 0.0
    empty = torch.isneginf(lp).all(-1, keepdim=True)
    p = torch.exp(lp)
    want = e64 * (torch.special.entr(p) - p * H[:, None]) - g64 * p
    want.scatter_add_(1, tok.masked_fill(pad, 0)[:, None], g64)
    want = want.masked_fill(empty, 0.0)
    size = p * (g64.abs() + (e64.abs() if entropy else 0.0) * (H[:, None] + lp.abs().clamp_max(1e4)))
    size.scatter_add_(1, tok.masked_fill(pad, 0)[:, None], g64.abs())
    size = size.masked_fill(empty, 0.0)
    off = (gx.double() - want).abs()
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 1e-37
    assert gx.dtype == x.dtype
    assert bool((off <= 100 * 2.0 ** -24 * size + HALF_ULP[x.dtype] * want.abs() * 1.01 + tiny).all())
    return gx


@pytest.mark.parametrize("V", [512, 50001])
def test_grad_of_uniform_rows_of_the_lowest_value(fw, V):
    """A mask of large negative numbers that leaves nothing: the row is uniform, p = 1 / V."""
    for low in (torch.finfo(torch.float32).min, -1e9, 1e9):
        x = torch.full((2, V), low, device=DEV)
        tok = torch.tensor([3, IGNORE], device=DEV)
        check_grad(fw, x, tok, check(fw, x, tok, 2))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,V", [(1, 1), (3, 7), (40, 512), (5, 1000), (300, 64), (7, 5001), (3, 65536), (2, 131071)])
def test_grad(fw, T, V, dt):
    x, tok = make(T, V, DT[dt], seed=V)
    x[:, 1::5] = -math.inf
    got = fw.token_logprobs(x, tok)
    check_grad(fw, x, tok, got)
    check_grad(fw, x, tok, got, entropy=False)


def test_grad_in_place(fw):
    for V in (512, 5001):
        x, tok = make(9, V, torch.bfloat16)
        got = fw.token_logprobs(x, tok)
        want = check_grad(fw, x, tok, got)
        place = x.clone()
        g = torch.Generator(device=DEV).manual_seed(3)
        gl, ge = (torch.randn(9, generator=g, device=DEV) for _ in range(2))
        out = fw.token_logprobs_backward(place, tok, got.stats, gl, ge, out=place)
        assert out is place and torch.equal(place, want)


def test_grad_against_differences(fw):
    """Central differences in 64 bits of sum(gl logprob + ge entropy): error about step^2."""
    x, tok = make(3, 19, torch.float32, spread=1.0)
    got = fw.token_logprobs(x, tok)
    gl, ge = torch.tensor([0.7, -1.0, 2.0], device=DEV), torch.tensor([0.3, 1.5, -0.4], device=DEV)
    gx = fw.token_logprobs_backward(x, tok, got.stats, gl, ge).double()
    xd, d = x.double(), 1e-4

    def loss(y):
        lp, en = definition(y, tok)[:2]
        return (gl.double() * lp + ge.double() * en).sum()

    for t in range(3):
        for v in range(19):
            e = torch.zeros_like(xd)
            e[t, v] = d
            assert abs((loss(xd + e) - loss(xd - e)) / (2 * d) - gx[t, v]) < 1e-5


def test_other_stream_and_graph(fw):
    for T, V in ((30, 512), (3, 50001), (1, 131072)):
        x, tok = make(T, V, torch.bfloat16)
        want = fw.token_logprobs(x, tok, top_k=5)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = fw.token_logprobs(x, tok, top_k=5)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = fw.token_logprobs(x, tok, top_k=5)
        x.copy_(make(T, V, torch.bfloat16, seed=4)[0])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, fw.token_logprobs(x, tok, top_k=5)))


def test_offsets_past_32_bits(fw):
    T, V = 16500, 131072                                     # 2.16e9 logits
    x = torch.zeros(T, V, dtype=torch.bfloat16, device=DEV)
    tail, tok_tail = make(8, V, torch.bfloat16)
    x[-8:] = tail
    tok = torch.zeros(T, dtype=torch.int64, device=DEV)
    tok[-8:] = tok_tail
    got = fw.token_logprobs(x, tok, top_k=3)
    want = fw.token_logprobs(tail, tok_tail, top_k=3)
    torch.testing.assert_close(got.lse[-8:], want.lse, rtol=1e-6, atol=0)
    assert torch.equal(got.top_ids[-8:], want.top_ids)
    gl = torch.ones(T, device=DEV)
    gx = fw.token_logprobs_backward(x, tok, got.stats, gl)
    ref = fw.token_logprobs_backward(tail, tok_tail, got.stats[-8:], gl[-8:])
    assert torch.equal(gx[-8:], ref)


def test_refusals(fw):
    x, tok = make(4, 100, torch.bfloat16)
    got = fw.token_logprobs(x, tok)
    one = torch.ones(4, device=DEV)
    bad = [lambda: fw.token_logprobs(x.double(), tok), lambda: fw.token_logprobs(x, tok[:3]),
           lambda: fw.token_logprobs(x, tok.int()), lambda: fw.token_logprobs(x, tok.cpu()),
           lambda: fw.token_logprobs(x, tok, top_k=-1), lambda: fw.token_logprobs(x, tok, top_k=101),
           lambda: fw.token_logprobs(x.t(), tok), lambda: fw.token_logprobs(x[:1].expand(4, 100), tok),
           lambda: fw.token_logprobs_backward(x, tok, got.lse, one),
           lambda: fw.token_logprobs_backward(x, tok, got.stats[:3], one),
           lambda: fw.token_logprobs_backward(x, tok, got.stats, one[:3]),
           lambda: fw.token_logprobs_backward(x, tok, got.stats, one, out=torch.empty(4, 99, device=DEV)),
           lambda: fw.token_logprobs_backward(x[1:], tok[1:], got.stats[1:], one[1:], out=x[:3])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fw.UnsupportedFeatureError):
        fw.token_logprobs(x, tok, top_k=33)
    with pytest.raises(fw.UnsupportedFeatureError):
        fw.token_logprobs(x.clone().requires_grad_(), tok)


@pytest.mark.parametrize("T,V,dt,k", [(2500, 16658, "f16", 5), (2500, 16658, "f16", 9), (310, 16658, "bf16", 32), (160, 33000, "bf16", 20),
                                      (140, 33000, "bf16", 20), (140, 131072, "bf16", 5), (76, 70001, "f32", 32), (77, 70001, "f32", 32),
                                      (6, 33000, "bf16", 32), (12, 228, "bf16", 32)])
def test_forms(fw, T, V, dt, k):
    """Many rows and few, a CTA or a cluster a row, among them rows of equal and of few different logits, whose
    alternatives are the lowest ids."""
    x, tok = make(T, V, DT[dt], seed=T + V)
    x[1] = -math.inf
    x[2] = 1.5
    x[3] = (torch.arange(V, device=DEV) % 3).to(x.dtype)
    x[4, : V // 2] = -math.inf
    x[5, 40:] = -math.inf
    check(fw, x, tok, k)
