"""The product of 8-bit integers with a scale for each token and channel, bit for bit: the
sums are whole numbers, so 64-bit integer sums (torch on the host, or on the GPU in fp64,
exact below 2^53) scaled in fp32 in the stated order give every output's bits."""
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
    yield pkg
    from bit_exact_fp8_gb300 import _lib
    assert _lib.emu_ops_device_status() == 0


def codes(gen, rows, cols, low=-128, high=128):
    return torch.randint(low, high, (rows, cols), generator=gen, device=DEV, dtype=torch.int8)


def expected(a, w, sa, sb, dt):
    acc = a.double() @ w.double().t() + 0.0                  # a whole number's zero has no sign: 0.0 * -5.0 has
    return (acc.float() * sa.reshape(-1, 1) * sb.reshape(1, -1)).to(dt)


def check(fw, a, w, sa, sb, dt=torch.bfloat16, **kw):
    got = fw.int8_scaled_mm(a, w.t(), sa, sb, out_dtype=dt, **kw)
    want = expected(a, w, sa, sb, dt)
    assert got.dtype == dt and got.shape == want.shape
    bits = torch.int32 if dt == torch.float32 else torch.int16
    bad = (got.contiguous().view(bits) != want.contiguous().view(bits)).sum().item()
    assert bad == 0, f"{bad} of {want.numel()} outputs differ"
    return got


def make(M, N, K, seed=0, low=-128, high=128):
    g = torch.Generator(device=DEV).manual_seed(seed)
    a, w = codes(g, M, K, low, high), codes(g, N, K, low, high)
    sa = 0.001 + 0.01 * torch.rand(M, generator=g, device=DEV)
    sb = 0.001 + 0.01 * torch.rand(N, generator=g, device=DEV)
    return a, w, sa, sb


SIZES = [(1, 1, 1), (1, 16, 16), (1, 5760, 1920), (2, 17, 33), (3, 64, 256), (7, 100, 1111), (8, 128, 512),
         (9, 130, 64), (16, 256, 4096), (17, 1000, 1000), (33, 65, 48), (64, 5760, 1920), (100, 96, 1040),
         (127, 129, 131), (128, 128, 128), (129, 257, 1024), (200, 640, 2064), (256, 512, 3000), (300, 777, 1025),
         (512, 512, 5000), (1000, 1500, 100), (1024, 768, 2048), (2048, 1920, 1920)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(fw, M, N, K):
    a, w, sa, sb = make(M, N, K, seed=M + N + K)
    for dt in DT.values():
        check(fw, a, w, sa, sb, dt)


@pytest.mark.parametrize("M", [1, 4, 12, 64, 150, 500])
@pytest.mark.parametrize("K", [1024, 1040, 4096, 131071])
def test_largest_sums_are_exact(fw, M, K):
    """Every code -128, or the extremes of alternating sign in blocks: sums up to 2^31 - 2^14."""
    N = 200
    one = torch.ones(1, device=DEV)
    a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    a[:, -1] = 127                                           # an odd last term, lost if the sum were rounded
    w[1::2] = 127
    w[:, -1] = 1
    check(fw, a, w, one, one, torch.float32)
    a[:, ::2] = 127
    w[::3, : K // 2] = 127
    check(fw, a, w, one, one, torch.float32)


@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (20, 100, 300), (300, 520, 700), (700, 900, 1024)])
@pytest.mark.parametrize("pad,skip", [(16, 0), (16, 16), (5, 3)])
def test_strides_and_alignment(fw, M, N, K, pad, skip):
    a, w, sa, sb = make(M, N, K + pad)
    check(fw, a[:, skip:skip + K], w[:, skip:skip + K], sa, sb)


@pytest.mark.parametrize("M", [1, 20, 700])
def test_one_scale_for_all(fw, M):
    a, w, sa, sb = make(M, 320, 640)
    one = torch.full((1,), 0.02, device=DEV)
    check(fw, a, w, one, sb)
    check(fw, a, w, sa, one)
    check(fw, a, w, one.reshape(()), one.reshape(1, 1))
    check(fw, a, w, sa.reshape(-1, 1), sb.reshape(1, -1))


@pytest.mark.parametrize("M", [1, 20, 700])
def test_empty_and_single(fw, M):
    one = torch.ones(1, device=DEV)
    e = torch.empty(M, 0, dtype=torch.int8, device=DEV)
    w = torch.empty(5, 0, dtype=torch.int8, device=DEV)
    out = torch.full((M, 5), 9.0, device=DEV)
    fw.int8_scaled_mm(e, w.t(), one, one, out_dtype=torch.float32, out=out)
    assert not bool(out.any())
    assert fw.int8_scaled_mm(e[:0], w.t(), one, one).shape == (0, 5)
    assert fw.int8_scaled_mm(e, w[:0].t(), one, one).shape == (M, 0)


@pytest.mark.parametrize("M,N,K", [(1, 5760, 1920), (64, 1000, 2048), (600, 1000, 2048)])
def test_same_bits_on_a_side_stream_in_a_graph_and_with_a_workspace(fw, M, N, K):
    a, w, sa, sb = make(M, N, K)
    want = check(fw, a, w, sa, sb)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fw.int8_scaled_mm(a, w.t(), sa, sb)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.full((fw.int8_workspace_bytes(M, N, K) + 1,), 0xFF, dtype=torch.uint8, device=DEV)   # NaN everywhere
    out = torch.full_like(want, float("nan"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fw.int8_scaled_mm(a, w.t(), sa, sb, out=out, workspace=ws)
    a2, w2, _, _ = make(M, N, K, seed=9)
    a.copy_(a2)
    w.copy_(w2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, expected(a, w, sa, sb, torch.bfloat16))


def test_outputs_past_32_bits(fw):
    M, N, K = 66000, 33000, 32                               # 2.18e9 outputs
    a, w, sa, sb = make(M, N, K)
    got = fw.int8_scaled_mm(a, w.t(), sa, sb)
    for rows in (slice(0, 300), slice(M - 300, M), slice(65000, 65300)):
        assert torch.equal(got[rows], expected(a[rows], w, sa[rows], sb, torch.bfloat16))


def test_special_scales(fw):
    a, w, sa, sb = make(20, 40, 64)
    sa[3], sb[5], sa[7] = float("inf"), float("nan"), 0.0
    got = fw.int8_scaled_mm(a, w.t(), sa, sb, out_dtype=torch.float32)
    torch.testing.assert_close(got, expected(a, w, sa, sb, torch.float32), rtol=0, atol=0, equal_nan=True)


def test_refusals(fw):
    a, w, sa, sb = make(4, 8, 32)
    bad = [lambda: fw.int8_scaled_mm(a.float(), w.t(), sa, sb), lambda: fw.int8_scaled_mm(a, w.float().t(), sa, sb),
           lambda: fw.int8_scaled_mm(a, w, sa, sb), lambda: fw.int8_scaled_mm(a, w.t().contiguous(), sa, sb),
           lambda: fw.int8_scaled_mm(a, w.t(), sa[:3], sb), lambda: fw.int8_scaled_mm(a, w.t(), sa, sb[:3]),
           lambda: fw.int8_scaled_mm(a, w.t(), sa.double(), sb), lambda: fw.int8_scaled_mm(a, w.t(), sa.cpu(), sb),
           lambda: fw.int8_scaled_mm(a, w.t(), sa, sb, out=torch.empty(4, 8, device=DEV)),
           lambda: fw.int8_scaled_mm(a[:1].expand(4, 32), w.t(), sa, sb)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    big = torch.zeros(1, 131072, dtype=torch.int8, device=DEV)
    one = torch.ones(1, device=DEV)
    with pytest.raises(fw.UnsupportedFeatureError):
        fw.int8_scaled_mm(big, big.t(), one, one)
    with pytest.raises(fw.UnsupportedFeatureError):
        fw.int8_scaled_mm(a, w.t(), sa, sb, out_dtype=torch.int32)


@pytest.mark.parametrize("M,N,K", [(1, 9, 513), (2, 4000, 512), (1, 60, 20000), (3, 61, 20001), (4, 700, 5001), (4, 3001, 2049),
                                   (150, 333, 7001), (300, 5764, 301), (400, 1001, 2999), (700, 255, 4096), (1000, 258, 64),
                                   (3000, 1602, 191)])
def test_forms(fw, M, N, K):
    """K shared by a CTA's warps or not, slices, tiles whose output rows start at any address."""
    a, w, sa, sb = make(M, N, K, seed=M + N + K)
    for dt in DT.values():
        check(fw, a, w, sa, sb, dt)


@pytest.mark.parametrize("M,N", [(1, 5), (3, 130), (20, 40), (150, 9), (600, 300)])
@pytest.mark.parametrize("K", [1, 15, 17, 31, 47, 130, 1023])
def test_codes_beside_the_operands_do_not_count(fw, M, N, K):
    """Operands in the middle of other codes, at every address modulo 16 in turn."""
    a, w, sa, sb = make(M, N, K, seed=K)
    for off in range(0, 16, 3):
        parts = []
        for x in (a, w):
            buf = torch.full((x.numel() + 64,), 127, dtype=torch.int8, device=DEV)
            at = buf[off:off + x.numel()].view(x.shape)
            at.copy_(x)
            parts.append(at)
        check(fw, parts[0], parts[1], sa, sb, torch.float32)
