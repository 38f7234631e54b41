"""The FP8 products with block scales against 64-bit products of the codes' values: dense in every
layout, by expert, and the experts' weights' gradients."""
import itertools

import pytest
import torch

from block_helpers import (COLUMNS, DEV, DT, QT, ROWS, SQUARES, blocks, check_product, gen, operand, value)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


def flipped(block):
    return (block[1], block[0])


def side(g, rows, K, by_k, block, fmt, extreme=False, pad=0, skip=0):
    """(codes, scales) [rows, K] with blocks as given, the codes of a row (by_k) or of a K position contiguous."""
    shape, bl = ((rows, K), block) if by_k else ((K, rows), flipped(block))
    codes, scale = operand(g, (shape[0], shape[1] + pad), bl, fmt, extreme)
    codes, scale = codes[:, skip:skip + shape[1]], scale[:, :blocks(shape[1], bl[1])]
    return (codes, scale) if by_k else (codes.t(), scale.t())


def dense(fw, M, N, K, *, by_k=(True, True), block=(ROWS, SQUARES), fmt=("e4m3", "e4m3"), dt=torch.float32, seed=0, extreme=False,
          pad=0, skip=0, **kw):
    g = gen(seed)
    a, sa = side(g, M, K, by_k[0], block[0], fmt[0], extreme, pad, skip)
    b, sb = side(g, N, K, by_k[1], block[1], fmt[1], extreme, pad, skip)
    got = fw.block_scaled_mm(a, b.t(), sa, sb.t(), out_dtype=dt, **kw)
    assert got.shape == (M, N) and got.dtype == dt
    check_product(got, value(a, sa, block[0]), value(b, sb, block[1]).t(), f"{M} x {N} x {K} {by_k} {block} {fmt}")
    return a, b, sa, sb, got


SIZES = [(1, 1, 1), (1, 16, 16), (1, 5760, 1920), (2, 17, 33), (3, 64, 256), (5, 300, 1000), (7, 100, 1111), (8, 128, 512), (9, 130, 64),
         (16, 256, 4096), (17, 1000, 1000), (31, 48, 128), (33, 65, 48), (64, 5760, 1920), (100, 96, 1040), (127, 129, 131),
         (128, 128, 128), (129, 257, 1024), (200, 640, 2064), (256, 512, 300), (300, 777, 1025), (512, 512, 5000), (1000, 1500, 100),
         (1024, 768, 2048), (2048, 1920, 640)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(fw, M, N, K):
    for dt in DT.values():
        dense(fw, M, N, K, dt=dt, seed=M + N + K)


@pytest.mark.parametrize("by_k", list(itertools.product([True, False], repeat=2)))
@pytest.mark.parametrize("block", list(itertools.product([ROWS, SQUARES], repeat=2)))
@pytest.mark.parametrize("M,N,K", [(1, 200, 300), (3, 48, 144), (40, 272, 384), (130, 400, 272), (333, 517, 391), (1024, 1280, 640)])
def test_layouts_and_blocks(fw, M, N, K, by_k, block):
    dense(fw, M, N, K, by_k=by_k, block=block, seed=M)


@pytest.mark.parametrize("fmt", list(itertools.product(QT, repeat=2)))
@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (12, 100, 130), (70, 144, 272), (500, 640, 512)])
def test_formats_and_every_code(fw, M, N, K, fmt):
    dense(fw, M, N, K, fmt=fmt, extreme=True, seed=K)
    dense(fw, M, N, K, fmt=fmt, extreme=True, by_k=(False, False), block=(SQUARES, ROWS), seed=K)


@pytest.mark.parametrize("by_k", list(itertools.product([True, False], repeat=2)))
@pytest.mark.parametrize("M,N,K", [(1, 70, 300), (20, 100, 300), (300, 520, 700)])
@pytest.mark.parametrize("pad,skip", [(16, 0), (16, 16), (5, 3), (8, 4)])
def test_strides_and_alignment(fw, M, N, K, by_k, pad, skip):
    dense(fw, M, N, K, by_k=by_k, pad=pad, skip=skip)


@pytest.mark.parametrize("M,N", [(1, 5), (3, 130), (20, 40), (150, 9), (600, 300)])
@pytest.mark.parametrize("by_k", [(True, True), (False, False), (True, False)])
@pytest.mark.parametrize("K", [1, 15, 130])
def test_codes_beside_the_operands_do_not_count(fw, M, N, by_k, K):
    """Operands in the middle of NaN codes, at addresses of every kind."""
    for off in (0, 1, 4, 16):
        g = gen(K)
        parts = []
        for rows, k in ((M, by_k[0]), (N, by_k[1])):
            codes, scale = side(g, rows, K, k, ROWS, "e4m3")
            plain = codes if k else codes.t()
            buf = torch.full((plain.numel() + 256,), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
            at = buf[off:off + plain.numel()].view(plain.shape)
            at.copy_(plain)
            parts.append((at if k else at.t(), scale))
        (a, sa), (b, sb) = parts
        check_product(fw.block_scaled_mm(a, b.t(), sa, sb.t(), out_dtype=torch.float32), value(a, sa, ROWS), value(b, sb, ROWS).t())


@pytest.mark.parametrize("M,N,K", [(1, 40, 256), (20, 200, 300), (300, 600, 520)])
def test_nan_touches_its_row_and_column_alone(fw, M, N, K):
    g = gen(5)
    a, sa = side(g, M, K, True, ROWS, "e4m3")
    b, sb = side(g, N, K, True, ROWS, "e4m3")
    a, b, sb = a.clone(), b.clone(), sb.clone()
    nan = torch.tensor([0x7F], dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    a[M // 2, K - 1] = nan[0]
    b[N // 3, 0] = nan[0]
    sb[N - 1, blocks(K) - 1] = float("nan")
    got = fw.block_scaled_mm(a, b.t(), sa, sb.t(), out_dtype=torch.float32)
    want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    want[M // 2] = True
    want[:, N // 3] = want[:, N - 1] = True
    assert torch.equal(got.isnan(), want)


@pytest.mark.parametrize("M", [1, 20, 700])
def test_empty(fw, M):
    e, s = torch.empty(M, 0, device=DEV).to(QT["e4m3"]), torch.empty(M, 0, device=DEV)
    w, sw = torch.empty(5, 0, device=DEV).to(QT["e4m3"]), torch.empty(5, 0, device=DEV)
    out = torch.full((M, 5), 9.0, device=DEV)
    fw.block_scaled_mm(e, w.t(), s, sw.t(), out_dtype=torch.float32, out=out)
    assert not bool(out.any())
    assert fw.block_scaled_mm(e[:0], w.t(), s[:0], sw.t()).shape == (0, 5)
    assert fw.block_scaled_mm(e, w[:0].t(), s, sw[:0].t()).shape == (M, 0)


@pytest.mark.parametrize("M,N,K,by_k,pad", [(1, 5760, 1920, (True, True), 0), (64, 1000, 2048, (True, True), 0), (64, 1000, 2047, (True, True), 0),
                                            (600, 1000, 2048, (True, False), 0), (600, 1001, 999, (False, False), 0)])
def test_same_bits_on_a_side_stream_in_a_graph_and_with_a_workspace(fw, M, N, K, by_k, pad):
    a, b, sa, sb, want = dense(fw, M, N, K, by_k=by_k)
    torch.cuda.synchronize()
    side_stream = torch.cuda.Stream()
    with torch.cuda.stream(side_stream):
        got = fw.block_scaled_mm(a, b.t(), sa, sb.t(), out_dtype=torch.float32)
    side_stream.synchronize()
    assert torch.equal(got, want)
    need = fw.block_mm_workspace_bytes(a, b.t())
    ws = torch.full((need + 1,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full_like(want, float("nan"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fw.block_scaled_mm(a, b.t(), sa, sb.t(), out_dtype=torch.float32, out=out, workspace=ws)
    a2, b2, sa2, sb2, want2 = dense(fw, M, N, K, by_k=by_k, seed=9)
    for t, u in ((a, a2), (b, b2), (sa, sa2), (sb, sb2)):
        t.copy_(u)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


def test_one_scale_tensor_for_many_rows(fw):
    """Scales of stride zero, and of every other column of a wider tensor."""
    g = gen(3)
    a, _ = operand(g, (40, 512), ROWS)
    b, sb = operand(g, (300, 512), SQUARES)
    one = torch.full((1, 1), 0.02, device=DEV)
    got = fw.block_scaled_mm(a, b.t(), one.expand(40, 4), sb.t(), out_dtype=torch.float32)
    check_product(got, value(a, one.expand(40, 4), ROWS), value(b, sb, SQUARES).t())
    wide = torch.rand(40, 8, generator=g, device=DEV)
    got = fw.block_scaled_mm(a, b.t(), wide[:, ::2], sb.t(), out_dtype=torch.float32)
    check_product(got, value(a, wide[:, ::2], ROWS), value(b, sb, SQUARES).t())


def test_outputs_past_32_bits(fw):
    M, N, K = 66000, 33000, 32
    g = gen(1)
    a, sa = operand(g, (M, K), ROWS)
    b, sb = operand(g, (N, K), SQUARES)
    got = fw.block_scaled_mm(a, b.t(), sa, sb.t())
    for rows in (slice(0, 300), slice(M - 300, M), slice(65000, 65300)):
        check_product(got[rows], value(a[rows], sa[rows], ROWS), value(b, sb, SQUARES).t())


def test_refusals(fw):
    g = gen(0)
    a, sa = operand(g, (4, 256), ROWS)
    b, sb = operand(g, (8, 256), SQUARES)
    f = fw.block_scaled_mm
    bad = [lambda: f(a.float(), b.t(), sa, sb.t()), lambda: f(a, b.t().float(), sa, sb.t()), lambda: f(a, b, sa, sb),
           lambda: f(a, b.t(), sa[:3], sb.t()), lambda: f(a, b.t(), sa[:, :1], sb.t()), lambda: f(a, b.t(), sa, sb),
           lambda: f(a, b.t(), sa.double(), sb.t()), lambda: f(a, b.t(), sa.cpu(), sb.t()), lambda: f(a, b.t().cpu(), sa, sb.t()),
           lambda: f(a[:1].expand(4, 256), b.t(), sa, sb.t()), lambda: f(a[:, ::2], b[:, ::2].t(), sa[:, :1], sb.t()[:1]),
           lambda: f(a[0], b.t(), sa, sb.t()), lambda: f(a, b.t(), sa, sb.t(), out=torch.empty(4, 8, device=DEV)),
           lambda: f(a, b.t(), sa, sb.t(), out_dtype=torch.float32, out=sa.expand(2, 4, 2).reshape(4, 4)),
           lambda: f(a, b.t(), sa, sb.t(), workspace=torch.empty(4096, dtype=torch.uint8))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fw.UnsupportedFeatureError):
        f(a, b.t(), sa, sb.t(), out_dtype=torch.int32)
    with pytest.raises(TypeError):
        f(a, b.t(), sa, None)


# ------------------------------------------------------------------------------- by expert
def ends_of(sizes, first=0):
    return torch.tensor([first] + list(itertools.accumulate(sizes, initial=first))[1:], dtype=torch.int32, device=DEV)


def grouped(fw, sizes, N, K, *, rest=0, first=0, by_k=True, block=(ROWS, SQUARES), fmt=("e4m3", "e4m3"), dt=torch.float32, seed=0, pad=0):
    g = gen(seed)
    E, T = len(sizes), first + sum(sizes) + rest
    offsets = ends_of(sizes, first)
    a, sa = operand(g, (T, K + pad), block[0], fmt[0])
    a, sa = a[:, pad // 2:pad // 2 + K], sa[:, :blocks(K)]
    shape, bl = ((E, N, K), block[1]) if by_k else ((E, K, N), flipped(block[1]))
    b, sb = operand(g, (*shape[:2], shape[2] + pad), bl, fmt[1])
    b, sb = b[..., pad // 2:pad // 2 + shape[2]], sb[..., :blocks(shape[2], bl[1])]
    if by_k:
        b, sb = b.transpose(1, 2), sb.transpose(1, 2)
    got = fw.grouped_block_scaled_mm(a, b, offsets, sa, sb, out_dtype=dt)
    kept = torch.full((T, N), 7.0, dtype=dt, device=DEV)
    assert fw.grouped_block_scaled_mm(a, b, offsets, sa, sb, out_dtype=dt, out=kept) is kept
    va = value(a, sa, block[0])
    ends = offsets.tolist()
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        vb = value(b[e], sb[e], flipped(block[1]))
        check_product(got[lo:hi], va[lo:hi], vb, f"expert {e} of {sizes}, {N} x {K}")
    assert torch.equal(got[first:T - rest], kept[first:T - rest])
    for outside, n in ((slice(0, first), first), (slice(T - rest, T), rest)):
        assert not bool(got[outside].any()) and bool((kept[outside] == 7.0).all()), n
    return a, b, offsets, sa, sb, got


GROUPS = [[1], [0, 1, 0], [5, 0, 3, 1], [8] * 6, [1] * 40, [17, 9, 33, 0, 2], [64, 1, 130], [128, 128], [300, 0, 0, 7, 129], [1000],
          [3, 500, 0, 259, 1, 1]]


@pytest.mark.parametrize("sizes", GROUPS)
@pytest.mark.parametrize("N,K", [(5, 3), (64, 128), (200, 300), (384, 640), (517, 1111)])
def test_grouped(fw, sizes, N, K):
    grouped(fw, sizes, N, K, seed=N)
    grouped(fw, sizes, N, K, seed=N, by_k=False, rest=9, first=2, dt=torch.bfloat16)


@pytest.mark.parametrize("sizes", [[2, 0, 5], [20, 70, 1], [200, 310]])
@pytest.mark.parametrize("block", list(itertools.product([ROWS, SQUARES], repeat=2)))
@pytest.mark.parametrize("fmt", list(itertools.product(QT, repeat=2)))
def test_grouped_blocks_and_formats(fw, sizes, block, fmt):
    grouped(fw, sizes, 272, 400, block=block, fmt=fmt, rest=3)
    grouped(fw, sizes, 272, 400, block=block, fmt=fmt, by_k=False, dt=torch.float16)


@pytest.mark.parametrize("sizes", [[2, 0, 5], [20, 70, 1], [200, 310]])
@pytest.mark.parametrize("pad", [6, 16, 32])
@pytest.mark.parametrize("by_k", [True, False])
def test_grouped_strides(fw, sizes, pad, by_k):
    grouped(fw, sizes, 144, 272, pad=pad, by_k=by_k)


def test_grouped_of_nothing(fw):
    grouped(fw, [], 64, 64, rest=5)
    grouped(fw, [0, 0, 0], 64, 64, rest=4)
    grouped(fw, [0, 0], 64, 64)


def test_grouped_many_experts(fw):
    sizes = [(7 * e) % 5 for e in range(1024)]
    grouped(fw, sizes, 48, 144)
    grouped(fw, [0] * 1000 + [700] + [0] * 23, 48, 144)
    with pytest.raises(fw.UnsupportedFeatureError):
        grouped(fw, [1] * 1025, 16, 16)


@pytest.mark.parametrize("offsets", [[-5, 10, 900], [4, 2, 9], [50, 3, 2], [0, 60, 30], [2 ** 31 - 1, -2 ** 31, 7]])
@pytest.mark.parametrize("N,K", [(64, 128), (300, 400)])
def test_offsets_are_taken_within_the_rows_and_rising(fw, offsets, N, K):
    T, E = 50, 2
    g = gen(2)
    a, sa = operand(g, (T, K), ROWS)
    b, sb = operand(g, (E, N, K), SQUARES)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    ends, last = [], 0
    for o in offsets:
        last = max(last, min(T, max(0, o)))
        ends.append(last)
    got = fw.grouped_block_scaled_mm(a, b.transpose(1, 2), off, sa, sb.transpose(1, 2), out_dtype=torch.float32)
    va = value(a, sa, ROWS)
    for e in range(E):
        check_product(got[ends[e]:ends[e + 1]], va[ends[e]:ends[e + 1]], value(b[e], sb[e], SQUARES).t())
    assert not bool(got[:ends[0]].any()) and not bool(got[ends[-1]:].any())
    ga, sga = operand(g, (T, N), SQUARES)
    xa, sxa = operand(g, (T, K), SQUARES)
    gw = fw.grouped_block_scaled_wgrad(ga, xa, off, sga, sxa)
    for e in range(E):
        rows = slice(ends[e], ends[e + 1])
        check_product(gw[e], value(ga, sga, SQUARES)[rows].t(), value(xa, sxa, SQUARES)[rows])


@pytest.mark.parametrize("sizes,N,K", [([2, 0, 5, 1], 200, 300), ([40, 0, 3, 77], 256, 512), ([300, 200, 0, 190], 512, 391)])
def test_grouped_in_a_graph_with_other_groups(fw, sizes, N, K):
    """Captured once, replayed for another routing: the groups are read on the device."""
    a, b, offsets, sa, sb, _ = grouped(fw, sizes, N, K, rest=4)
    out = torch.empty(a.shape[0], N, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fresh = fw.grouped_block_scaled_mm(a, b, offsets, sa, sb, out_dtype=torch.float32)
        out.copy_(fresh)
    other = ends_of(list(reversed(sizes)))
    offsets.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, fw.grouped_block_scaled_mm(a, b, other, sa, sb, out_dtype=torch.float32))
    ends = other.tolist()
    va = value(a, sa, ROWS)
    for e in range(len(sizes)):
        check_product(out[ends[e]:ends[e + 1]], va[ends[e]:ends[e + 1]], value(b[e], sb[e], SQUARES))


def wgrad(fw, sizes, N, K, *, rest=0, first=0, block=(SQUARES, SQUARES), fmt=("e5m2", "e4m3"), dt=torch.float32, seed=0, pad=0):
    g = gen(seed)
    E, T = len(sizes), first + sum(sizes) + rest
    offsets = ends_of(sizes, first)
    a, sa = operand(g, (T, N + pad), block[0], fmt[0])
    b, sb = operand(g, (T, K + pad), block[1], fmt[1])
    a, sa, b, sb = a[:, pad // 2:pad // 2 + N], sa[:, :blocks(N, block[0][1])], b[:, pad // 2:pad // 2 + K], sb[:, :blocks(K, block[1][1])]
    got = fw.grouped_block_scaled_wgrad(a, b, offsets, sa, sb, out_dtype=dt)
    assert got.shape == (E, N, K) and got.dtype == dt
    ends = offsets.tolist()
    va, vb = value(a, sa, block[0]), value(b, sb, block[1])
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        check_product(got[e], va[lo:hi].t(), vb[lo:hi], f"expert {e} of {sizes}, {N} x {K}")
    return a, b, offsets, sa, sb, got


@pytest.mark.parametrize("sizes", GROUPS + [[127, 2, 127], [130, 126, 256], [0, 128, 0, 64, 64]])
@pytest.mark.parametrize("N,K", [(5, 3), (64, 128), (200, 300), (384, 640), (517, 391)])
def test_wgrad(fw, sizes, N, K):
    wgrad(fw, sizes, N, K, seed=N)
    wgrad(fw, sizes, N, K, seed=N, rest=9, first=2, block=(COLUMNS, COLUMNS), dt=torch.bfloat16)


@pytest.mark.parametrize("sizes", [[2, 0, 5], [20, 300, 1]])
@pytest.mark.parametrize("block", list(itertools.product([COLUMNS, SQUARES], repeat=2)))
@pytest.mark.parametrize("fmt", list(itertools.product(QT, repeat=2)))
@pytest.mark.parametrize("pad", [0, 5, 32])
def test_wgrad_blocks_formats_and_strides(fw, sizes, block, fmt, pad):
    wgrad(fw, sizes, 272, 400, block=block, fmt=fmt, pad=pad, dt=torch.float16 if pad == 5 else torch.float32)


def test_wgrad_of_nothing(fw):
    wgrad(fw, [0, 0, 0], 64, 48)
    wgrad(fw, [0, 3], 64, 48)
    assert wgrad(fw, [], 64, 48, rest=5)[-1].shape == (0, 64, 48)


def test_wgrad_ignores_other_experts_nan(fw):
    """NaN codes in one expert's rows, in the same block of 128 as the others', stay in its gradient."""
    sizes = [30, 60, 50]
    g = gen(4)
    a, sa = operand(g, (140, 256), SQUARES, "e5m2")
    b, sb = operand(g, (140, 144), SQUARES)
    offsets = ends_of(sizes)
    want = fw.grouped_block_scaled_wgrad(a, b, offsets, sa, sb)
    nan = torch.full((60, 256), 0x7F, dtype=torch.uint8, device=DEV)
    a, b = a.clone(), b.clone()
    a[30:90] = nan.view(QT["e5m2"])
    b[30:90] = nan[:, :144].contiguous().view(QT["e4m3"])
    got = fw.grouped_block_scaled_wgrad(a, b, offsets, sa, sb)
    assert bool(got[1].isnan().all())
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_wgrad_out_and_workspace(fw):
    a, b, offsets, sa, sb, want = wgrad(fw, [100, 0, 77], 250, 333)
    out = torch.full((3, 250, 333), float("nan"), device=DEV)
    ws = torch.full((fw.block_wgrad_workspace_bytes(a, b) + 1,), 0xFF, dtype=torch.uint8, device=DEV)
    assert fw.grouped_block_scaled_wgrad(a, b, offsets, sa, sb, out=out, workspace=ws) is out
    assert torch.equal(out, want)


def test_grouped_refusals(fw):
    g = gen(0)
    a, sa = operand(g, (6, 256), ROWS)
    w, sw = operand(g, (2, 48, 256), SQUARES)
    off = ends_of([2, 3])
    b, sb = w.transpose(1, 2), sw.transpose(1, 2)
    f, h = fw.grouped_block_scaled_mm, fw.grouped_block_scaled_wgrad
    ga, sga = operand(g, (6, 48), SQUARES)
    xa, sxa = operand(g, (6, 256), SQUARES)
    at = operand(g, (256, 6), ROWS)[0].t()
    bad = [lambda: f(a, b, off.long(), sa, sb), lambda: f(a, b, off[:2], sa, sb), lambda: f(a, b, off.cpu(), sa, sb),
           lambda: f(a, b[0], off, sa, sb), lambda: f(a, w, off, sa, sb), lambda: f(a, b, off, sa[:4], sb), lambda: f(a, b, off, sa, sb[:1]),
           lambda: f(at, b, off, sa, sb), lambda: f(a, w[:1].expand(2, 48, 256).transpose(1, 2), off, sa, sb),
           lambda: f(a, b, off, sa, sb, out=torch.empty(6, 48, device=DEV)),
           lambda: h(ga, xa, off.long(), sga, sxa), lambda: h(ga.t(), xa, off, sga, sxa), lambda: h(ga, xa[:5], off, sga, sxa),
           lambda: h(ga, xa, off, sga[:, :0], sxa), lambda: h(ga, xa, off[None], sga, sxa), lambda: h(ga[:1].expand(6, 48), xa, off, sga, sxa),
           lambda: h(ga, xa, off, sga, sxa, out=torch.empty(2, 256, 48, device=DEV)),
           lambda: h(ga, xa, off, sga, sxa, out=torch.empty(2, 48, 512, device=DEV)[:, :, ::2])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fw.UnsupportedFeatureError):
        f(a, b, off, sa, sb, out_dtype=torch.float64)


@pytest.mark.parametrize("M,N,K,by_k", [(2600, 2100, 4200, (True, True)), (2500, 2048, 4096, (False, False)), (700, 1100, 3000, (True, False))])
def test_tiles_in_rounds_and_slices(fw, M, N, K, by_k):
    """More tiles than the device holds, the last few in slices of K; and few tiles in slices."""
    for block in ((ROWS, SQUARES), (SQUARES, SQUARES), (ROWS, ROWS)):
        dense(fw, M, N, K, by_k=by_k, block=block, dt=torch.bfloat16)


def big_codes(g, rows, cols):
    """FP8 codes of values within [1, 2) and their negatives, without a 32-bit copy of them."""
    codes = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    codes.random_(0, 256, generator=g)
    return codes.bitwise_and_(0x87).bitwise_or_(0x38).view(torch.float8_e4m3fn)


def test_operands_past_32_bits(fw):
    """More than 2^31 codes on a side: many rows, the same across its rows, and many experts' weights."""
    g = gen(6)
    M, K, N = 70000, 32768, 24
    a, sa = big_codes(g, M, K), torch.rand(M, blocks(K), generator=g, device=DEV)
    b, sb = operand(g, (N, K), SQUARES)
    vb = value(b, sb, SQUARES).t()
    got = fw.block_scaled_mm(a, b.t(), sa, sb.t(), out_dtype=torch.float32)
    for rows in (slice(0, 70), slice(65500, 65600), slice(M - 70, M)):
        check_product(got[rows], value(a[rows], sa[rows], ROWS), vb)
    # [K, M] codes: rows of the product across them
    st = torch.rand(blocks(M), K, generator=g, device=DEV)               # blocks along the M tokens that are summed over
    x, sx = operand(g, (M, 48), COLUMNS)
    got = fw.block_scaled_mm(a.t(), x, st.t(), sx, out_dtype=torch.float32)
    vx = value(x, sx, COLUMNS)
    for cols in (slice(0, 40), slice(K - 40, K)):
        check_product(got[cols], value(a[:, cols], st[:, cols], COLUMNS).t(), vx)
    del a, got
    E, N, K = 36, 8192, 8192
    w = big_codes(g, E * N, K).view(E, N, K)
    sw = torch.rand(E, N // 128, K // 128, generator=g, device=DEV)
    sizes = [0] * E
    sizes[0], sizes[17], sizes[-1] = 3, 150, 41
    offsets = ends_of(sizes)
    t, st = operand(g, (sum(sizes), K), ROWS)
    got = fw.grouped_block_scaled_mm(t, w.transpose(1, 2), offsets, st, sw.transpose(1, 2), out_dtype=torch.float32)
    ends = offsets.tolist()
    for e in (0, 17, E - 1):
        r = slice(ends[e], ends[e + 1])
        check_product(got[r], value(t[r], st[r], ROWS), value(w[e], sw[e], SQUARES).t())
