"""A block's sum times its two scales, in every form of the products, for scales of every size that they may have
together."""
import itertools

import pytest
import torch

from block_helpers import COLUMNS, DEV, QT, ROWS, SQUARES, blocks, gen, spread

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


#: powers of two that the two sides' scales lie between: each side's from 2^-90 to 2^88, all products from 2^-126 to 2^118
RANGES = [((-90, -40), (-36, 80)), ((-36, 80), (-90, -40)), ((20, 88), (-88, 30)), ((-88, 30), (20, 88)), ((-1, 1), (-90, 88))]


def scales(g, n, between):
    return torch.exp2(between[0] + (between[1] - between[0]) * torch.rand(n, generator=g, device=DEV))


def ones(rows, K, by_k, at=0):
    """Codes of 1 in one block of K, zeros elsewhere and in every third row, so that each sum is exactly 128 (or the block's
    length) or 0."""
    c = torch.zeros(rows, K, device=DEV)
    c[:, at * 128:(at + 1) * 128] = 1
    c[2::3] = 0
    c = c.to(QT["e4m3"])
    return c if by_k else c.t().contiguous().t()


def check(got, a, b, sa, sb):
    """a [M, K] and b [N, K] with a scale for each row in the one block of K that counts: two factors, each rounded."""
    want = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()[None, :]
    assert bool(((got.double() - want).abs() <= 2 * 2.0 ** -24 * (1 + 2.0 ** -24) * want).all())


def flipped(block):
    return (block[1], block[0])


def per_row(scale, block, rows):
    return spread(scale, (block[0], 1), (rows, 1))[:, 0]


@pytest.mark.parametrize("M,N,K,by_k", [(1, 300, 128, True), (8, 500, 1000, True), (20, 300, 128, True), (40, 700, 64, True), (250, 4100, 1921, True),
                                        (250, 4096, 4096, True), (600, 900, 128, True), (300, 520, 128, False), (300, 520, 700, False),
                                        (2500, 2600, 384, True), (700, 1100, 3000, True)])
@pytest.mark.parametrize("block", list(itertools.product([ROWS, SQUARES], repeat=2)))
@pytest.mark.parametrize("between", RANGES)
def test_dense(fw, M, N, K, by_k, block, between):
    g = gen(M)
    at = blocks(K) // 2
    a, b = ones(M, K, by_k, at), ones(N, K, True, at)
    sa, sb = torch.ones(blocks(M, block[0][0]), blocks(K), device=DEV), torch.ones(blocks(N, block[1][0]), blocks(K), device=DEV)
    sa[:, at], sb[:, at] = (scales(g, s.shape[0], p) for s, p in zip((sa, sb), between))
    got = fw.block_scaled_mm(a, b.t(), sa, sb.t(), out_dtype=torch.float32)
    check(got, a, b, per_row(sa[:, at:at + 1], block[0], M), per_row(sb[:, at:at + 1], block[1], N))


@pytest.mark.parametrize("sizes", [[9, 3, 0, 20], [40, 64, 33], [200, 0, 310]])
@pytest.mark.parametrize("block", list(itertools.product([ROWS, SQUARES], repeat=2)))
@pytest.mark.parametrize("between", RANGES)
def test_grouped(fw, sizes, block, between):
    g = gen(sum(sizes))
    T, N, K, E = sum(sizes), 400, 128, len(sizes)
    off = torch.tensor([0] + list(itertools.accumulate(sizes)), dtype=torch.int32, device=DEV)
    a, b = ones(T, K, True), ones(N, K, True)
    sa = scales(g, blocks(T, block[0][0]), between[0])[:, None]
    sb = scales(g, E * blocks(N, block[1][0]), between[1]).view(E, -1, 1)
    w = b.view(torch.uint8)[None].expand(E, N, K).contiguous().view(QT["e4m3"])
    got = fw.grouped_block_scaled_mm(a, w.transpose(1, 2), off, sa, sb.transpose(1, 2), out_dtype=torch.float32)
    rows, ends = per_row(sa, block[0], T), off.tolist()
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        check(got[r], a[r], b, rows[r], per_row(sb[e], block[1], N))


@pytest.mark.parametrize("block", list(itertools.product([COLUMNS, SQUARES], repeat=2)))
@pytest.mark.parametrize("between", RANGES)
def test_weights_gradients(fw, block, between):
    g = gen(3)
    T, N, K = 128, 600, 520
    a, b = ones(N, T, True), ones(K, T, True)
    sa, sb = scales(g, blocks(N, block[0][1]), between[0])[None], scales(g, blocks(K, block[1][1]), between[1])[None]
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    got = fw.grouped_block_scaled_wgrad(a.t().contiguous(), b.t().contiguous(), off, sa, sb)
    check(got[0], a, b, per_row(sa.t(), flipped(block[0]), N), per_row(sb.t(), flipped(block[1]), K))
