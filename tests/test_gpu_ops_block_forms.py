"""The forms of the products with block scales that only larger calls take, each with several rounds of its work,
against the formulas in 64 bits."""
import itertools
import random

import pytest

from block_helpers import DT, ROWS, SQUARES
from test_gpu_ops_block_mm import dense, grouped

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    import torch
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


# ------------------------------------------------------------------------------- tiles of 64 tokens
@pytest.mark.parametrize("M,N,K", [(256, 4096, 4096), (192, 4000, 2050), (250, 4100, 1921)])
def test_dense_by_64_tokens(fw, M, N, K):
    for block in itertools.product([ROWS, SQUARES], repeat=2):
        dense(fw, M, N, K, block=block, dt=DT["bf16"])
    dense(fw, M, N, K, by_k=(True, False), fmt=("e5m2", "e4m3"))


@pytest.mark.parametrize("sizes", [[33] * 12, [64] * 9, ragged(1, 24, 48), ragged(2, 40, 40), [0, 100] * 4, [50] + [0] * 3 + [170]])
@pytest.mark.parametrize("N,K", [(1000, 1024), (1536, 2050), (513, 1400)])
def test_grouped_by_64_tokens(fw, sizes, N, K):
    """33 to 64 rows an expert on average; with the widest weights more tiles than the device has SMs, each of 8 blocks of K
    or more, so that every stage of the ring is met in several of its phases and tiles follow one another on an SM."""
    E, T = len(sizes), sum(sizes)
    assert 33 <= -(-T // E) <= 64
    grouped(fw, sizes, N, K, seed=E, dt=DT["bf16"])
    grouped(fw, sizes, N, K, seed=E, block=(ROWS, ROWS), by_k=False)


# ------------------------------------------------------------------------------- slices of K
@pytest.mark.parametrize("M,N,K,by_k", [(16, 1920, 2048, True), (16, 2048, 2048, True), (30, 2432, 4100, True), (9, 4608, 2048, True), (16, 4864, 1024, True),
                                        (60, 1930, 2048, True), (1000, 2304, 4096, False), (1000, 2400, 4096, False), (250, 9700, 2048, False)])
def test_few_tiles_in_slices(fw, M, N, K, by_k):
    """As many tiles as there are clusters of two, four and eight CTAs at once, and a few more."""
    dense(fw, M, N, K, by_k=(by_k, True), dt=DT["bf16"])
    dense(fw, M, N, K, by_k=(by_k, True), block=(ROWS, ROWS))


@pytest.mark.parametrize("M,N,K", [(1, 512, 8192), (8, 300, 8193), (3, 64, 16384), (8, 1000, 12290), (1, 130, 65535), (5, 512, 32768)])
def test_few_tokens_of_a_long_k(fw, M, N, K):
    dense(fw, M, N, K, dt=DT["bf16"])
    dense(fw, M, N, K, block=(ROWS, ROWS), fmt=("e5m2", "e4m3"))
