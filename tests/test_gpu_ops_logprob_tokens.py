"""What a token outside the vocabulary, an ignored one and a row of nothing or of NaN mean for the
log probability and its gradient, in all their combinations."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
IGNORE = -100


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 512, 50001])
def test_tokens_outside_the_vocabulary(fw, V, dt):
    x = torch.randn(6, V, device=DEV).to(dt)
    x[3:] = -math.inf                                        # the same tokens on rows of nothing
    tok = torch.tensor([V, IGNORE, 7, -1, IGNORE, 7], device=DEV)
    got = fw.token_logprobs(x, tok)
    assert got.logprob.isnan().tolist() == [True, False, False, True, False, False]
    assert got.logprob[[1, 4]].tolist() == [0.0, 0.0] and got.logprob[5] == -math.inf
    one = torch.ones(6, device=DEV)
    for gl in (one, None):
        for ge in (one, None):
            gx = fw.token_logprobs_backward(x, tok, got.stats, gl, ge)
            assert gx.isnan().all(-1).tolist() == [True, False, False, True, False, False], (gl is None, ge is None)
            assert not bool(gx[[1, 2, 4, 5]].isnan().any()) and not bool(gx[4:].any())
            if gl is None and ge is None:
                assert not bool(gx[1:3].any())


@pytest.mark.parametrize("V", [40, 512, 50001])
def test_ignored_tokens_of_rows_of_nan(fw, V):
    x = torch.randn(2, V, device=DEV)
    x[:, V // 2] = math.nan
    tok = torch.tensor([IGNORE, 3], device=DEV)
    got = fw.token_logprobs(x, tok)
    assert got.logprob[0] == 0.0 and bool(got.logprob[1].isnan()) and bool(got.entropy.isnan().all())
