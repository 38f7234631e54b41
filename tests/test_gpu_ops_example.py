"""The operators run together as a user would: the example's 8-bit output head, its scores
and its gradients, each step against the formulas on the same inputs in 64 bits."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_exact_fp8_gb300 import build
    build.build()
    import score_tokens
    return score_tokens


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("T,H,V", [(1, 256, 64), (33, 1920, 512)])
def test_scores_and_gradients(ex, kind, T, H, V):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, r = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    head, hs = ex.quantise_head(torch.randn(V, H, generator=g, device="cuda") / H ** 0.5 * 3,
                                torch.int8 if kind == "int8" else torch.float8_e4m3fn)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    n, logits = ex.head_logits(x, r, w, head, hs, torch.full((1,), 8 / 448, device="cuda"))
    act = n.q.double() * (n.scale.double()[:, None] if kind == "int8" else n.scale.double())
    wide = head.double() * (hs.double()[:, None] if kind == "int8" else hs.double())
    # int8: exact sums, rounded to bf16; fp8: each block's terms cut to 13 bits, a chain of H / 32 blocks
    size = act.abs() @ wide.abs().t()
    bound = 2.0 ** -8 * (act @ wide.t()).abs() + (1e-6 if kind == "int8" else 2.0 ** -12 * (H / 32 + 32)) * size
    assert bool(((logits.double() - act @ wide.t()).abs() <= bound).all())
    s = ex.token_logprobs(logits, tokens, top_k=5)
    lp = torch.log_softmax(logits.double(), -1)
    torch.testing.assert_close(s.logprob.double(), lp.gather(1, tokens[:, None])[:, 0], rtol=2e-5, atol=2e-5)
    gx, gw = ex.training_gradients(n, logits, s, tokens, w, head, hs, entropy_bonus=0.1)
    # the same by autograd: the loss of the logits, then of the norm given the logits' gradient
    z = logits.double().requires_grad_()
    p = torch.log_softmax(z, -1)
    loss = -p.gather(1, tokens[:, None]).mean() + 0.1 * (p.exp() * p).sum(-1).mean()
    gz, = torch.autograd.grad(loss, z)
    h = n.residual.double().requires_grad_()
    wd = w.double().requires_grad_()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * wd
    wx, ww = torch.autograd.grad(y, (h, wd), gz @ wide)
    # the gradients of the logits, the dequantised head and their product are each rounded to bf16 on the way
    for got, want in ((gx, wx), (gw, ww)):
        assert float((got.double() - want).norm() / want.norm()) < 4 * 2.0 ** -8


def test_main_runs(ex, capsys):
    out = ex.main(["--tokens", "16", "--width", "256", "--vocabulary", "128"])
    assert set(out) == {"fp8", "int8"} and "mean log probability" in capsys.readouterr().out
