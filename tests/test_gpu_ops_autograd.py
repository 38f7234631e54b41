"""The operators beside autograd: what would pass by it is refused, and what they write in place is
known to it."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_exact_fp8_gb300 as pkg
    from bit_exact_fp8_gb300 import build
    build.build()
    return pkg


def calls(fw):
    """(call, its floating arguments by name), every one of them."""
    T, H, V = 4, 64, 100
    f = lambda *s: torch.randn(*s, device=DEV)               # noqa: E731
    i8 = torch.randint(-9, 9, (T, H), dtype=torch.int8, device=DEV)
    w8 = torch.randint(-9, 9, (V, H), dtype=torch.int8, device=DEV)
    tok = torch.zeros(T, dtype=torch.int64, device=DEV)
    stats = fw.token_logprobs(f(T, V), tok).stats
    return [
        (lambda x, weight, residual, scale, residual_out: fw.rms_norm_quant(x, weight, residual, scale=scale, residual_out=residual_out),
         dict(x=f(T, H), weight=f(H), residual=f(T, H), scale=torch.ones(1, device=DEV), residual_out=f(T, H))),
        (lambda grad_y, hidden, rstd, weight, grad_residual: fw.rms_norm_backward(grad_y, hidden, rstd, weight, grad_residual),
         dict(grad_y=f(T, H), hidden=f(T, H), rstd=f(T), weight=f(H), grad_residual=f(T, H))),
        (lambda scale_a, scale_b, out: fw.int8_scaled_mm(i8, w8.t(), scale_a, scale_b, out_dtype=torch.float32, out=out),
         dict(scale_a=f(T), scale_b=f(V), out=f(T, V))),
        (lambda logits: fw.token_logprobs(logits, tok), dict(logits=f(T, V))),
        (lambda logits, stats, grad_logprob, grad_entropy, out:
         fw.token_logprobs_backward(logits, tok, stats, grad_logprob, grad_entropy, out=out),
         dict(logits=f(T, V), stats=stats, grad_logprob=f(T), grad_entropy=f(T), out=f(T, V)))]


def test_inputs_that_require_grad_are_refused(fw):
    for call, args in calls(fw):
        call(**args)
        for name in args:
            some = dict(args, **{name: args[name].clone().requires_grad_()})
            with pytest.raises(fw.UnsupportedFeatureError, match="requires grad"):
                call(**some)
            with torch.no_grad():                            # as everywhere in torch
                call(**some)
            with torch.inference_mode():
                call(**some)


def test_inputs_with_tangents_are_refused(fw):
    for call, args in calls(fw):
        for name in args:
            with fwd.dual_level():
                dual = fwd.make_dual(args[name], torch.ones_like(args[name]))
                with pytest.raises(fw.UnsupportedFeatureError, match="tangent"):
                    call(**dict(args, **{name: dual}))
            call(**args)


def test_writes_in_place_are_known(fw):
    x, w, r = torch.randn(4, 64, device=DEV), torch.ones(64, device=DEV), torch.randn(4, 64, device=DEV)
    q = torch.empty(4, 64, dtype=torch.int8, device=DEV)
    before = [t._version for t in (x, w, r, q)]
    fw.rms_norm_quant(x, w, r, out_dtype=torch.int8, out=q, residual_out=r)
    assert [t._version - b for t, b in zip((x, w, r, q), before)] == [0, 0, 1, 1]
    out = torch.empty(4, 4, device=DEV)
    one = torch.ones(1, device=DEV)
    fw.int8_scaled_mm(q, q.t(), one, one, out_dtype=torch.float32, out=out)
    assert out._version == 1
    tok = torch.zeros(4, dtype=torch.int64, device=DEV)
    s = fw.token_logprobs(x, tok)
    fw.token_logprobs_backward(x, tok, s.stats, torch.ones(4, device=DEV), out=x)
    assert x._version == before[0] + 1
    # a product that saved r: its gradient would use other values now
    p = torch.ones(4, 64, device=DEV, requires_grad=True)
    y = (p * r).sum()
    fw.rms_norm_quant(x, w, r, residual_out=r)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    with torch.inference_mode():                             # inference tensors have no versions
        t = torch.randn(4, 64, device=DEV)
        fw.rms_norm_quant(x, w, t, residual_out=t)
    assert fw.rms_norm_quant(x, w, t.clone(), residual_out=t).residual is t
