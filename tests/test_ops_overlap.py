"""The operators' C entry points refuse outputs and workspaces that overlap inputs or one another, before
anything is launched (CPU: the addresses are never dereferenced)."""
import pytest

A = [i << 24 for i in range(1, 16)]          # aligned addresses 16 MiB apart
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from bit_exact_fp8_gb300 import _lib, build
    build.build()
    return _lib


def refused(lib, status):
    return status == -1 and "overlap" in lib.emu_ops_last_error()


@pytest.mark.parametrize("name", ["q", "scale_out", "rstd", "residual_out"])
@pytest.mark.parametrize("other", ["x", "residual", "weight", "q", "scale_out", "rstd", "residual_out"])
@pytest.mark.parametrize("by", [0, 8])
def test_norm(lib, name, other, by):
    if name == other or (name == "residual_out" and other in ("x", "residual") and by == 0):
        return                               # the same tensor; updated in place
    at = dict(x=A[0], residual=A[1], weight=A[2], q=A[3], scale_out=A[4], rstd=A[5], residual_out=A[6])
    at[name] = at[other] + by                # its first value in the other's memory
    T, H = 4, 64
    assert refused(lib, lib.load().emu_rms_norm_quant(at["x"], H, at["residual"], H, at["weight"], BF16, BF16, T, H, 1e-6,
                                                      0, 2, at["q"], at["scale_out"], at["residual_out"], H, at["rstd"], 0))


@pytest.mark.parametrize("name", ["q", "rstd", "residual_out"])
def test_norm_over_the_given_scale(lib, name):
    at = dict(q=A[3], rstd=A[5], residual_out=A[6])
    at[name] = A[7]
    assert refused(lib, lib.load().emu_rms_norm_quant(A[0], 64, A[1], 64, A[2], BF16, BF16, 4, 64, 1e-6, A[7], 2, at["q"], 0,
                                                      at["residual_out"], 64, at["rstd"], 0))


@pytest.mark.parametrize("name", ["grad_x", "grad_weight", "workspace"])
@pytest.mark.parametrize("other", ["grad_y", "hidden", "rstd", "weight", "grad_residual", "grad_x", "grad_weight", "workspace"])
def test_norm_backward(lib, name, other):
    if name == other:
        return
    at = dict(grad_y=A[0], hidden=A[1], rstd=A[2], weight=A[3], grad_residual=A[4], grad_x=A[5], grad_weight=A[6], workspace=A[7])
    at[name] = at[other]
    T, H = 4, 64
    assert refused(lib, lib.load().emu_rms_norm_backward(at["grad_y"], H, at["hidden"], H, at["rstd"], at["weight"], BF16,
                                                         at["grad_residual"], H, BF16, T, H, at["grad_x"], at["grad_weight"],
                                                         at["workspace"], 1 << 20, 0))


@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (40, 64, 64), (2048, 1920, 1920)])
@pytest.mark.parametrize("name", ["out", "workspace"])
@pytest.mark.parametrize("other", ["a", "b", "scale_a", "scale_b", "out", "workspace"])
def test_int8(lib, M, N, K, name, other):
    need = lib.load().emu_int8_workspace_bytes(M, N, K)
    if name == other or (need == 0 and "workspace" in (name, other)):
        return
    at = dict(a=A[0], b=A[1], scale_a=A[2], scale_b=A[3], out=A[4], workspace=A[8])
    at[name] = at[other]
    assert refused(lib, lib.load().emu_int8_scaled_mm(at["a"], K, at["b"], K, M, N, K, at["scale_a"], M, at["scale_b"], N,
                                                      at["out"], BF16, at["workspace"], need, 0))


OUTS = ["logprob", "entropy", "lse", "stats", "top_logprobs", "top_ids"]


@pytest.mark.parametrize("name", OUTS)
@pytest.mark.parametrize("other", ["logits", "tokens"] + OUTS)
def test_logprobs(lib, name, other):
    if name == other:
        return
    at = dict(zip(["logits", "tokens"] + OUTS, A))
    at[name] = at[other]
    assert refused(lib, lib.load().emu_token_logprobs(at["logits"], 100, F32, at["tokens"], 4, 100, 5, -100, at["logprob"],
                                                      at["entropy"], at["lse"], at["stats"], at["top_logprobs"], at["top_ids"], 0))


@pytest.mark.parametrize("other", ["tokens", "stats", "grad_logprob", "grad_entropy", "logits"])
def test_logprobs_backward(lib, other):
    at = dict(logits=A[0], tokens=A[1], stats=A[2], grad_logprob=A[3], grad_entropy=A[4])
    over = at[other] + (400 if other == "logits" else 0)     # the logits themselves may be replaced, not a row further
    assert refused(lib, lib.load().emu_token_logprobs_backward(at["logits"], 100, F32, at["tokens"], 4, 100, -100, at["stats"],
                                                               at["grad_logprob"], at["grad_entropy"], over, 100, 0))
