"""CPU tests of the operators around the 8-bit product: their C entry points and their
torch-facing calls refuse bad arguments before anything is launched (no GPU is touched),
and sizes of workspaces."""
import pytest
import torch

FAKE = 1 << 20                    # a non-null aligned address; never dereferenced here
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from bit_exact_fp8_gb300 import _lib, build
    build.build()
    return _lib


def norm(L, **kw):
    a = dict(x=FAKE, ldx=64, r=0, ldr=0, w=FAKE, wt=BF16, t=BF16, T=4, H=64, eps=1e-6, scale=0, qf=0, q=FAKE,
             so=FAKE, ro=0, ldo=0, rstd=FAKE)
    a.update(kw)
    return L.load().emu_rms_norm_quant(a["x"], a["ldx"], a["r"], a["ldr"], a["w"], a["wt"], a["t"], a["T"], a["H"],
                                       a["eps"], a["scale"], a["qf"], a["q"], a["so"], a["ro"], a["ldo"], a["rstd"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(T=1 << 31), -3), (dict(H=(1 << 22) + 1, ldx=1 << 23), -3),
    (dict(t=3), -1), (dict(t=-1), -1), (dict(wt=F16), -1), (dict(qf=3), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(x=0), -1), (dict(w=0), -1), (dict(q=0), -1), (dict(rstd=0), -1),
    (dict(so=0), -1), (dict(ldx=63), -1), (dict(r=2 * FAKE, ldr=63), -1), (dict(ro=2 * FAKE, ldo=63), -1),
    (dict(x=FAKE + 1), -1), (dict(w=FAKE + 2, wt=F32), -1), (dict(rstd=FAKE + 2), -1),
    (dict(ro=FAKE + 128, ldo=64), -1),                     # the output one row further on in the input
    (dict(ro=FAKE, ldo=65), -1),
    (dict(r=2 * FAKE, ldr=64, ro=2 * FAKE + 2, ldo=64), -1)])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status, lib.emu_ops_last_error()
    assert lib.emu_ops_last_error() != ""


def test_norm_of_no_rows_is_nothing(lib):
    assert norm(lib, T=0, x=0, w=0, q=0, rstd=0, so=0) == 0


def norm_grad(L, **kw):
    need = L.load().emu_rms_norm_backward_workspace_bytes(4, 64)
    a = dict(gy=FAKE, ldy=64, h=2 * FAKE, ldh=64, rstd=FAKE, w=FAKE, wt=BF16, gr=0, ldg=0, t=BF16, T=4, H=64,
             gx=3 * FAKE, gw=FAKE, ws=FAKE, wb=need)
    a.update(kw)
    return L.load().emu_rms_norm_backward(a["gy"], a["ldy"], a["h"], a["ldh"], a["rstd"], a["w"], a["wt"], a["gr"],
                                          a["ldg"], a["t"], a["T"], a["H"], a["gx"], a["gw"], a["ws"], a["wb"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(t=4), -1), (dict(wt=F16), -1), (dict(gy=0), -1), (dict(h=0), -1),
    (dict(rstd=0), -1), (dict(w=0), -1), (dict(gx=0), -1), (dict(gw=0), -1), (dict(gw=FAKE + 1), -1),
    (dict(ldy=63), -1), (dict(ldh=63), -1), (dict(gr=FAKE, ldg=63), -1), (dict(ws=0), -1), (dict(wb=1023), -1),
    (dict(ws=FAKE + 8), -1), (dict(gx=FAKE), -1), (dict(gx=2 * FAKE + 64), -1),
    (dict(gr=3 * FAKE, ldg=64), -1)])
def test_norm_grad_refusals(lib, kw, status):
    assert norm_grad(lib, **kw) == status, lib.emu_ops_last_error()
    assert lib.emu_ops_last_error() != ""


def test_norm_grad_workspace(lib):
    f = lib.load().emu_rms_norm_backward_workspace_bytes
    assert f(0, 64) == 0 and f(4, 0) == 0 and f(-1, 64) == 0
    assert f(4, 64) >= 4 * 64 * 4
    assert f(1 << 20, 64) == f(1 << 30, 64)                # does not grow with the rows


def int8(L, **kw):
    a = dict(A=FAKE, lda=32, B=FAKE, ldb=32, M=4, N=8, K=32, sa=FAKE, na=4, sb=FAKE, nb=8, out=FAKE, od=BF16,
             ws=FAKE, wb=1 << 40)
    a.update(kw)
    return L.load().emu_int8_scaled_mm(a["A"], a["lda"], a["B"], a["ldb"], a["M"], a["N"], a["K"], a["sa"], a["na"],
                                       a["sb"], a["nb"], a["out"], a["od"], a["ws"], a["wb"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), -1), (dict(N=-1), -1), (dict(K=-1), -1), (dict(M=1 << 31), -3), (dict(N=1 << 31), -3),
    (dict(K=131072, lda=1 << 18, ldb=1 << 18), -3), (dict(na=3), -1), (dict(nb=4), -1), (dict(na=0), -1),
    (dict(out=0), -1), (dict(sa=0), -1), (dict(sb=0), -1), (dict(A=0), -1), (dict(B=0), -1), (dict(lda=31), -1),
    (dict(ldb=31), -1), (dict(od=3), -1), (dict(out=FAKE + 1), -1), (dict(sa=FAKE + 2), -1)])
def test_int8_refusals(lib, kw, status):
    assert int8(lib, **kw) == status, lib.emu_ops_last_error()
    assert lib.emu_ops_last_error() != ""


def test_int8_empty_and_workspace(lib):
    assert int8(lib, M=0, na=1, A=0, out=0, sa=0) == 0
    assert int8(lib, N=0, nb=1, B=0, out=0, sb=0) == 0
    L = lib.load()
    assert L.emu_int8_workspace_bytes(-1, 8, 8) == 0 and L.emu_int8_workspace_bytes(0, 8, 8) == 0
    need = L.emu_int8_workspace_bytes(8192, 5760, 1920)
    if need:
        a = dict(M=8192, N=5760, K=1920, lda=1920, ldb=1920, na=8192, nb=5760)
        assert int8(lib, **a, wb=need - 1) == -1 and "workspace" in lib.emu_ops_last_error()
        assert int8(lib, **a, ws=0, wb=0) == -1


def logprobs(L, **kw):
    a = dict(x=FAKE, ldx=100, t=BF16, tok=FAKE, T=4, V=100, k=5, lp=FAKE, en=FAKE, lse=FAKE, st=FAKE, tv=FAKE, ti=FAKE)
    a.update(kw)
    return L.load().emu_token_logprobs(a["x"], a["ldx"], a["t"], a["tok"], a["T"], a["V"], a["k"], -100, a["lp"],
                                       a["en"], a["lse"], a["st"], a["tv"], a["ti"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(V=0), -1), (dict(T=1 << 31), -3), (dict(V=(1 << 30) + 1, ldx=1 << 31), -3),
    (dict(t=3), -1), (dict(x=0), -1), (dict(tok=0), -1), (dict(ldx=99), -1), (dict(x=FAKE + 1), -1),
    (dict(tok=FAKE + 4), -1), (dict(k=-1), -1), (dict(k=33), -3), (dict(V=4, k=5), -1), (dict(lp=0), -1),
    (dict(en=0), -1), (dict(lse=0), -1), (dict(st=0), -1), (dict(tv=0), -1), (dict(ti=0), -1), (dict(ti=FAKE + 4), -1)])
def test_logprob_refusals(lib, kw, status):
    assert logprobs(lib, **kw) == status, lib.emu_ops_last_error()
    assert lib.emu_ops_last_error() != ""


def logprobs_grad(L, **kw):
    a = dict(x=FAKE, ldx=100, t=BF16, tok=FAKE, T=4, V=100, st=FAKE, gl=FAKE, ge=FAKE, gx=2 * FAKE, ldo=100)
    a.update(kw)
    return L.load().emu_token_logprobs_backward(a["x"], a["ldx"], a["t"], a["tok"], a["T"], a["V"], -100, a["st"],
                                                a["gl"], a["ge"], a["gx"], a["ldo"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(V=0), -1), (dict(t=4), -1), (dict(x=0), -1), (dict(tok=0), -1), (dict(st=0), -1),
    (dict(gx=0), -1), (dict(ldo=99), -1), (dict(ldx=99), -1), (dict(gx=2 * FAKE + 1), -1),
    (dict(gl=FAKE + 2), -1), (dict(gx=FAKE + 2), -1), (dict(gx=FAKE, ldo=101), -1)])
def test_logprob_grad_refusals(lib, kw, status):
    assert logprobs_grad(lib, **kw) == status, lib.emu_ops_last_error()
    assert lib.emu_ops_last_error() != ""


def test_logprobs_of_no_rows_are_nothing(lib):
    assert logprobs(lib, T=0, x=0, tok=0, lp=0, en=0, lse=0, st=0, tv=0, ti=0) == 0
    assert logprobs_grad(lib, T=0, x=0, tok=0, st=0, gx=0) == 0


def test_python_calls_refuse_host_tensors_and_shapes():
    from bit_exact_fp8_gb300 import (UnsupportedFeatureError, int8_scaled_mm, rms_norm_backward, rms_norm_quant,
                                     token_logprobs, token_logprobs_backward)
    x, w, one = torch.zeros(4, 32), torch.ones(32), torch.ones(1)
    i8 = torch.zeros(4, 32, dtype=torch.int8)
    tok = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: rms_norm_quant(x, w), lambda: rms_norm_quant(x[0], w),
                 lambda: rms_norm_backward(x, x, one, w), lambda: rms_norm_backward(x[0], x[0], one, w),
                 lambda: int8_scaled_mm(i8, i8.t(), one, one), lambda: int8_scaled_mm(i8[0], i8.t(), one, one),
                 lambda: token_logprobs(x, tok), lambda: token_logprobs(x[0], tok),
                 lambda: token_logprobs_backward(x, tok, one, one)):
        with pytest.raises(ValueError):
            call()
    assert issubclass(UnsupportedFeatureError, NotImplementedError)
