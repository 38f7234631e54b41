"""CPU tests of the operators with block scales: their C entry points and torch-facing calls refuse bad
arguments and overlaps before anything is launched (addresses are never dereferenced)."""
import ctypes

import pytest
import torch

A = [i << 26 for i in range(1, 12)]           # aligned addresses 64 MiB apart
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from bit_exact_fp8_gb300 import _lib, build
    build.build()
    return _lib


def quant(L, **kw):
    a = dict(x=A[0], ldx=256, t=BF16, T=4, H=256, block=0, qf=0, q=A[1], s=A[2])
    a.update(kw)
    return L.load().emu_block_quant(a["x"], a["ldx"], a["t"], a["T"], a["H"], a["block"], a["qf"], a["q"], a["s"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(H=-1), -1), (dict(T=1 << 31), -3), (dict(H=1 << 30, ldx=1 << 31), -3), (dict(t=3), -1), (dict(block=3), -1),
    (dict(block=-1), -1), (dict(qf=2), -1), (dict(x=0), -1), (dict(q=0), -1), (dict(s=0), -1), (dict(ldx=255), -1), (dict(x=A[0] + 1), -1),
    (dict(s=A[2] + 2), -1), (dict(q=A[0]), -1), (dict(s=A[0] + 512), -1), (dict(s=A[1]), -1), (dict(q=A[2], block=1), -1)])
def test_quant_refusals(lib, kw, status):
    assert quant(lib, **kw) == status and lib.emu_ops_last_error() != ""


def test_quant_of_nothing(lib):
    assert quant(lib, T=0, x=0, q=0, s=0) == 0 and quant(lib, H=0, x=0, q=0, s=0) == 0


def swiglu(L, **kw):
    a = dict(x=A[0], ldx=512, t=BF16, T=4, H=256, block=0, qf=0, q=A[1], s=A[2], c=A[3], cs=A[4])
    a.update(kw)
    return L.load().emu_swiglu_quant(a["x"], a["ldx"], a["t"], a["T"], a["H"], a["block"], a["qf"], a["q"], a["s"], a["c"], a["cs"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(T=1 << 31), -3), (dict(t=4), -1), (dict(block=1), -1), (dict(qf=-1), -1), (dict(c=0), -1), (dict(cs=0), -1),
    (dict(x=0), -1), (dict(q=0), -1), (dict(s=0), -1), (dict(ldx=511), -1), (dict(cs=A[4] + 1), -1), (dict(c=A[0]), -1), (dict(cs=A[3]), -1),
    (dict(q=A[3] + 2047), -1)])
def test_swiglu_refusals(lib, kw, status):
    assert swiglu(lib, **kw) == status and lib.emu_ops_last_error() != ""


def swiglu_grad(L, **kw):
    a = dict(gy=A[0], ldy=256, t=BF16, T=4, H=256, c=A[3], cs=A[4], out=A[5])
    a.update(kw)
    return L.load().emu_swiglu_backward(a["gy"], a["ldy"], a["t"], a["T"], a["H"], a["c"], a["cs"], a["out"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(t=-1), -1), (dict(gy=0), -1), (dict(c=0), -1), (dict(cs=0), -1), (dict(out=0), -1), (dict(ldy=255), -1),
    (dict(out=A[5] + 1), -1), (dict(out=A[0]), -1), (dict(out=A[3]), -1), (dict(out=A[4] + 4), -1)])
def test_swiglu_grad_refusals(lib, kw, status):
    assert swiglu_grad(lib, **kw) == status and lib.emu_ops_last_error() != ""


def operand(lib, at, rows, K, scale_at, groups=0, **kw):
    o = dict(codes=at, format=0, row_stride=K, k_stride=1, group_stride=rows * K if groups else 0, scale=scale_at, scale_rows=1,
             scale_row_stride=-(-K // 128), scale_k_stride=1, scale_group_stride=rows * -(-K // 128) if groups else 0)
    o.update(kw)
    return lib.emu_block_operand_t(**o)


def mm(L, a=None, b=None, M=40, N=64, K=256, out=A[4], od=BF16, ws=A[5], wb=1 << 40):
    a = operand(L, A[0], M, K, A[1], **(a or {}))
    b = operand(L, A[2], N, K, A[3], **(b or {}))
    return L.load().emu_block_scaled_mm(ctypes.byref(a), ctypes.byref(b), M, N, K, out, od, ws, wb, 0)


BAD_OPERANDS = [dict(codes=0), dict(scale=0), dict(format=2), dict(scale_rows=64), dict(scale_rows=0), dict(k_stride=2), dict(row_stride=255),
                dict(row_stride=1, k_stride=39), dict(scale_k_stride=-1), dict(scale_row_stride=-2)]


@pytest.mark.parametrize("which", ["a", "b"])
@pytest.mark.parametrize("kw", BAD_OPERANDS)
def test_product_refuses_operands(lib, which, kw):
    if which == "b" and "row_stride" in kw and "k_stride" in kw:
        kw = dict(kw, k_stride=63)
    assert mm(lib, **{which: kw}) == -1 and lib.emu_ops_last_error().startswith(which)


def test_product_refusals(lib):
    for kw, status in ((dict(M=-1), -1), (dict(N=-1), -1), (dict(K=-1), -1), (dict(M=1 << 31), -3), (dict(N=1 << 31), -3), (dict(K=1 << 31), -3),
                       (dict(od=3), -1), (dict(out=0), -1), (dict(out=A[4] + 1), -1), (dict(out=A[0]), -1), (dict(out=A[1]), -1), (dict(out=A[2]), -1),
                       (dict(out=A[3] + 4), -1), (dict(a=dict(scale=A[1] + 2)), -1)):
        assert mm(lib, **kw) == status, kw
        assert lib.emu_ops_last_error() != ""
    L = lib.load()
    assert L.emu_block_scaled_mm(None, None, 4, 4, 4, A[4], BF16, 0, 0, 0) == -1
    assert mm(lib, M=0, a=dict(codes=0, scale=0), out=0) == 0 and mm(lib, N=0, b=dict(codes=0, scale=0), out=0) == 0


def grouped(L, a=None, b=None, off=A[6], E=3, T=40, N=64, K=256, out=A[4], od=BF16, ws=A[5], wb=1 << 40):
    a = operand(L, A[0], T, K, A[1], **(a or {}))
    b = operand(L, A[2], N, K, A[3], groups=E, **(b or {}))
    return L.load().emu_grouped_block_scaled_mm(ctypes.byref(a), ctypes.byref(b), off, E, T, N, K, out, od, 1, ws, wb, 0)


def test_grouped_refusals(lib):
    for kw, status in ((dict(E=-1), -1), (dict(E=1025), -3), (dict(T=-1), -1), (dict(off=0), -1), (dict(off=A[6] + 2), -1), (dict(od=4), -1),
                       (dict(out=A[6]), -1), (dict(out=A[2] + 2 * 64 * 256), -1), (dict(out=A[3] + 4 * 2 * 64 * 2), -1),
                       (dict(b=dict(group_stride=64 * 256 - 1)), -1), (dict(b=dict(group_stride=-1)), -1), (dict(b=dict(scale_group_stride=-1)), -1),
                       (dict(a=dict(row_stride=1, k_stride=40)), -1), (dict(a=dict(codes=0)), -1), (dict(b=dict(codes=0)), -1)):
        assert grouped(lib, **kw) == status, kw
        assert lib.emu_ops_last_error() != ""
    assert grouped(lib, T=0, a=dict(codes=0, scale=0), out=0, off=0) == 0


def wgrad(L, a=None, b=None, off=A[6], E=3, T=40, N=64, K=256, out=A[4], od=F32, ws=A[5], wb=1 << 40):
    rows = dict(row_stride=1, scale_row_stride=1)
    a = operand(L, A[0], N, T, A[1], **{**rows, "k_stride": N, "scale_k_stride": N, **(a or {})})
    b = operand(L, A[2], K, T, A[3], **{**rows, "k_stride": K, "scale_k_stride": K, **(b or {})})
    return L.load().emu_grouped_block_scaled_wgrad(ctypes.byref(a), ctypes.byref(b), off, E, T, N, K, out, od, ws, wb, 0)


def test_wgrad_refusals(lib):
    for kw, status in ((dict(E=-1), -1), (dict(E=1025), -3), (dict(T=-1), -1), (dict(off=0), -1), (dict(od=3), -1), (dict(out=0), -1),
                       (dict(out=A[0]), -1), (dict(out=A[6]), -1), (dict(a=dict(k_stride=63)), -1), (dict(b=dict(k_stride=255)), -1),
                       (dict(a=dict(row_stride=40, k_stride=1)), -1), (dict(b=dict(row_stride=40, k_stride=1)), -1), (dict(b=dict(scale=0)), -1)):
        assert wgrad(lib, **kw) == status, kw
        assert lib.emu_ops_last_error() != ""
    assert wgrad(lib, E=0, off=0, out=0) == 0 and wgrad(lib, N=0, out=0, a=dict(codes=0, scale=0)) == 0


def test_workspaces(lib):
    """None for aligned operands; what is given otherwise has to be enough and aligned."""
    L = lib.load()
    for rows, K, odd in ((40, 256, False), (40, 250, True), (3000, 251, True)):
        a, b = operand(lib, A[0], rows, K, A[1]), operand(lib, A[2], rows, K, A[3])
        need = L.emu_block_mm_workspace_bytes(ctypes.byref(a), ctypes.byref(b), rows, rows, K)
        assert odd or need == 0
        if need:
            kw = dict(M=rows, N=rows, K=K)
            assert mm(lib, **kw, wb=need - 1) == -1 and "workspace" in lib.emu_ops_last_error()
            assert mm(lib, **kw, ws=A[5] + 64) == -1 and mm(lib, **kw, ws=0) == -1
            assert mm(lib, **kw, ws=A[0]) == -1 and mm(lib, **kw, ws=A[4]) == -1 and "overlap" in lib.emu_ops_last_error()


def test_python_calls_refuse_host_tensors():
    import bit_exact_fp8_gb300 as fw
    x, s = torch.zeros(4, 256), torch.ones(4, 2)
    q = x.to(torch.float8_e4m3fn)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: fw.block_quant(x), lambda: fw.block_quant(x[0]), lambda: fw.swiglu_quant(x), lambda: fw.swiglu_backward(x, q, s),
                 lambda: fw.block_scaled_mm(q, q.t(), s, s.t()), lambda: fw.grouped_block_scaled_mm(q, q.t()[None], off, s, s.t()[None]),
                 lambda: fw.grouped_block_scaled_wgrad(q, q, off, s, s), lambda: fw.block_mm_workspace_bytes(q, q.t()),
                 lambda: fw.block_wgrad_workspace_bytes(q, q)):
        with pytest.raises(ValueError):
            call()
