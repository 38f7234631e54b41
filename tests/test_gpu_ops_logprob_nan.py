"""Rows that hold NaN: every alternative of theirs is NaN with the id -1, whatever the outputs'
memory held before, and the rows beside them come out as without them."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": (torch.float32, 0), "bf16": (torch.bfloat16, 1), "f16": (torch.float16, 2)}
IGNORE = -100


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_exact_fp8_gb300 import _lib, build
    build.build()
    return _lib


def nan_of(dt, sign):
    """A NaN with this sign bit (torch's fills take the sign of none)."""
    bits = {"f32": (0x7FC00000, torch.int32), "bf16": (0x7FC0, torch.int16), "f16": (0x7E00, torch.int16)}[dt]
    word = bits[0] if sign > 0 else bits[0] - (1 << (31 if dt == "f32" else 15))
    return torch.tensor([word], dtype=bits[1], device=DEV).view(DT[dt][0])


def call(lib, x, tok, k, code):
    """The C call, into outputs filled beforehand."""
    T, V = x.shape
    f = {n: torch.full(s, 7.25, device=DEV) for n, s in
         (("lp", (T,)), ("en", (T,)), ("lse", (T,)), ("st", (T, 3)), ("tv", (T, k)))}
    ids = torch.full((T, k), 123456789, dtype=torch.int64, device=DEV)
    st = lib.load().emu_token_logprobs(x.data_ptr(), x.stride(0), code, tok.data_ptr(), T, V, k, IGNORE,
                                       f["lp"].data_ptr(), f["en"].data_ptr(), f["lse"].data_ptr(), f["st"].data_ptr(),
                                       f["tv"].data_ptr(), ids.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0, lib.emu_ops_last_error()
    torch.cuda.synchronize()
    return f, ids


# a warp a row; CTAs of 128, 256 and 512 threads; clusters
FORMS = [(9, 40), (9, 512), (12, 5001), (400, 40003), (400, 70001), (9, 40003), (160, 70001), (9, 131072)]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,V", FORMS)
def test_alternatives_of_rows_of_nan(lib, T, V, dt, sign):
    g = torch.Generator(device=DEV).manual_seed(V)
    clean = (3 * torch.randn(T, V, generator=g, device=DEV)).to(DT[dt][0])
    tok = torch.randint(0, V, (T,), generator=g, device=DEV)
    tok[7] = IGNORE
    nan = nan_of(dt, sign)
    x = clean.clone()
    x[0] = nan                                               # nothing else
    x[2] = nan
    x[2, V // 3] = 1.0                                       # one logit left
    x[3] = nan
    x[3, ::V // 4] = -2.0                                    # four or five, in vectors of their own
    x[4, : V - 3] = nan
    x[5, 1:] = nan                                           # the first one
    x[6] = -math.inf
    x[6, 5:] = nan                                           # nothing above -inf
    bad = [0, 2, 3, 4, 5, 6]
    good = [i for i in range(min(T, 9)) if i not in bad]
    for k in (1, 5, 32):
        f, ids = call(lib, x, tok, k, DT[dt][1])
        assert bool(f["tv"][bad].isnan().all()), (k, f["tv"][bad])
        assert bool((ids[bad] == -1).all()), (k, ids[bad])
        for n in ("lp", "en", "lse"):
            assert bool(f[n][bad].isnan().all())
        f0, ids0 = call(lib, clean, tok, k, DT[dt][1])
        for n in f:
            assert torch.equal(f[n][good], f0[n][good])
        assert torch.equal(ids[good], ids0[good])
