"""CPU checks of the norm, 8-bit product and mixture-of-experts entry points:
every argument that a call refuses is refused on the host, before any device
work."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def s12():
    from decode_split12_b200 import build
    from decode_split12_b200 import s12 as mod
    if not build.up_to_date():
        build.build()
    return mod


OK_PTR, ODD, FOUR = C.c_void_p(0x100000), C.c_void_p(0x100001), C.c_void_p(0x100004)


def norm(s12, x=OK_PTR, xt=0, res=None, out=None, rt=0, w=None, rows=4, cols=64, eps=1e-6, y=OK_PTR, q=None, scale=None):
    return s12.lib().s12_rmsnorm(x, xt, res, out, rt, w, rows, cols, eps, y, q, scale, None)


def test_norm_refusals(s12):
    A, S, L = s12.S12_ERR_ARG, s12.S12_ERR_SHAPE, s12.S12_ERR_ALIGN
    assert norm(s12, x=None) == A
    assert norm(s12, y=None) == A
    assert norm(s12, q=OK_PTR) == A  # no scale
    for t in (-1, 2):
        assert norm(s12, xt=t) == A and norm(s12, rt=t) == A
    for eps in (-1e-6, float("inf"), float("nan")):
        assert norm(s12, eps=eps) == A
    assert norm(s12, rows=-1) == A and norm(s12, cols=0) == A and norm(s12, cols=-8) == A
    assert norm(s12, rows=1 << 31) == S
    for cols in (4, 12, 1001, 32776, 1 << 40):
        assert norm(s12, cols=cols) == S
    for name in ("x", "res", "out", "w", "y"):
        assert norm(s12, **{name: ODD}) == L and norm(s12, **{name: FOUR}) == L
    assert norm(s12, q=FOUR, scale=OK_PTR) == L
    assert norm(s12, q=OK_PTR, scale=ODD) == L
    # no rows: nothing to do, whatever the pointers
    assert norm(s12, x=None, y=None, rows=0) == s12.S12_OK


def test_quant_refusals(s12):
    lib = s12.lib()
    A, S, L = s12.S12_ERR_ARG, s12.S12_ERR_SHAPE, s12.S12_ERR_ALIGN

    def quant(x=OK_PTR, t=0, rows=4, cols=64, q=OK_PTR, scale=OK_PTR):
        return lib.s12_quant_i8(x, t, rows, cols, q, scale, None)

    assert quant(x=None) == A and quant(q=None) == A and quant(scale=None) == A and quant(t=5) == A
    assert quant(cols=20) == S and quant(cols=32776) == S and quant(rows=1 << 31) == S
    assert quant(x=ODD) == L and quant(q=ODD) == L and quant(scale=ODD) == L
    assert quant(rows=0, x=None, q=None, scale=None) == s12.S12_OK
