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


def views(s12, E=4, H=256, F=128, version=1):
    out = []
    for rows, cols in ((E * 2 * F, H), (E * H, F)):
        v = s12.View()
        v.rows, v.cols, v.n_tiles, v.version = rows, cols, rows * cols // 128, version
        for f in ("container", "raw", "code", "base", "esc_off", "esc", "tmeta", "row_esc"):
            setattr(v, f, 0x100000)
        out.append(v)
    return out


def test_moe_refusals(s12):
    lib = s12.lib()
    A, S, L = s12.S12_ERR_ARG, s12.S12_ERR_SHAPE, s12.S12_ERR_ALIGN

    def moe(up=None, down=None, E=4, x=OK_PTR, T=3, router=OK_PTR, k=2, y=OK_PTR, yt=0, ids=None, w=None, ws=OK_PTR,
            n=1 << 40, err=None):
        u, d = views(s12)
        return lib.s12_moe(C.byref(up or u), C.byref(down or d), E, x, T, router, k, 1, y, yt, ids, w, ws, n, err, None)

    def routed(E=4, x=OK_PTR, T=3, ids=OK_PTR, w=OK_PTR, k=2, y=OK_PTR, yt=0, ws=OK_PTR, n=1 << 40):
        u, d = views(s12)
        return lib.s12_moe_routed(C.byref(u), C.byref(d), E, x, T, ids, w, k, y, yt, ws, n, None, None)

    for call in (moe, routed):
        assert call(x=None) == A and call(y=None) == A and call(ws=None) == A and call(yt=7) == A
        assert call(E=3) == S and call(E=0) == S and call(E=-1) == S and call(E=257) == S
        assert call(T=-1) == S and call(T=65) == S
        assert call(k=0) == S and call(k=9) == S
        assert call(x=FOUR) == L and call(ws=FOUR) == L and call(y=ODD) == L and call(y=C.c_void_p(0x100002), yt=1) == L
        assert call(T=0, x=None, y=None, ws=None) == s12.S12_OK
    assert moe(k=5) == S  # more than experts
    assert moe(router=None) == A and moe(router=FOUR) == L
    assert moe(ids=ODD) == L and moe(w=ODD) == L and moe(err=ODD) == L
    assert routed(ids=None) == A and routed(w=None) == A and routed(ids=ODD) == L and routed(w=ODD) == L
    # containers: versions that differ, or that the products do not read; shapes that do not belong together
    u2, d2 = views(s12, version=2)
    assert moe(up=u2) == A and moe(down=d2) == A
    u3, d3 = views(s12, version=3)
    assert moe(up=u3, down=d3) == A
    u, d = views(s12)
    assert moe(up=d, down=u) == S
    u.rows += 16
    assert moe(up=u) == S
    assert moe(up=s12.View()) == A
    assert lib.s12_moe_ws_bytes(C.byref(u), C.byref(d), 4, 3, 2) == 0
    u, d = views(s12)
    assert lib.s12_moe_ws_bytes(C.byref(u), C.byref(d), 4, 65, 2) == 0
    assert lib.s12_moe_ws_bytes(C.byref(u), C.byref(d), 4, 3, 9) == 0


def test_gemm_i8_refusals(s12):
    lib = s12.lib()
    A, S, L = s12.S12_ERR_ARG, s12.S12_ERR_SHAPE, s12.S12_ERR_ALIGN

    def call(x=OK_PTR, sx=OK_PTR, w=OK_PTR, sw=OK_PTR, M=3, N=40, K=64, y=OK_PTR, yt=0, ws=OK_PTR, n=1 << 40, err=None):
        return lib.s12_gemm_i8(x, sx, w, sw, M, N, K, y, yt, ws, n, err, None)

    for name in ("x", "sx", "w", "sw", "y", "ws"):
        assert call(**{name: None}) == A
    assert call(yt=2) == A
    assert call(M=-1) == S and call(N=-1) == S and call(M=1 << 31) == S and call(N=1 << 31) == S
    for K in (0, -16, 8, 24, 131072, 1 << 40):
        assert call(K=K) == S
    for name in ("x", "w", "ws"):
        assert call(**{name: FOUR}) == L
    assert call(sx=ODD) == L and call(sw=ODD) == L and call(y=ODD) == L and call(err=ODD) == L
    assert call(y=C.c_void_p(0x100002), yt=1) == L
    assert call(M=0, x=None, y=None) == s12.S12_OK and call(N=0, w=None, ws=None) == s12.S12_OK
    assert lib.s12_gemm_i8_ws_bytes(-1) == 0 and lib.s12_gemm_i8_ws_bytes(1 << 31) == 0


def test_moe_refuses_rows_whose_places_pass_32_bits(s12):
    """512 pairs of rows of more than 2^22 columns: their pieces would no longer count in 31 bits."""
    lib = s12.lib()
    most = 1 << 22
    for H, F in ((most + 128, 128), (128, most + 128)):
        u, d = views(s12, E=1, H=H, F=F)
        assert lib.s12_moe_ws_bytes(C.byref(u), C.byref(d), 1, 1, 1) == 0
        assert lib.s12_moe(C.byref(u), C.byref(d), 1, OK_PTR, 1, OK_PTR, 1, 1, OK_PTR, 0, None, None, OK_PTR, 1 << 40,
                           None, None) == s12.S12_ERR_SHAPE
    u, d = views(s12, E=1, H=most, F=128)
    assert lib.s12_moe(C.byref(u), C.byref(d), 1, OK_PTR, 0, OK_PTR, 1, 1, OK_PTR, 0, None, None, OK_PTR, 0, None,
                       None) == s12.S12_OK
