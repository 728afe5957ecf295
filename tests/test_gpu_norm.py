"""s12_rmsnorm and s12_quant_i8 on the GPU against plain 64-bit arithmetic.

Tolerances.  In FP32 the sum s = x + residual and the product s * w are each
off by at most 2^-24 of themselves.  A thread adds up to 32 squares and ten
more levels of a tree follow, so the sum of squares is off by at most
42 * 2^-24 of itself and its inverse root by half of that plus 2^-24.  All
together v is within 2^-19 of itself.  A BF16 result adds half a step, 2^-8
of the value.  scale is within 2^-19, too.  q = rint(p * (127 / max|p|)) is
taken of a quotient within 127 * 2^-21, so it is within 1/2 + 2^-14 of the
exact one."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

V_REL = 2.0 ** -19
HALF = 0.5 + 2.0 ** -14
COLS = [8, 64, 256, 264, 1000, 1024, 1032, 2056, 4096, 8192, 8200, 14336, 28672, 32768]


@pytest.fixture(scope="module")
def s12(cuda_ok):
    from decode_split12_b200 import s12 as mod
    mod.device_check()
    return mod


def bf16(t):
    return t.view(torch.bfloat16).double()


def exact(x, res, w, eps):
    s = x.double() + (res.double() if res is not None else 0.0)
    v = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    if w is not None:
        v = v * w.double()
    return s, v


def check_y(y, v):
    err = (bf16(y) - v).abs()
    assert bool((err <= v.abs() * (2.0 ** -8 + V_REL) + 1e-40).all()), float((err / v.abs().clamp(min=1e-300)).max())


def check_q(q, scale, v):
    top = v.abs().amax(-1)
    assert bool(((scale.double() - top / 127).abs() <= top / 127 * V_REL).all())
    want = v / (top / 127)[..., None].clamp(min=1e-300)
    assert float((q.double() - want).abs().max()) <= HALF
    assert bool((q.abs().amax(-1)[top > 0] == 127).all())


def make(rows, cols, f32, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.float32 if f32 else torch.bfloat16
    x = torch.randn(rows, cols, generator=g, device="cuda").to(t)
    res = (torch.randn(rows, cols, generator=g, device="cuda") * 4).to(t)
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)
    return x, res, w


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows,f32", [(1, False), (5, True), (301, False)])
def test_norm_both_outputs(s12, rows, cols, f32):
    x, res, w = make(rows, cols, f32, rows * 7 + cols)
    s, v = exact(x, res, w, 1e-6)
    before = res.clone()
    y, q, scale, out = s12.s12_rmsnorm(x, w, 1e-6, residual=res, residual_out=torch.empty_like(res), int8=True)
    check_y(y, v)
    check_q(q, scale, v)
    # the stored sum: one rounding of the exact sum (FP32 sums of BF16 values are rounded twice)
    step = 2.0 ** -24 if f32 else 2.0 ** -8 + 2.0 ** -24
    assert bool(((out.double() - s).abs() <= s.abs() * step).all())
    assert torch.equal(res, before)


@pytest.mark.parametrize("x_f32,res_f32", [(False, True), (True, False)])
@pytest.mark.parametrize("cols", [512, 4104])
def test_norm_mixed_types(s12, x_f32, res_f32, cols):
    x, _, w = make(6, cols, x_f32, 1)
    _, res, _ = make(6, cols, res_f32, 2)
    s, v = exact(x, res, w, 1e-5)
    y, q, scale, out = s12.s12_rmsnorm(x, w, 1e-5, residual=res, bf16=True, int8=True)
    assert out is res  # in place
    check_y(y, v)
    check_q(q, scale, v)
    step = 2.0 ** -24 if res_f32 else 2.0 ** -8 + 2.0 ** -24
    assert bool(((res.double() - s).abs() <= s.abs() * step).all())


def test_norm_without_weight_residual_and_single_outputs(s12):
    x, _, w = make(9, 2048, False, 3)
    _, v = exact(x, None, None, 1e-6)
    y, q, scale, out = s12.s12_rmsnorm(x)
    assert q is None and scale is None and out is None
    check_y(y, v)
    y2, q2, scale2, _ = s12.s12_rmsnorm(x, bf16=False, int8=True)
    assert y2 is None
    check_q(q2, scale2, v)
    # residual_out without a residual is a copy of x
    copy = torch.empty(9, 2048, dtype=torch.float32, device="cuda")
    s12.s12_rmsnorm(x, residual_out=copy)
    assert torch.equal(copy, x.float())
    # a residual written over x itself
    x2 = x.clone()
    s12.s12_rmsnorm(x2, residual=x, residual_out=x2)
    assert torch.equal(x2, (x.float() * 2).to(torch.bfloat16))


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows,f32", [(1, True), (6, False), (301, True)])
def test_quant(s12, rows, cols, f32):
    x, _, _ = make(rows, cols, f32, rows + cols)
    q, scale = s12.s12_quant_i8(x)
    check_q(q, scale, x.double())


def test_quant_rows_of_integers_are_exact(s12):
    """Integers of at most 127 with a 127 in each row come back as they are, with scale 1."""
    g = torch.Generator().manual_seed(0)
    w = torch.randint(-127, 128, (40, 1040), generator=g)
    w[:, 5] = 127
    q, scale = s12.s12_quant_i8(w.to(torch.bfloat16).cuda())
    assert torch.equal(q.cpu(), w.to(torch.int8)) and bool((scale == 1).all())


@pytest.mark.parametrize("cols", [256, 4096])
def test_rows_that_are_zero_tiny_large_or_not_finite(s12, cols):
    x = torch.randn(8, cols, generator=torch.Generator().manual_seed(4))
    x[1] = 0
    x[2] *= 1e-38
    x[3] *= 1e30
    x[4, 7] = float("inf")
    x[5, cols - 1] = float("nan")
    x[6] = 0
    x[6, 3] = 1.4e-45  # the smallest magnitude there is
    x = x.cuda()
    q, scale = s12.s12_quant_i8(x)
    assert bool((q[1] == 0).all()) and float(scale[1]) == 0
    for r in (4, 5):
        assert bool((q[r] == 0).all()) and bool(torch.isnan(scale[r]))
    assert int(q[6, 3]) == 127 and int(q[6].abs().sum()) == 127
    for r in (0, 2, 3, 7):
        want = x[r].double() / (x[r].double().abs().max() / 127)
        assert float((q[r].double() - want).abs().max()) <= HALF
    fine = [0, 3, 7]
    assert bool(((scale[fine].double() * 127 / x[fine].double().abs().amax(1) - 1).abs() <= 2.0 ** -22).all())
    # the norm: zeros stay zeros, also with eps = 0; the other rows are not touched by their neighbours
    for eps in (1e-6, 0.0):
        y, q, scale, _ = s12.s12_rmsnorm(x, eps=eps, int8=True)
        assert bool((bf16(y)[1] == 0).all()) and bool((q[1] == 0).all()) and float(scale[1]) == 0
        assert bool(torch.isnan(scale[4])) and bool(torch.isnan(scale[5])) and bool((q[4:6] == 0).all())
        assert bool(torch.isnan(bf16(y)[5]).all())
        _, v = exact(x[[0, 7]], None, None, eps)
        check_y(y[[0, 7]], v)
        check_q(q[[0, 7]], scale[[0, 7]], v)


def test_no_rows_and_leading_dimensions(s12):
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, q, scale, _ = s12.s12_rmsnorm(torch.empty(0, 64, device="cuda"), w, int8=True)
    assert y.shape == (0, 64) and q.shape == (0, 64) and scale.shape == (0,)
    q, scale = s12.s12_quant_i8(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 64)
    x, _, _ = make(12, 64, True, 5)
    y, q, scale, _ = s12.s12_rmsnorm(x.view(3, 4, 64), w, int8=True)
    assert y.shape == (3, 4, 64) and scale.shape == (3, 4)
    _, v = exact(x, None, None, 1e-6)
    check_y(y.view(12, 64), v)
    check_q(q.view(12, 64), scale.view(12), v)


def test_offsets_past_32_bits(s12):
    """More than 2^31 values: the last rows are those of the same rows alone."""
    cols, rows = 32768, 65540
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.random_(-100, 100, generator=torch.Generator(device="cuda").manual_seed(6))
    q, scale = s12.s12_quant_i8(x)
    q1, scale1 = s12.s12_quant_i8(x[-3:].clone())
    assert torch.equal(q[-3:], q1) and torch.equal(scale[-3:], scale1)
    assert torch.equal(q[:3], s12.s12_quant_i8(x[:3].clone())[0])


def test_neighbours_of_the_outputs_stay(s12):
    """Nothing before or behind the rows is written, with a number of rows that fills no block."""
    x, _, _ = make(5, 200, False, 7)
    y = torch.full((7, 200), 77, dtype=torch.int16, device="cuda")
    q = torch.full((7, 200), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((7,), 77.0, device="cuda")
    s12.s12_rmsnorm(x, y=y[1:6], q=None, bf16=True)
    # int8 rows of 200 bytes: the slice starts 16-byte aligned at row 2
    s12.s12_quant_i8(x, q=q[2:7], scale=scale[1:6])
    assert bool((y[0] == 77).all()) and bool((y[6] == 77).all())
    assert bool((q[:2] == 77).all()) and float(scale[0]) == 77 and float(scale[6]) == 77


def test_another_stream_and_a_replayed_graph(s12):
    x, res, w = make(33, 4096, False, 8)
    y0, q0, s0, r0 = s12.s12_rmsnorm(x, w, residual=res, residual_out=torch.empty_like(res), int8=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y1, q1, s1, r1 = s12.s12_rmsnorm(x, w, residual=res, residual_out=torch.empty_like(res), int8=True)
    side.synchronize()
    for a, b in ((y0, y1), (q0, q1), (s0, s1), (r0, r1)):
        assert torch.equal(a, b)
    y, q, scale, out = (torch.empty_like(t) for t in (y0, q0, s0, r0))
    xs = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s12.s12_rmsnorm(xs, w, residual=res, residual_out=out, int8=True, y=y, q=q, scale=scale)
    for seed in (9, 10):
        x2, _, _ = make(33, 4096, False, seed)
        xs.copy_(x2)
        graph.replay()
        y2, q2, s2, r2 = s12.s12_rmsnorm(x2, w, residual=res, residual_out=torch.empty_like(res), int8=True)
        for a, b in ((y, y2), (q, q2), (scale, s2), (out, r2)):
            assert torch.equal(a, b)


def test_binding_refusals(s12):
    x, res, w = make(4, 64, False, 11)
    with pytest.raises(ValueError):
        s12.s12_rmsnorm(x, bf16=False)
    with pytest.raises(ValueError):
        s12.s12_rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        s12.s12_rmsnorm(x, residual=res[:2])
    with pytest.raises(ValueError):
        s12.s12_rmsnorm(x, residual=res, residual_out=torch.empty(4, 64, device="cuda"))
    with pytest.raises(ValueError):
        s12.s12_rmsnorm(x.t())
    with pytest.raises(ValueError):
        s12.s12_rmsnorm(x, y=torch.empty(4, 64, device="cuda"))
    with pytest.raises(TypeError):
        s12.s12_rmsnorm(x.half())
    with pytest.raises(ValueError):
        s12.s12_rmsnorm(x.cpu())
    with pytest.raises(s12.S12Error):
        s12.s12_quant_i8(torch.zeros(4, 12, device="cuda"))
    with pytest.raises(s12.S12Error):
        s12.s12_rmsnorm(x, eps=float("nan"))
