"""s12_rmsnorm over all of FP32's range: rows whose squares leave it, with every eps that is allowed, against 64-bit
arithmetic.

Tolerance.  Such a row is scaled by a power of two, which is exact (a value that becomes subnormal is below 2^-100
of the row's largest and v is off by 2^-140 there), then as in test_gpu_norm.py: the sum, its inverse root, and one
product more (with the factor before the weight instead of after it), 2^-24: V_REL covers it.  In rows
of ordinary size (a mean square with eps of 2^-40 or more) a product s * w that is subnormal is off by 2^-150, which
the factor of at most 2^20 makes 2^-130 of v.  Half a step of a subnormal BF16 result is 2^-134: their steps are
2^-133, whatever the value.  So a y may be off by SMALL = 2^-130 + 2^-134 beside its relative error (a scale, whose
steps are 2^-149, by less)."""
import pytest
import torch

from test_gpu_norm import HALF, V_REL, bf16, s12  # noqa: F401  (s12 is a fixture)

pytestmark = pytest.mark.gpu

SIZES = [1e-45, 3e-42, 1e-38, 1e-30, 2.6e-23, 1e-20, 1e-12, 1e-7, 1.0, 1e10, 4e17, 2e19, 1e30, 7e37]
SMALL = 2.0 ** -130 + 2.0 ** -134
EPS = [0.0, 1e-45, 1e-40, 1e-30, 1e-12, 1e-6, 1.0, 1e30, 3e38]


def exact(s, w, eps):
    s = s.double()
    n = s.abs().amax(-1, keepdim=True).clamp(min=1e-300)
    # (1e-45 as the call gets it: in FP32)
    e = torch.tensor(eps, dtype=torch.float32).double().item()
    length = torch.sqrt(((s / n) ** 2).mean(-1, keepdim=True) * n * n + e)
    return torch.where(length > 0, s / length, 0.0) * w.double()


def check(y, q, scale, v):
    err = (bf16(y) - v).abs()
    assert bool((err <= v.abs() * (2.0 ** -8 + V_REL) + SMALL).all()), float((err / v.abs().clamp(min=1e-300)).max())
    top = v.abs().amax(-1)
    assert bool(((scale.double() - top / 127).abs() <= top / 127 * V_REL + SMALL).all())
    # (of a row whose v fit FP32's normal range: the integers are what the definition gives)
    fine = top > 1e-30
    want = v / (top / 127)[..., None].clamp(min=1e-300)
    assert not bool(fine.any()) or float((q.double() - want)[fine].abs().max()) <= HALF
    assert bool((q.abs().amax(-1)[fine] == 127).all())
    assert bool((q[top == 0] == 0).all()) and bool((scale[top == 0] == 0).all())


@pytest.mark.parametrize("cols", [64, 1000, 4104, 14336, 32768])
@pytest.mark.parametrize("copies", [1, 23])
def test_rows_of_every_size(s12, cols, copies):  # noqa: F811
    """A row of each size, few of them and many (more than two an SM), with every eps."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    size = torch.tensor(SIZES, dtype=torch.float64).repeat(copies).cuda()
    x = (torch.randn(len(size), cols, generator=g, device="cuda", dtype=torch.float64).clamp(-4, 4) * size[:, None]).float()
    assert bool(torch.isfinite(x).all())
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)
    for eps in EPS:
        y, q, scale, _ = s12.s12_rmsnorm(x, w, eps=eps, int8=True)
        check(y, q, scale, exact(x, w, eps))


@pytest.mark.parametrize("cols", [256, 4096])
@pytest.mark.parametrize("f32", [True, False])
def test_residual_in_place(s12, cols, f32):  # noqa: F811
    """The sum is taken once: a row that is scaled is not read again from the residual that was overwritten."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    t = torch.float32 if f32 else torch.bfloat16
    size = torch.tensor([1e-30, 1.0, 1e30, 1e-24], device="cuda")[:, None]
    x, res = ((torch.randn(4, cols, generator=g, device="cuda") * size).to(t) for _ in range(2))
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)
    total = x.float() + res.float()  # (one FP32 addition, as the call's)
    for eps in (0.0, 1e-6):
        r = res.clone()
        y, q, scale, out = s12.s12_rmsnorm(x, w, eps=eps, residual=r, int8=True)
        assert out is r and torch.equal(r, total.to(t))
        check(y, q, scale, exact(total, w, eps))


def test_one_loud_value_among_tiny_ones(s12):  # noqa: F811
    """Scaling by the largest leaves the rest at zero relative to it, as they are."""
    x = torch.full((4, 4096), 1e-38, device="cuda")
    x[0, 77], x[1, 4095], x[2, 0] = 1e38, 1e-3, 3e-20
    w = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    for eps in EPS:
        y, q, scale, _ = s12.s12_rmsnorm(x, w, eps=eps, int8=True)
        check(y, q, scale, exact(x, w, eps))


@pytest.mark.parametrize("cols", [128, 8192])
def test_infinities_and_nan_beside_rows_that_are_scaled(s12, cols):  # noqa: F811
    """Not finite: q 0 and scale NaN, whatever the size of the rest; weights that are 0 or infinite, too."""
    x = torch.randn(6, cols, generator=torch.Generator().manual_seed(1))
    x[0] *= 1e-30
    x[0, 5] = float("inf")
    x[1] *= 1e30
    x[1, cols - 1] = float("nan")
    x[2] *= 1e30
    x[3] *= 1e-30
    x[4] = 0
    x = x.cuda()
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    for eps in (0.0, 1e-6):
        y, q, scale, _ = s12.s12_rmsnorm(x, w, eps=eps, int8=True)
        assert bool((q[:2] == 0).all()) and bool(torch.isnan(scale[:2]).all())
        assert bool(torch.isnan(bf16(y)[1]).all()) and bool(torch.isnan(bf16(y)[0, 5]))
        check(y[2:], q[2:], scale[2:], exact(x[2:], w, eps))
        w0 = torch.zeros_like(w)
        y, q, scale, _ = s12.s12_rmsnorm(x[2:], w0, eps=eps, int8=True)
        assert bool((bf16(y) == 0).all()) and bool((q == 0).all()) and bool((scale == 0).all())
        w0[3] = float("inf")
        y, q, scale, _ = s12.s12_rmsnorm(x[2:4], w0, eps=eps, int8=True)
        assert bool((q == 0).all()) and bool(torch.isnan(scale).all())
