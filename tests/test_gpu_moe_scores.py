"""The routing of s12_moe against scores in 64 bits: orders that hang on terms which 32 bits lose, scores whose
products leave FP32's range, and scores that are NaN.  Tolerances of y: test_gpu_moe.py."""
import numpy as np
import pytest
import torch

from gpu_util import new_flag
from test_gpu_moe import Layer, check, choose, reference, s12  # noqa: F401  (s12 is a fixture)

pytestmark = pytest.mark.gpu

# T, E, k, H, F: every CTA for itself; by the grid, a token and expert at a time and in blocks of them; the kernel
# for many pairs, both ways
FORMS = {"own": (2, 6, 2, 256, 128), "grid": (5, 20, 3, 4096, 128), "blocks": (37, 40, 8, 384, 128),
         "many": (64, 9, 8, 512, 2944), "many blocks": (64, 24, 8, 512, 2944)}


def layer(s12, form):  # noqa: F811
    T, E, k, H, F = FORMS[form]
    assert form.startswith("many") == (T * k * 3 * H * F > 2 ** 31)
    return Layer(s12, E, H, F, 41), T, k


def routed_right(s12, L, x, k, renorm=True):  # noqa: F811
    flag = new_flag()
    y, ids, w = s12.s12_moe(*L.views, L.E, x, L.router, k, renorm=renorm, err_flag=flag)
    want, weights = choose(L, x, k, renorm)
    assert np.array_equal(ids.cpu().numpy(), want)
    # (a weight: expf within 2 steps of its argument rounded to FP32, at most 8 terms or E, one division)
    assert np.abs(w.cpu().numpy() - weights).max() <= 2.0 ** -20
    check(y, *reference(L, x, want, weights))
    assert int(flag.item()) == 0


@pytest.mark.parametrize("form", FORMS)
def test_order_that_32_bits_lose(s12, form):  # noqa: F811
    """Rows whose sums differ by less than FP32 can tell, the larger one later: in neighbouring columns, across a
    cancellation, and far apart.  Each sum is exact in 64 bits: its terms span less than 2^40."""
    L, T, k = layer(s12, form)
    E, H = L.E, L.H
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    x *= (2.0 ** (torch.arange(T, device="cuda") % 3 - 1))[:, None].to(torch.bfloat16)  # 1/2, 1, 2
    for lay in range(4):
        r = torch.zeros(E, H, dtype=torch.float64)
        for e in range(E):
            c = 8 * ((5 * e) % (H // 8))
            if lay == 0:  # 1 + a little in columns beside it
                r[e, c] = 1.0
                r[e, c + 1:c + 1 + e % 7] = 2.0 ** -24
            elif lay == 1:  # what two large terms leave
                r[e, c], r[e, c + 2] = 4096.0, -4096.0
                r[e, c + 1] = (e % 5) * 2.0 ** -13
            elif lay == 2:  # the same with the large terms far apart
                r[e, 0], r[e, H - 1] = 4096.0, -4096.0
                r[e, H // 2] = (e % 5) * 2.0 ** -13
            else:  # all columns, signs that cancel but for a little
                r[e] = torch.where(torch.arange(H) % 2 == 0, 3.0, -3.0)
                r[e, c + 3] -= (e % 6) * 2.0 ** -6
        L.router = r.to(torch.bfloat16).cuda()
        assert torch.equal(L.router.double().cpu(), r)
        routed_right(s12, L, x, k)


@pytest.mark.parametrize("form", FORMS)
def test_order_of_random_scores_near_one_another(s12, form):  # noqa: F811
    """Experts that are one row in other orders of its values: their scores with a token of ones are equal, so the
    lower index comes first, whatever order the sum is taken in.  (Values of 8 bits
    between 2^-14 and 2^13: every partial sum is a multiple of 2^-21 below 2^25.)"""
    L, T, k = layer(s12, form)
    g = torch.Generator().manual_seed(5)
    row = (torch.randn(L.H, generator=g) * 2.0 ** torch.randint(-10, 11, (L.H,), generator=g)).to(torch.bfloat16)
    row = torch.where(row.abs() < 2.0 ** -14, torch.zeros_like(row), row)
    L.router = torch.stack([row[torch.randperm(L.H, generator=g)] for _ in range(L.E)]).cuda()
    x = torch.ones(T, L.H, dtype=torch.bfloat16, device="cuda")
    _, ids, w = s12.s12_moe(*L.views, L.E, x, L.router, k)
    assert torch.equal(ids.cpu(), torch.arange(k, dtype=torch.int32).expand(T, k))
    assert bool(((w - 1 / k).abs() <= 2.0 ** -20).all())


@pytest.mark.parametrize("form", FORMS)
def test_products_outside_the_range_of_32_bits(s12, form):  # noqa: F811
    """Terms that are too large or too small for FP32, subnormal operands among them, and sums that are not."""
    L, T, k = layer(s12, form)
    x = torch.zeros(T, L.H, dtype=torch.float64)
    r = torch.zeros(L.E, L.H, dtype=torch.float64)
    x[:, 0], x[:, 9], x[:, 18] = 2.0 ** 100, 2.0 ** -100, 2.0 ** -130
    for e in range(L.E):
        r[e, 0] = (0, 2.0 ** 100, -2.0 ** 100)[e % 3]  # 2^200 either way
        r[e, 9] = (e // 3 % 4) * 2.0 ** -90            # a few 2^-190
        r[e, 18] = (e // 12 % 2) * 2.0 ** -132         # 2^-262
    L.router = r.to(torch.bfloat16).cuda()
    assert torch.equal(L.router.double().cpu(), r)
    xb = x.to(torch.bfloat16)
    assert torch.equal(xb.double(), x)
    want, weights = choose(L, xb.cuda(), k, True)
    _, ids, w = s12.s12_moe(*L.views, L.E, xb.cuda(), L.router, k)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.abs(w.cpu().numpy() - weights).max() <= 2.0 ** -20


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("form", FORMS)
def test_nan_in_one_router_row_reaches_every_token(s12, form, renorm):  # noqa: F811
    """Every token has one score that is NaN, and top_k or more that are not: weights and y are NaN; the others'
    order is theirs, and the NaN comes behind them."""
    L, T, k = layer(s12, form)
    x = L.tokens(T, 2)
    bad = L.E // 2
    L.router[bad, L.H - 3] = float("nan")
    y, ids, w = s12.s12_moe(*L.views, L.E, x, L.router, k, renorm=renorm)
    assert bool(torch.isnan(w).all()) and bool(torch.isnan(y.view(torch.bfloat16)).all())
    score = torch.nan_to_num(x.double() @ L.router.double().T, nan=-np.inf).cpu().numpy()
    assert np.array_equal(ids.cpu().numpy(), np.stack([np.lexsort((np.arange(L.E), -s))[:k] for s in score]))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("form", FORMS)
def test_infinite_router_value_reaches_the_tokens_it_meets(s12, form, renorm):  # noqa: F811
    """One infinity in a router row: a token with 0 there has a NaN score, one above 0 a score of infinity (both make
    its weights NaN), one below 0 minus infinity, which leaves that expert out and nothing else."""
    L, T, k = layer(s12, form)
    x = L.tokens(T, 3)
    bad, c = L.E - 1, 11
    kind = torch.arange(T, device="cuda") % 3
    x[:, c] = torch.where(kind == 0, -1.0, torch.where(kind == 1, 0.0, 1.0)).to(torch.bfloat16)
    L.router[bad, c] = float("inf")
    y, ids, w = s12.s12_moe(*L.views, L.E, x, L.router, k, renorm=renorm)
    y = y.view(torch.bfloat16)
    assert bool(torch.isnan(w[kind > 0]).all()) and bool(torch.isnan(y[kind > 0]).all())
    fine = kind == 0
    want, weights = choose(L, x[fine], k, renorm)
    assert np.array_equal(ids[fine].cpu().numpy(), want) and not bool((ids[fine] == bad).any())
    assert np.abs(w[fine].cpu().numpy() - weights).max() <= 2.0 ** -20
    check(y[fine].view(torch.int16), *reference(L, x[fine], want, weights))
