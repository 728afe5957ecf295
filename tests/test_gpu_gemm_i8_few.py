"""s12_gemm_i8 with a few tokens (dot products) and at the edges of that form, against exact integers in 64 bits.

Sums are exact; the product of the rounded sum and two scales has three roundings of 2^-24, and a BF16 y one of 2^-8."""
import pytest
import torch

from gpu_util import new_flag

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def s12(cuda_ok):
    from decode_split12_b200 import s12 as mod
    mod.device_check()
    return mod


def make(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8, device="cuda")
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8, device="cuda")
    sx, sw = (torch.rand(n, generator=g, device="cuda") + 0.01 for n in (M, N))
    return x, sx, w, sw


def check(y, x, sx, w, sw, f32):
    ref = (x.double() @ w.double().T) * sx.double()[:, None] * sw.double()
    got = y.double() if f32 else y.view(torch.bfloat16).double()
    bound = (4 * 2.0 ** -24 + (0 if f32 else 2.0 ** -8 * (1 + 2.0 ** -20))) * ref.abs()
    assert bool(((got - ref).abs() <= bound).all())


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 16), (3, 32), (5, 496), (129, 512), (1000, 4112), (33, 16400), (4099, 2064),
                                 (7, 131056), (4736, 7184), (9473, 1024)])
def test_shapes(s12, M, N, K):
    c = make(M, N, K, M * 7 + N)
    ws, flag = s12.gemm_i8_workspace(M), new_flag()
    check(s12.s12_gemm_i8(*c, ws=ws, err_flag=flag), *c, False)
    check(s12.s12_gemm_i8(*c, ws=ws, err_flag=flag, f32=True), *c, True)
    assert int(flag.item()) == 0 and int(ws[:s12.S12_WS_HEAD].to(torch.int32).sum()) == 0


@pytest.mark.parametrize("M", [1, 4, 8])
def test_a_token_alone_and_among_many(s12, M):
    """The same values whether a token comes alone, with a few (dot products) or with many (tensor cores)."""
    x, sx, w, sw = make(40, 1003, 2064, 5)
    many = s12.s12_gemm_i8(x, sx, w, sw, f32=True)
    few = s12.s12_gemm_i8(x[:M], sx[:M], w, sw, f32=True)
    assert torch.equal(few, many[:M])


@pytest.mark.parametrize("value", [-128, 127])
def test_largest_sums(s12, value):
    K = 131056
    x = torch.full((5, K), value, dtype=torch.int8, device="cuda")
    w = torch.full((6, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(6, device="cuda")
    y = s12.s12_gemm_i8(x, one[:5], w, one, f32=True)
    assert bool((y == torch.tensor(float(-128 * value * K), device="cuda")).all())


def test_rows_past_the_last_are_left(s12):
    """y inside a larger buffer: nothing before or after it changes."""
    x, sx, w, sw = make(3, 41, 528, 2)
    room = torch.full((3 * 41 + 64,), 7.0, device="cuda")
    y = room[32:32 + 3 * 41].view(3, 41)
    s12.s12_gemm_i8(x, sx, w, sw, y=y, f32=True)
    check(y, x, sx, w, sw, True)
    assert bool((room[:32] == 7).all()) and bool((room[32 + 3 * 41:] == 7).all())


def test_more_than_2_31_weights(s12):
    """Offsets of w past 32 bits."""
    N, K = 20000, 131056
    x = torch.randint(-128, 128, (1, K), dtype=torch.int8, device="cuda")
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda")
    one = torch.ones(N, device="cuda")
    y = s12.s12_gemm_i8(x, one[:1], w, one, f32=True)
    rows = torch.tensor([0, 1, 16383, 16384, 19998, 19999], device="cuda")
    ref = x.double() @ w[rows].double().T
    assert torch.equal(y[:, rows], ref.float())


def test_chain_of_quantiser_and_products_in_a_graph(s12):
    """Quantiser, product, quantiser, product for one token, eagerly and replayed with new inputs."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, 1024, generator=g, device="cuda").to(torch.bfloat16)
    ws = s12.gemm_i8_workspace(1)
    w1, s1 = s12.s12_quant_i8(torch.randn(2048, 1024, generator=g, device="cuda").to(torch.bfloat16))
    w2, s2 = s12.s12_quant_i8(torch.randn(1024, 2048, generator=g, device="cuda").to(torch.bfloat16))

    def run():
        q, s = s12.s12_quant_i8(x)
        h = s12.s12_gemm_i8(q, s, w1, s1, ws=ws)
        q, s = s12.s12_quant_i8(h.view(torch.bfloat16))
        return s12.s12_gemm_i8(q, s, w2, s2, ws=ws)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in range(3):
        x.copy_(torch.randn(1, 1024, generator=g, device="cuda"))
        graph.replay()
        assert torch.equal(out, run())
