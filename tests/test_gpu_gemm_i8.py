"""s12_gemm_i8 on the GPU.  The integer sums are exact, so y differs from the
64-bit product by the conversion of the sum to FP32, two multiplications
(2^-24 each) and, for BF16, half a step (2^-8)."""
import pytest
import torch

from gpu_util import new_flag

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def s12(cuda_ok):
    from decode_split12_b200 import s12 as mod
    mod.device_check()
    return mod


def make(M, N, K, seed, low=-128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(low, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(low, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(M, generator=g, device="cuda") + 0.01
    sw = torch.rand(N, generator=g, device="cuda") * 1e-3 + 1e-6
    return x, sx, w, sw


def check(y, x, sx, w, sw, bf16):
    ref = (x.double() @ w.double().T) * sx.double()[:, None] * sw.double()
    got = y.view(torch.bfloat16).double() if bf16 else y.double()
    rel = 3 * 2.0 ** -24 * (1 + 2.0 ** -20) + (2.0 ** -8 if bf16 else 0)
    assert bool(((got - ref).abs() <= ref.abs() * rel).all()), float(((got - ref).abs() / ref.abs().clamp(min=1e-30)).max())


SHAPES = [(1, 1, 16), (1, 128, 128), (2, 129, 144), (3, 7, 32), (16, 256, 1024), (17, 127, 4096), (1, 4096, 14336),
          (19, 5000, 2064), (33, 4097, 256), (64, 1000, 8192), (100, 384, 48), (128, 640, 640), (240, 129, 528),
          (256, 2048, 1024), (257, 2049, 1040), (300, 19000, 272), (513, 260, 2048), (1000, 3000, 400),
          (4096, 16, 512), (2049, 4200, 1056)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(s12, M, N, K):
    x, sx, w, sw = make(M, N, K, M + N + K)
    ws, flag = s12.gemm_i8_workspace(M), new_flag()
    y = s12.s12_gemm_i8(x, sx, w, sw, ws=ws, err_flag=flag)
    check(y, x, sx, w, sw, True)
    y32 = torch.full((M, N), float("nan"), device="cuda")
    s12.s12_gemm_i8(x, sx, w, sw, y=y32, ws=ws, err_flag=flag)
    check(y32, x, sx, w, sw, False)
    assert torch.equal(y32.to(torch.bfloat16), y.view(torch.bfloat16))
    assert int(flag.item()) == 0
    # the counters are zero again
    assert int(ws[:s12.S12_WS_HEAD].to(torch.int32).sum()) == 0


@pytest.mark.parametrize("K", [131056, 65536])
def test_largest_sums(s12, K):
    """All -128: the largest sum of all, exactly."""
    x = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((130, K), -128, dtype=torch.int8, device="cuda")
    one, ones = torch.ones(2, device="cuda"), torch.ones(130, device="cuda")
    y = s12.s12_gemm_i8(x, one, w, ones, f32=True)
    assert bool((y.double() == float(torch.tensor(K * 16384, dtype=torch.float32))).all())


def test_every_pair_of_values(s12):
    """256 x 256 products with K = 16 and one column that is not zero: each pair of int8 values, signs included."""
    v = torch.arange(-128, 128, dtype=torch.int8, device="cuda")
    x = torch.zeros(256, 16, dtype=torch.int8, device="cuda")
    w = torch.zeros(256, 16, dtype=torch.int8, device="cuda")
    x[:, 5], w[:, 5] = v, v
    one = torch.ones(256, device="cuda")
    y = s12.s12_gemm_i8(x, one, w, one, f32=True)
    assert torch.equal(y, torch.outer(v.float(), v.float()))


def test_one_workspace_for_calls_of_any_shape(s12):
    ws = s12.gemm_i8_workspace(256)
    cases = [make(M, N, K, M) for M, N, K in ((1, 4096, 4096), (256, 1000, 2048), (33, 129, 8192), (700, 300, 1024),
                                              (5, 20000, 64), (1, 128, 131056))]
    for _ in range(2):
        for c in cases:
            check(s12.s12_gemm_i8(*c, ws=ws), *c, True)


def test_nan_scales_stay_in_their_rows_and_columns(s12):
    x, sx, w, sw = make(5, 200, 64, 1)
    x[2] = 0
    sx[2] = float("nan")
    sw[7] = float("nan")
    y = s12.s12_gemm_i8(x, sx, w, sw, f32=True)
    bad = torch.isnan(y)
    assert bool(bad[2].all()) and bool(bad[:, 7].all()) and int(bad.sum()) == 200 + 5 - 1


def test_no_rows_or_columns(s12):
    x, sx, w, sw = make(3, 40, 64, 1)
    assert s12.s12_gemm_i8(x[:0], sx[:0], w, sw).shape == (0, 40)
    assert s12.s12_gemm_i8(x, sx, w[:0], sw[:0]).shape == (3, 0)


def test_other_streams_and_replayed_graphs(s12):
    c = make(70, 3000, 1024, 3)
    ref = s12.s12_gemm_i8(*c)
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream() for _ in range(2)], []
    spaces = [s12.gemm_i8_workspace(70) for _ in streams]
    torch.cuda.synchronize()
    for st, ws in zip(streams, spaces):
        with torch.cuda.stream(st):
            out += [s12.s12_gemm_i8(*c, ws=ws) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(ref, y) for y in out)
    ws = s12.gemm_i8_workspace(70)
    xs, graphs, ys = c[0].clone(), [], []
    for M in (70, 9):
        y = torch.empty(M, 3000, dtype=torch.int16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s12.s12_gemm_i8(xs[:M], c[1][:M], c[2], c[3], y=y, ws=ws)
        graphs.append(graph)
        ys.append(y)
    for seed in (5, 6):
        xs.copy_(make(70, 3000, 1024, seed)[0])
        for graph, y in zip(graphs, ys):
            graph.replay()
            assert torch.equal(y, s12.s12_gemm_i8(xs[:y.shape[0]], c[1][:y.shape[0]], c[2], c[3]))


def test_more_than_2_31_outputs(s12):
    """Offsets of y past 32 bits: the last rows are those of the same rows alone."""
    x, sx, w, sw = make(70000, 32000, 32, 9)
    y = s12.s12_gemm_i8(x, sx, w, sw)
    for rows in (slice(0, 40), slice(35000, 35040), slice(69960, 70000)):
        check(y[rows], x[rows], sx[rows], w, sw, True)


def test_binding_refusals(s12):
    x, sx, w, sw = make(4, 40, 64, 1)
    with pytest.raises(ValueError):
        s12.s12_gemm_i8(x, sx[:3], w, sw)
    with pytest.raises(ValueError):
        s12.s12_gemm_i8(x, sx, w[:, :48], sw)
    with pytest.raises(ValueError):
        s12.s12_gemm_i8(x.short(), sx, w, sw)
    with pytest.raises(ValueError):
        s12.s12_gemm_i8(x, sx.double(), w, sw)
    with pytest.raises(ValueError):
        s12.s12_gemm_i8(x, sx, w.cpu(), sw)
    with pytest.raises(ValueError):
        s12.s12_gemm_i8(x[:, :32], sx, w[:, :32].contiguous(), sw)
    with pytest.raises(s12.S12Error):
        s12.s12_gemm_i8(x[:, :40].contiguous(), sx, w[:, :40].contiguous(), sw)
    with pytest.raises(s12.S12Error):
        s12.s12_gemm_i8(x, sx, w, sw, ws=torch.zeros(1024, dtype=torch.uint8, device="cuda"))
