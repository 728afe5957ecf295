"""The new calls as a decoder uses them: the norm in front of a mixture-of-
experts block, the block, the norm after it with the residual's addition and
an 8-bit output, and an 8-bit projection of that.  The steps share one
workspace and run on a side stream, eagerly and as a replayed graph; each is
checked in 64 bits on the input that it actually received."""
import numpy as np
import pytest
import torch

from gpu_util import new_flag
from test_gpu_gemm_i8 import check as check_product
from test_gpu_moe import Layer, check as check_moe, choose, reference
from test_gpu_norm import check_q, check_y, exact

pytestmark = pytest.mark.gpu

E, K, H, F, N = 8, 2, 512, 384, 1000


@pytest.fixture(scope="module")
def s12(cuda_ok):
    from decode_split12_b200 import s12 as mod
    mod.device_check()
    return mod


@pytest.mark.parametrize("T", [1, 7, 33])
def test_norm_experts_norm_and_projection(s12, T):
    L = Layer(s12, E, H, F, 5)
    g = torch.Generator(device="cuda").manual_seed(T)
    stream0 = torch.randn(T, H, generator=g, device="cuda")  # the residual stream, FP32
    w1 = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    w2 = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    proj = torch.randn(N, H, generator=g, device="cuda").to(torch.bfloat16)
    pq, ps = s12.s12_quant_i8(proj)
    check_q(pq, ps, proj.double())
    ws = s12._workspace(max(s12.s12_moe_ws_bytes(*L.views, E, T, K), s12.s12_gemm_i8_ws_bytes(T)), "cuda")
    flag = new_flag()
    res = stream0.clone()
    a = torch.empty(T, H, dtype=torch.int16, device="cuda")
    y = torch.empty(T, H, dtype=torch.int16, device="cuda")
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    wt = torch.empty(T, K, device="cuda")
    q = torch.empty(T, H, dtype=torch.int8, device="cuda")
    scale = torch.empty(T, device="cuda")
    out = torch.empty(T, N, device="cuda")

    def step():
        s12.s12_rmsnorm(res, w1, 1e-6, y=a)
        s12.s12_moe(*L.views, E, a, L.router, K, y=y, ids=ids, weights=wt, ws=ws, err_flag=flag)
        # the block's output joins the residual stream, in place
        s12.s12_rmsnorm(y.view(torch.bfloat16).float(), w2, 1e-6, residual=res, bf16=False, int8=True, q=q, scale=scale)
        s12.s12_gemm_i8(q, scale, pq, ps, y=out, ws=ws, err_flag=flag)

    def verify(before):
        torch.cuda.synchronize()
        _, v = exact(before, None, w1, 1e-6)
        check_y(a, v)
        ab = a.view(torch.bfloat16)
        want, weights = choose(L, ab, K, True)
        assert np.array_equal(ids.cpu().numpy(), want)
        check_moe(y, *reference(L, ab, want, weights))
        s, v = exact(y.view(torch.bfloat16), before, w2, 1e-6)
        assert bool(((res.double() - s).abs() <= s.abs() * 2.0 ** -24).all())
        check_q(q, scale, v)
        check_product(out, q, scale, pq, ps, False)
        assert int(flag.item()) == 0

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    verify(stream0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(2):
        before = res.clone()
        graph.replay()
        verify(before)
