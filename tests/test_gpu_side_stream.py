"""A call with a stream runs there alone: what it allocates (outputs, workspaces with their zero bytes) belongs to
that stream, so that work still waiting on the current stream does not disturb it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def s12(cuda_ok):
    from decode_split12_b200 import s12 as mod
    mod.device_check()
    return mod


def calls(s12):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(9, 512, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randint(-128, 128, (300, 512), generator=g, dtype=torch.int8, device="cuda")
    one = torch.ones(300, device="cuda")
    E, H, F = 8, 512, 256
    up = torch.randn(E * 2 * F, H, generator=g, device="cuda").div(22).to(torch.bfloat16)
    down = torch.randn(E * H, F, generator=g, device="cuda").div(16).to(torch.bfloat16)
    views = [s12.s12_open(s12.s12_encode(w)) for w in (up, down)]
    router = torch.randn(E, H, generator=g, device="cuda").div(22).to(torch.bfloat16)
    ids = torch.randint(0, E, (9, 2), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.rand(9, 2, generator=g, device="cuda")
    return {
        "norm": lambda **k: s12.s12_rmsnorm(x, int8=True, **k)[:3],
        "quant": lambda **k: s12.s12_quant_i8(x, **k),
        "product": lambda **k: (s12.s12_gemm_i8(q, one, q, one, f32=True, **k),),
        "few": lambda **k: (s12.s12_gemm_i8(q[:3], one[:3], q, one, f32=True, **k),),
        "experts": lambda **k: s12.s12_moe(*views, E, x, router, 2, **k),
        "routed": lambda **k: (s12.s12_moe_routed(*views, E, x, ids, weights, f32=True, **k),),
    }


@pytest.mark.parametrize("name", ["norm", "quant", "product", "few", "experts", "routed"])
def test_call_on_a_stream_of_its_own(s12, name):
    call = calls(s12)[name]
    ref = [t.cpu() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(stream=side)  # (its memory is there from here on)
    torch.cuda.synchronize()
    # memory that the allocator hands out again is not zero
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            rubbish = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (4096, 1 << 20, 1 << 23)]
            del rubbish
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s on the current stream
    out = call(stream=side)
    with torch.cuda.stream(side):
        host = [t.cpu() for t in out]
    # (the expert layers are cooperative launches, which may wait for the device to be free of other kernels)
    assert name in ("experts", "routed") or not torch.cuda.current_stream().query()
    assert all(torch.equal(a, b) for a, b in zip(ref, host))
    torch.cuda.synchronize()
