"""Each call as the first that a host thread makes: a thread of its own has no CUDA context until something gives it
one."""
import ctypes as C
import threading

import pytest
import torch

from test_gpu_moe import Layer, s12  # noqa: F401  (s12 is a fixture)

pytestmark = pytest.mark.gpu


def calls(s12):  # noqa: F811
    """name: (call, outputs, what has to stay alive); raw calls, so that nothing but the call itself touches CUDA."""
    L = Layer(s12, 4, 256, 128, 47)
    lib, stream = s12.lib(), torch.cuda.current_stream().cuda_stream
    view = s12.s12_open(s12.s12_encode(torch.randn(256, 256, device="cuda").to(torch.bfloat16)))
    x = L.tokens(32, 1)
    x8, scale = s12.s12_quant_i8(x)
    y, y16 = torch.zeros(32, 256, device="cuda"), torch.zeros(256, 256, dtype=torch.int16, device="cuda")
    ids, weights = torch.zeros(32, 2, dtype=torch.int32, device="cuda"), torch.ones(32, 2, device="cuda")
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    p = {n: t.data_ptr() for n, t in (("x", x), ("x8", x8), ("s", scale), ("y", y), ("y16", y16), ("i", ids),
                                      ("w", weights), ("ws", ws))}
    n, v, up, down = ws.numel(), C.byref(view), C.byref(L.views[0]), C.byref(L.views[1])
    made = {
        "gemv": lambda: lib.s12_gemv(v, p["x"], 3, p["y"], p["ws"], n, None, stream),
        "gemv without workspace": lambda: lib.s12_gemv_noalloc(v, p["x"], 3, p["y"], None, stream),
        "skinny": lambda: lib.s12_gemm_skinny(v, p["x"], 32, p["y"], p["ws"], n, None, stream),
        "decode": lambda: lib.s12_decode(v, p["y16"], None, stream),
        "norm": lambda: lib.s12_rmsnorm(p["x"], 0, None, None, 0, None, 32, 256, 1e-6, p["y16"], None, None, stream),
        "quant": lambda: lib.s12_quant_i8(p["x"], 0, 32, 256, p["y16"], p["y"], stream),
        "product": lambda: lib.s12_gemm_i8(p["x8"], p["s"], p["x8"], p["s"], 32, 32, 256, p["y"], 1, p["ws"], n, None,
                                           stream),
        "few": lambda: lib.s12_gemm_i8(p["x8"], p["s"], p["x8"], p["s"], 1, 32, 256, p["y"], 1, p["ws"], n, None, stream),
        "experts": lambda: lib.s12_moe_routed(up, down, 4, p["x"], 32, p["i"], p["w"], 2, p["y"], 1, p["ws"], n, None,
                                              stream)}
    return made, (y, y16), (L, view, x, x8, scale, ids, weights, ws)


NAMES = ["gemv", "gemv without workspace", "skinny", "decode", "norm", "quant", "product", "few", "experts"]


@pytest.mark.parametrize("name", NAMES)
def test_first_call_of_a_thread(s12, name):  # noqa: F811
    made, outs, alive = calls(s12)
    assert list(made) == NAMES
    call = made[name]
    assert call() == s12.S12_OK
    torch.cuda.synchronize()
    alone = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    codes = []
    thread = threading.Thread(target=lambda: codes.append(call()))
    thread.start()
    thread.join()
    assert codes == [s12.S12_OK]
    torch.cuda.synchronize()
    for got, want in zip(outs, alone):
        assert torch.equal(got, want)
    del alive
