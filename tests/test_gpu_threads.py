"""Calls from two host threads at once, each with sizes of its own (and so with other amounts of shared memory), on a
stream and a workspace of its own: every call succeeds and gives what it gives alone."""
import ctypes as C
import threading

import pytest
import torch

from gpu_util import new_flag
from test_gpu_moe import Layer, s12  # noqa: F401  (s12 is a fixture)

pytestmark = pytest.mark.gpu


def together(s12, jobs, calls):  # noqa: F811
    """jobs: (call(flag, stream), output) of each thread."""
    alone, flags = [], [new_flag() for _ in jobs]
    for (call, out), flag in zip(jobs, flags):
        assert call(flag.data_ptr(), torch.cuda.current_stream().cuda_stream) == s12.S12_OK
        torch.cuda.synchronize()
        alone.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams, codes = [torch.cuda.Stream() for _ in jobs], [set() for _ in jobs]
    start = threading.Barrier(len(jobs))

    def work(i):
        call, handle, flag = jobs[i][0], streams[i].cuda_stream, flags[i].data_ptr()
        start.wait()
        for n in range(calls):
            codes[i].add(call(flag, handle))
            if n % 50 == 49:
                with torch.cuda.stream(streams[i]):
                    if codes[i] != {s12.S12_OK} or int(flags[i].item()):
                        break

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{s12.S12_OK}] * len(jobs)
    assert all(int(flag.item()) == 0 for flag in flags)
    for (_, out), want in zip(jobs, alone):
        assert torch.equal(out, want)


def test_product(s12):  # noqa: F811
    jobs = []
    for M in (16, 112):
        x = torch.randint(-128, 128, (M, 256), dtype=torch.int8, device="cuda")
        w = torch.randint(-128, 128, (512, 256), dtype=torch.int8, device="cuda")
        sx, sw = torch.rand(M, device="cuda"), torch.rand(512, device="cuda")
        y, ws = torch.empty(M, 512, device="cuda"), s12.gemm_i8_workspace(M)
        # (the tensors stay alive in the closure)
        jobs.append((lambda flag, st, t=(x, sx, w, sw, y, ws), M=M: s12.lib().s12_gemm_i8(
            t[0].data_ptr(), t[1].data_ptr(), t[2].data_ptr(), t[3].data_ptr(), M, 512, 256, t[4].data_ptr(), 1,
            t[5].data_ptr(), t[5].numel(), flag, st), y))
    together(s12, jobs, 3000)


def test_experts(s12):  # noqa: F811
    L = Layer(s12, 4, 256, 128, 43)
    jobs = []
    for T, routed in ((1, True), (40, True)):  # x in shared memory, and not
        x = L.tokens(T, T)
        ids = torch.randint(0, 4, (T, 2), dtype=torch.int32, device="cuda")
        weights = torch.rand(T, 2, device="cuda")
        y, ws = torch.empty(T, 256, device="cuda"), s12.moe_workspace(*L.views, 4, T, 2)
        jobs.append((lambda flag, st, t=(x, ids, weights, y, ws), T=T: s12.lib().s12_moe_routed(
            C.byref(L.views[0]), C.byref(L.views[1]), 4, t[0].data_ptr(), T, t[1].data_ptr(), t[2].data_ptr(), 2,
            t[3].data_ptr(), 1, t[4].data_ptr(), t[4].numel(), flag, st), y))
    together(s12, jobs, 500)


def test_fused_product(s12):  # noqa: F811
    w = torch.randn(256, 256, device="cuda").to(torch.bfloat16)
    view = s12.s12_open(s12.s12_encode(w))
    jobs = []
    for M in (16, 208):
        x = torch.randn(M, 256, device="cuda").to(torch.bfloat16)
        y = torch.empty(M, 256, device="cuda")
        ws = torch.zeros(max(s12.s12_gemm_ws_bytes(view, M), 256), dtype=torch.uint8, device="cuda")
        jobs.append((lambda flag, st, t=(x, y, ws), M=M: s12.lib().s12_gemm_skinny(
            C.byref(view), t[0].data_ptr(), M, t[1].data_ptr(), t[2].data_ptr(), t[2].numel(), flag, st), y))
    together(s12, jobs, 3000)
