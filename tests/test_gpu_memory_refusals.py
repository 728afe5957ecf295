"""Refusals of memory that a kernel would leave: an error word of fewer than four bytes, and a container that is not
on the current device (here on the host: its view's addresses are not looked at)."""
import pytest
import torch

from gpu_util import new_flag
from test_gpu_moe import Layer, s12  # noqa: F401  (s12 is a fixture)

pytestmark = pytest.mark.gpu
SMALL = [torch.zeros(1, dtype=torch.int8), torch.zeros(3, dtype=torch.uint8), torch.zeros(1, dtype=torch.bfloat16),
         torch.zeros(0, dtype=torch.int32)]


def test_error_words(s12):  # noqa: F811
    L = Layer(s12, 4, 256, 128, 53)
    x, ids, w = L.tokens(3, 1), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, 2, device="cuda")
    q, scale = s12.s12_quant_i8(x)
    calls = [lambda f: s12.s12_moe(*L.views, 4, x, L.router, 2, err_flag=f),
             lambda f: s12.s12_moe_routed(*L.views, 4, x, ids, w, err_flag=f),
             lambda f: s12.s12_gemm_i8(q, scale, q, scale, err_flag=f)]
    for call in calls:
        for small in SMALL:
            with pytest.raises(ValueError, match="err_flag"):
                call(small.cuda())
        with pytest.raises(ValueError):
            call(torch.zeros(1, dtype=torch.int32))  # on the host
        # four bytes or more, of any type
        for flag in (new_flag(), torch.zeros(4, dtype=torch.uint8, device="cuda"),
                     torch.zeros(2, dtype=torch.int64, device="cuda")):
            call(flag)
            assert int(flag.sum().item()) == 0


def test_containers_elsewhere(s12):  # noqa: F811
    L = Layer(s12, 4, 256, 128, 59)
    x, ids, w = L.tokens(3, 1), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, 2, device="cuda")
    for at in (0, 1):
        views = [s12.s12_open(b) for b in L.blobs]
        views[at]._blob = L.blobs[at].cpu()
        with pytest.raises(ValueError, match="current device"):
            s12.s12_moe(*views, 4, x, L.router, 2)
        with pytest.raises(ValueError, match="current device"):
            s12.s12_moe_routed(*views, 4, x, ids, w)
    # a view that does not know its container is taken as it is
    views = []
    for v in L.views:
        copy = s12.View.from_buffer_copy(v)
        assert not hasattr(copy, "_blob")
        views.append(copy)
    want = s12.s12_moe_routed(*L.views, 4, x, ids, w)
    assert torch.equal(s12.s12_moe_routed(*views, 4, x, ids, w), want)
