"""Every BF16 pattern through the expert layer, bit for bit: each output reads one weight.

gate is 128 where the token's column is, so silu(gate x) = 128 exactly (exp(-128) is below half a step of 1), and
h = 128 u for a weight u of up, which two BF16 values hold exactly (128 u has u's 8 bits and is not subnormal).  With
ones on down's diagonal y is 128 u.  The other way round up is 1 on its diagonal, h is 128 in one place, and y is
128 d for a weight d of down.  All other terms are products with 0.  Patterns are those below 2^121 (128 u is
finite), zeros and subnormals among them, in an order that makes most of them escapes."""
import pytest
import torch

from gpu_util import blob_to_dev, blob_to_host, new_flag
from test_gpu_moe import s12  # noqa: F401  (s12 is a fixture)

pytestmark = pytest.mark.gpu


def patterns(n):
    """n BF16 values that take every pattern below 2^121 in turn."""
    p = torch.arange(65536, dtype=torch.int64)
    p = p[((p >> 7) & 0xFF) < 248]
    p = p[torch.randperm(len(p), generator=torch.Generator().manual_seed(6))]
    p = p.repeat(-(-n // len(p)))[:n]
    return torch.where(p > 32767, p - 65536, p).to(torch.int16).view(torch.bfloat16)


def containers(s12, gate, up, down, version):  # noqa: F811
    E, F, H = up.shape
    both = s12.interleave_gate_up(gate.reshape(E * F, H).cuda(), up.reshape(E * F, H).cuda())
    blobs = [s12.s12_encode(both.contiguous()), s12.s12_encode(down.reshape(E * H, F).cuda().contiguous())]
    if version == 2:
        blobs = [blob_to_dev(s12.to_v2_host(blob_to_host(b))) for b in blobs]
    return [s12.s12_open(b) for b in blobs]


@pytest.mark.parametrize("version", [1, 2])
@pytest.mark.parametrize("side", ["up", "down"])
@pytest.mark.parametrize("E,n,k", [(4, 128, 1), (2, 1280, 8)])  # the kernels for few pairs and for many
def test_every_weight_is_read_exactly(s12, E, n, k, side, version):  # noqa: F811
    T = 64
    assert (T * k * 3 * n * n > 2 ** 31) == (k == 8)
    eye = torch.eye(n).to(torch.bfloat16).expand(E, n, n)
    gate = torch.full((E, n, n), 128.0, dtype=torch.bfloat16)
    weights = patterns(E * n * n).view(E, n, n)
    if side == "up":
        views = containers(s12, gate, weights, eye, version)
    else:
        views = containers(s12, gate, eye, weights, version)
    assert int(views[side == "down"].n_esc) > E * n * n // 4
    flag = new_flag()
    ws = s12.moe_workspace(*views, E, T, k)
    share = torch.zeros(T, k, device="cuda")
    share[:, 0] = 1  # (the other slots' experts are multiplied by 0)
    for c0 in list(range(0, n, T)):
        x = torch.eye(n)[c0:c0 + T].to(torch.bfloat16).cuda()
        for e in range(E):
            ids = ((torch.arange(k) + e) % E).to(torch.int32).expand(T, k).contiguous().cuda()
            y = s12.s12_moe_routed(*views, E, x, ids, share, ws=ws, err_flag=flag, f32=True)
            want = 128 * weights[e].float()[:, c0:c0 + T].T  # of a column: up's by hidden value, down's by output
            assert torch.equal(y.cpu(), want), int((y.cpu() != want).sum())
    assert int(flag.item()) == 0
