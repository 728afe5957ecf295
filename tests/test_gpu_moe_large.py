"""s12_moe and s12_moe_routed with many pairs an expert (products above 2^31 multiply-adds, which take the kernel
that decodes into the tensor cores' memory), against the layer in 64 bits.  Tolerances: test_gpu_moe.py."""
import numpy as np
import pytest
import torch

from gpu_util import blob_to_dev, blob_to_host, new_flag
from test_gpu_moe import Layer, check, choose, reference, s12  # noqa: F401  (s12 is a fixture)

pytestmark = pytest.mark.gpu


def many(T, k, H, F):
    return T * k * 3 * H * F > 2 ** 31


@pytest.mark.parametrize("T,E,k,H,F", [
    (64, 8, 8, 2176, 768),    # 17 tiles a row: ranges of one tile after ranges of 16; 6 tiles
    (64, 9, 8, 128, 11008),   # gate and up of a single tile a row
    (64, 8, 8, 11008, 128),   # down of a single tile a row
    (57, 10, 7, 640, 2816),   # 5 and 22 tiles
    (40, 64, 8, 2432, 1024),  # five pairs an expert
    (64, 200, 8, 1408, 1024),  # experts without a pair
    (9, 4, 2, 4224, 9472)])   # few tokens of large experts
def test_shapes(s12, T, E, k, H, F):  # noqa: F811
    assert many(T, k, H, F)
    L = Layer(s12, E, H, F, T + E)
    x, flag = L.tokens(T, E), new_flag()
    ws = s12.moe_workspace(*L.views, E, T, k)
    y, ids, w = s12.s12_moe(*L.views, E, x, L.router, k, ws=ws, err_flag=flag)
    want, weights = choose(L, x, k, True)
    assert np.array_equal(ids.cpu().numpy(), want)
    ref, tol = reference(L, x, want, weights)
    check(y, ref, tol)
    # FP32 output, and the same result on the same workspace
    y32, _, _ = s12.s12_moe(*L.views, E, x, L.router, k, ws=ws, f32=True, err_flag=flag)
    check(y32, ref, tol, bf16=False)
    assert torch.equal(y32.to(torch.bfloat16), y.view(torch.bfloat16))
    assert int(flag.item()) == 0
    assert int(ws[:s12.S12_WS_HEAD].to(torch.int32).sum()) == 0


@pytest.mark.parametrize("version", [1, 2])
@pytest.mark.parametrize("outliers,zeros", [(0.0, 0.0), (0.05, 0.0), (0.3, 0.1), (0.001, 0.5)])
def test_escapes_and_container_versions(s12, version, outliers, zeros):  # noqa: F811
    """From no escapes to many, with runs of zero weights (which are escapes beside ordinary ones)."""
    T, E, k, H, F = 64, 8, 8, 1152, 1280
    assert many(T, k, H, F)
    L = Layer(s12, E, H, F, 7, outliers, zeros, version)
    x, flag = L.tokens(T, 1), new_flag()
    y, ids, w = s12.s12_moe(*L.views, E, x, L.router, k, err_flag=flag)
    want, weights = choose(L, x, k, True)
    check(y, *reference(L, x, want, weights))
    assert int(flag.item()) == 0
    if version == 2:
        one = Layer(s12, E, H, F, 7, outliers, zeros, 1)
        y1, _, _ = s12.s12_moe(*one.views, E, x, L.router, k)
        assert torch.equal(y, y1)


def test_extreme_exponents(s12):  # noqa: F811
    """Every BF16 pattern that is finite and small enough decodes to itself, in rows full of escapes."""
    E, H, F, T, k = 1, 128, 11008, 64, 8
    assert many(T, k, H, F)
    L = Layer(s12, E, H, F, 3)
    pattern = (torch.arange(0, F * H, dtype=torch.int64) * 40503) % 65536
    exponent = (pattern >> 7) & 0xFF
    pattern = torch.where(exponent > 130, (pattern & 0x807F) | ((exponent % 104 + 27) << 7), pattern)
    pattern = torch.where(pattern > 32767, pattern - 65536, pattern)
    L.up = pattern.to(torch.int16).view(torch.bfloat16).view(1, F, H).cuda()
    both = s12.interleave_gate_up(L.gate.view(F, H), L.up.view(F, H))
    L.blobs[0] = s12.s12_encode(both.contiguous())
    L.views[0] = s12.s12_open(L.blobs[0])
    assert int(L.views[0].n_esc) > 100000
    x = torch.eye(H, device="cuda")[:T].to(torch.bfloat16)
    flag = new_flag()
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    weights = np.full((T, k), 0.125)
    y = s12.s12_moe_routed(*L.views, E, x, ids, torch.full((T, k), 0.125, device="cuda"), err_flag=flag, f32=True)
    assert int(flag.item()) == 0
    check(y, *reference(L, x, np.zeros((T, k), int), weights), bf16=False)


@pytest.mark.parametrize("case", ["some dropped", "all dropped", "out of range", "one expert for all", "twice",
                                  "one pair"])
def test_routed(s12, case):  # noqa: F811
    E, T, k, H, F = 3, 64, 8, 1920, 768
    assert many(T, k, H, F)
    L = Layer(s12, E, H, F, 13)
    x = L.tokens(T, 2)
    rng = np.random.default_rng(0)
    ids = rng.integers(0, E, size=(T, k))
    weights = rng.standard_normal((T, k)).astype(np.float32)
    if case == "some dropped":
        ids[rng.random((T, k)) < 0.5] = -1
        ids[7] = -1
    elif case == "all dropped":
        ids[:] = -1
        weights[:] = np.nan  # of a slot that is left out
    elif case == "out of range":
        bad = rng.choice([-1, -2 ** 31, E, 255, 32768, 65536, 2 ** 31 - 1], (T, k))
        ids = np.where(rng.random((T, k)) < 0.4, bad, ids)
    elif case == "one expert for all":
        ids[:] = 2  # 512 pairs: eight reads of its weights, and the longest stages
    elif case == "one pair":
        ids[:] = -1
        ids[40, 5] = 1
    else:
        ids[:, 1] = ids[:, 0]
    flag = new_flag()
    y = torch.full((T, H), float("nan"), device="cuda")
    s12.s12_moe_routed(*L.views, E, x, torch.from_numpy(ids.astype(np.int32)).cuda(),
                       torch.from_numpy(weights).cuda(), y=y, err_flag=flag)
    inside = np.where((ids >= 0) & (ids < E), ids, -1)
    ref, tol = reference(L, x, inside, np.where(inside >= 0, weights, 0))
    check(y, ref, tol, bf16=False)
    assert int(flag.item()) == 0
    none = (inside < 0).all(1)
    assert bool((y[torch.from_numpy(none).cuda()] == 0).all())


def test_nan_token_leaves_the_others(s12):  # noqa: F811
    L = Layer(s12, 8, 1920, 768, 19)
    x = L.tokens(64, 1)
    clean, ids0, _ = s12.s12_moe(*L.views, 8, x, L.router, 8)
    x[3, 17] = float("nan")
    x[6, 40] = float("inf")
    y, ids, w = s12.s12_moe(*L.views, 8, x, L.router, 8)
    got = y.view(torch.bfloat16)
    assert bool(torch.isnan(got[3].float()).all()) and not bool(torch.isfinite(got[6].float()).any())
    # (every token goes to all eight experts, so the others keep their columns and their sums)
    rest = [t for t in range(64) if t not in (3, 6)]
    assert torch.equal(y[rest], clean[rest])


def test_corrupt_offsets_and_bases_are_flagged(s12):  # noqa: F811
    """Escape offsets that point outside, a count that is off by one and a base above 241: read in bounds, and the
    word says so."""
    E, T, k, H, F = 8, 64, 8, 1920, 768
    L = Layer(s12, E, H, F, 23, outliers=0.01)
    x, v = L.tokens(T, 1), L.views[0]
    off, tiles = int(v.esc_off) - int(v.container), int(v.n_tiles)
    for change in ("outside", "one less"):
        host = blob_to_host(L.blobs[0]).copy()
        words = host[off:off + 4 * (tiles + 1)].view(np.uint32)
        if change == "outside":
            words[3:tiles:5] = 0xFFFFFFF0
        else:
            at = int(np.nonzero(np.diff(words.astype(np.int64)) == 3)[0][0])
            words[at + 1:] -= 1
        flag = new_flag()
        s12.s12_moe(s12.s12_open(blob_to_dev(host)), L.views[1], E, x, L.router, k, err_flag=flag)
        assert int(flag.item()) & (s12.S12_FLAG_ESC_COUNT | s12.S12_FLAG_ESC_RANGE)
    host = blob_to_host(L.blobs[0]).copy()
    base = int(v.base) - int(v.container)
    host[base:base + tiles] = 250
    flag = new_flag()
    s12.s12_moe(s12.s12_open(blob_to_dev(host)), L.views[1], E, x, L.router, k, err_flag=flag)
    assert int(flag.item()) & s12.S12_FLAG_BASE
    # and the same layer again, unharmed
    flag = new_flag()
    y, ids, w = s12.s12_moe(*L.views, E, x, L.router, k, err_flag=flag)
    check(y, *reference(L, x, *choose(L, x, k, True)))
    assert int(flag.item()) == 0


def test_graphs_and_streams_that_share(s12):  # noqa: F811
    """Calls of both kernels in captured graphs on one workspace, replayed in turn; two calls at once."""
    E, H, F, k = 8, 1920, 768, 8
    L = Layer(s12, E, H, F, 29)
    ws = s12.moe_workspace(*L.views, E, 64, k)
    xs, graphs, outs = L.tokens(64, 1), [], []
    for T in (64, 3, 63):
        io = (torch.empty(T, H, dtype=torch.int16, device="cuda"),
              torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s12.s12_moe(*L.views, E, xs[:T], L.router, k, y=io[0], ids=io[1], weights=io[2], ws=ws)
        graphs.append(graph)
        outs.append(io)
    for seed in (3, 4):
        xs.copy_(L.tokens(64, seed))
        for graph, io in zip(graphs, outs):
            graph.replay()
            want = s12.s12_moe(*L.views, E, xs[:io[0].shape[0]], L.router, k)
            assert all(torch.equal(a, b) for a, b in zip(io, want))
    ref, got = s12.s12_moe(*L.views, E, xs, L.router, k), []
    torch.cuda.synchronize()
    for st in [torch.cuda.Stream() for _ in range(2)]:
        mine = s12.moe_workspace(*L.views, E, 64, k)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(3):
                got.append(s12.s12_moe(*L.views, E, xs, L.router, k, ws=mine))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(ref, out))
