"""s12_moe and s12_moe_routed on the GPU against the layer in 64 bits.

Tolerance.  A sum of n products in FP32 is off by at most n * 2^-23 of the sum
of its terms' magnitudes (the tensor cores may truncate, hence a whole step).
So the gate and up sums are within e_g = H * 2^-23 * sum|W x|, h is within
1.1 |u| e_g + |silu(g)| e_u + 1.1 e_g e_u + 2^-17 |h| (|silu'| <= 1.1; two BF16
values hold 16 bits or more; expf and the division are within 2^-20), a down
sum adds F * 2^-23 * sum|W h|, and the weights and the sum over the slots add
(top_k + 8) * 2^-23 of their terms.  A BF16 y adds half a step, 2^-8 |y|."""
import numpy as np
import pytest
import torch

from gpu_util import blob_to_dev, blob_to_host, new_flag

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def s12(cuda_ok):
    from decode_split12_b200 import s12 as mod
    mod.device_check()
    return mod


class Layer:
    """Experts' matrices (BF16) and their containers."""

    def __init__(self, s12, E, H, F, seed, outliers=0.002, zeros=0.0, version=1):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weights(*shape):
            w = torch.randn(shape, generator=g, device="cuda") / shape[-1] ** 0.5
            u = torch.rand(shape, generator=g, device="cuda")
            w = torch.where(u < outliers, w * 40, w)
            return torch.where(u > 1 - zeros, torch.zeros_like(w), w).to(torch.bfloat16)

        self.E, self.H, self.F = E, H, F
        self.gate, self.up, self.down = weights(E, F, H), weights(E, F, H), weights(E, H, F)
        both = s12.interleave_gate_up(self.gate.view(E * F, H), self.up.view(E * F, H))
        blobs = [s12.s12_encode(both.contiguous()), s12.s12_encode(self.down.view(E * H, F))]
        if version == 2:
            blobs = [blob_to_dev(s12.to_v2_host(blob_to_host(b))) for b in blobs]
        self.blobs = blobs
        self.views = [s12.s12_open(b) for b in blobs]
        self.router = (torch.randn(E, H, generator=g, device="cuda") / H ** 0.5).to(torch.bfloat16)

    def tokens(self, T, seed):
        g = torch.Generator(device="cuda").manual_seed(1000 + seed)
        return torch.randn(T, self.H, generator=g, device="cuda").to(torch.bfloat16)


def choose(L, x, k, renorm):
    """ids and weights in 64 bits, the lower index first at a tie."""
    score = (x.double() @ L.router.double().T).cpu().numpy()
    ids = np.stack([np.lexsort((np.arange(L.E), -row))[:k] for row in score])
    top = np.take_along_axis(score, ids, 1)
    e = np.exp(top - top[:, :1])
    total = e.sum(1, keepdims=True) if renorm else np.exp(score - top[:, :1]).sum(1, keepdims=True)
    return ids, e / total


def reference(L, x, ids, weights):
    """(y, tolerance before y's own rounding) in 64 bits."""
    T, k = ids.shape
    y = torch.zeros(T, L.H, dtype=torch.float64, device="cuda")
    tol, terms = torch.zeros_like(y), torch.zeros_like(y)
    step = 2.0 ** -23
    for e in range(L.E):
        for s in range(k):
            t = torch.as_tensor(np.nonzero(ids[:, s] == e)[0], device="cuda")
            if not len(t):
                continue
            xs, w = x[t].double(), torch.as_tensor(weights[t.cpu().numpy(), s], device="cuda").double()[:, None]
            G, U, D = L.gate[e].double(), L.up[e].double(), L.down[e].double()
            g, u = xs @ G.T, xs @ U.T
            eg, eu = L.H * step * (xs.abs() @ G.abs().T), L.H * step * (xs.abs() @ U.abs().T)
            silu = g * torch.sigmoid(g)
            h = silu * u
            eh = 1.1 * u.abs() * eg + silu.abs() * eu + 1.1 * eg * eu + 2.0 ** -17 * h.abs()
            d, sd = h @ D.T, h.abs() @ D.abs().T
            y.index_add_(0, t, w * d)
            tol.index_add_(0, t, w.abs() * (eh @ D.abs().T + L.F * step * sd))
            terms.index_add_(0, t, (w * d).abs())
    return y, tol + (k + 8) * step * terms + 1e-30


def check(y, ref, tol, bf16=True):
    got = y.view(torch.bfloat16).double() if bf16 else y.double()
    bound = tol + (2.0 ** -8 * (ref.abs() + tol) if bf16 else 0)
    err = (got - ref).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((err <= bound).all()), float((err / bound).max())


SHAPES = [  # T, E, k, H, F
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 384), (3, 4, 4, 640, 128), (8, 2, 1, 128, 1152), (9, 5, 3, 384, 256),
    (16, 2, 2, 256, 256), (17, 3, 2, 384, 640), (33, 2, 2, 256, 128), (64, 2, 2, 128, 384), (64, 40, 8, 256, 128),
    (64, 256, 8, 128, 128), (2, 8, 2, 4096, 1408), (5, 16, 8, 2176, 896), (25, 8, 3, 1024, 2048)]


@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
def test_moe_small_and_odd_shapes(s12, T, E, k, H, F):
    L = Layer(s12, E, H, F, T * 31 + E)
    x, flag = L.tokens(T, E), new_flag()
    ws = s12.moe_workspace(*L.views, E, T, k)
    y, ids, w = s12.s12_moe(*L.views, E, x, L.router, k, ws=ws, err_flag=flag)
    want, weights = choose(L, x, k, True)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.abs(w.cpu().numpy() - weights).max() <= 2.0 ** -20
    ref, tol = reference(L, x, want, weights)
    check(y, ref, tol)
    assert int(flag.item()) == 0
    # FP32 output, and the same result on the same workspace
    y32, _, _ = s12.s12_moe(*L.views, E, x, L.router, k, ws=ws, f32=True)
    check(y32, ref, tol, bf16=False)
    assert torch.equal(y32.to(torch.bfloat16), y.view(torch.bfloat16))
    # the words that have to be zero between calls are
    assert int(ws[:s12.S12_WS_HEAD].to(torch.int32).sum()) == 0


def test_one_workspace_for_calls_of_any_shape(s12):
    """Only the first words have to be zero: layers of other shapes may use the workspace in turn."""
    cases = [(Layer(s12, E, H, F, E), T, k) for T, E, k, H, F in ((64, 4, 2, 384, 256), (1, 8, 2, 256, 640),
                                                                  (9, 40, 3, 128, 128), (33, 2, 1, 512, 128))]
    need = max([s12.s12_moe_ws_bytes(*L.views, L.E, T, k) for L, T, k in cases] + [s12.s12_gemm_i8_ws_bytes(300)])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    ws[:s12.S12_WS_HEAD] = 0
    q = torch.randint(-128, 128, (300, 256), dtype=torch.int8, device="cuda")
    one = torch.ones(300, device="cuda")
    for _ in range(2):
        for L, T, k in cases:
            # (the 8-bit product between them, with parts of tiles joined)
            prod = s12.s12_gemm_i8(q, one, q, one, ws=ws, f32=True)
            assert torch.equal(prod.double(), q.double() @ q.double().T)
            x = L.tokens(T, k)
            y, ids, w = s12.s12_moe(*L.views, L.E, x, L.router, k, ws=ws)
            check(y, *reference(L, x, *choose(L, x, k, True)))


@pytest.mark.parametrize("version", [1, 2])
@pytest.mark.parametrize("outliers,zeros", [(0.0, 0.0), (0.05, 0.0), (0.3, 0.1), (0.001, 0.5)])
def test_moe_escapes_and_container_versions(s12, version, outliers, zeros):
    """From no escapes to many, with runs of zero weights (which are escapes beside ordinary ones)."""
    L = Layer(s12, 3, 640, 384, 7, outliers, zeros, version)
    if outliers:
        assert int(L.views[0].n_esc) > 0
    x, flag = L.tokens(11, 1), new_flag()
    y, ids, w = s12.s12_moe(*L.views, 3, x, L.router, 2, err_flag=flag)
    want, weights = choose(L, x, 2, True)
    assert np.array_equal(ids.cpu().numpy(), want)
    check(y, *reference(L, x, want, weights))
    assert int(flag.item()) == 0
    if version == 1:
        return
    one = Layer(s12, 3, 640, 384, 7, outliers, zeros, 1)
    y1, _, _ = s12.s12_moe(*one.views, 3, x, L.router, 2)
    assert torch.equal(y, y1)


def test_moe_extreme_exponents(s12):
    """Every BF16 pattern that is finite and small enough decodes to itself: one token that is 1 in one column
    reads that column of gate and up through the whole path."""
    E, H, F = 1, 128, 128
    L = Layer(s12, E, H, F, 3)
    bits = torch.arange(0, F * H, dtype=torch.int32)
    pattern = (bits * 40503) % 65536
    exponent = (pattern >> 7) & 0xFF
    # exponents around and far below 1 (2^-100 .. 2^3), zeros and subnormals among them
    pattern = torch.where(exponent > 130, (pattern & 0x807F) | ((exponent % 104 + 27) << 7), pattern)
    L.up = pattern.to(torch.int16).view(torch.bfloat16).view(1, F, H).cuda()
    both = s12.interleave_gate_up(L.gate.view(F, H), L.up.view(F, H))
    L.blobs[0] = s12.s12_encode(both.contiguous())
    L.views[0] = s12.s12_open(L.blobs[0])
    assert int(L.views[0].n_esc) > 1000
    x = torch.eye(H, device="cuda")[:64].to(torch.bfloat16)
    flag = new_flag()
    ids = torch.zeros(64, 1, dtype=torch.int32, device="cuda")
    y = s12.s12_moe_routed(*L.views, 1, x, ids, torch.ones(64, 1, device="cuda"), err_flag=flag, f32=True)
    assert int(flag.item()) == 0
    check(y, *reference(L, x, np.zeros((64, 1), int), np.ones((64, 1))), bf16=False)


@pytest.mark.parametrize("renorm", [True, False])
def test_moe_ties_and_weights(s12, renorm):
    """Experts with equal router rows: the lower index comes first; weights over all experts or the chosen ones."""
    L = Layer(s12, 6, 256, 128, 11)
    L.router[4] = L.router[1]
    L.router[5] = L.router[1]
    x = L.tokens(24, 5)
    y, ids, w = s12.s12_moe(*L.views, 6, x, L.router, 3, renorm=renorm)
    want, weights = choose(L, x, 3, renorm)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.abs(w.cpu().numpy() - weights).max() <= 2.0 ** -20
    check(y, *reference(L, x, want, weights))


@pytest.mark.parametrize("case", ["some dropped", "all dropped", "out of range", "one expert for all", "twice"])
def test_routed(s12, case):
    E, T, k = 5, 64, 8
    L = Layer(s12, E, 384, 256, 13)
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
        ids = np.where(rng.random((T, k)) < 0.4, rng.choice([-1, -2 ** 31, E, 255, 32768, 65536, 2 ** 31 - 1], (T, k)), ids)
    elif case == "one expert for all":
        ids[:] = 3  # 512 pairs: eight reads of its weights
    else:
        ids[:, 1] = ids[:, 0]
    di = torch.from_numpy(ids.astype(np.int32)).cuda()
    flag = new_flag()
    y = torch.full((T, L.H), float("nan"), device="cuda")
    s12.s12_moe_routed(*L.views, E, x, di, torch.from_numpy(weights).cuda(), y=y, err_flag=flag)
    inside = np.where((ids >= 0) & (ids < E), ids, -1)
    ref, tol = reference(L, x, inside, np.where(inside >= 0, weights, 0))
    check(y, ref, tol, bf16=False)
    assert int(flag.item()) == 0
    none = (inside < 0).all(1)
    assert bool((y[torch.from_numpy(none).cuda()] == 0).all())


def test_one_workspace_for_calls_of_different_tokens(s12):
    L = Layer(s12, 8, 512, 256, 17)
    ws = s12.moe_workspace(*L.views, 8, 64, 2)
    first = {}
    for T in (1, 64, 7, 64, 1, 33, 7):
        x = L.tokens(T, T)
        y, ids, w = s12.s12_moe(*L.views, 8, x, L.router, 2, ws=ws)
        if T in first:
            assert all(torch.equal(a, b) for a, b in zip(first[T], (y, ids, w)))
        else:
            want, weights = choose(L, x, 2, True)
            check(y, *reference(L, x, want, weights))
            first[T] = (y, ids, w)


def test_workspace_grows_with_tokens(s12):
    """The size for the most tokens serves every smaller number of them."""
    for E, H, F in ((8, 512, 384), (64, 256, 128), (2, 384, 1152)):
        v = []
        for rows, cols in ((E * 2 * F, H), (E * H, F)):
            v.append(s12.s12_open(s12.s12_encode(torch.zeros(rows, cols, dtype=torch.int16, device="cuda"))))
        for k in (1, 2):
            sizes = [s12.s12_moe_ws_bytes(*v, E, T, k) for T in range(1, 65)]
            assert sizes == sorted(sizes)


def test_nan_token_leaves_the_others(s12):
    L = Layer(s12, 4, 256, 256, 19)
    x = L.tokens(10, 1)
    clean, ids0, _ = s12.s12_moe(*L.views, 4, x, L.router, 2)
    x[3, 17] = float("nan")
    x[6, 40] = float("inf")
    y, ids, w = s12.s12_moe(*L.views, 4, x, L.router, 2)
    assert bool(torch.isnan(y.view(torch.bfloat16)[3].float()).all()) and bool(torch.isnan(w[3]).all())
    assert not bool(torch.isfinite(y.view(torch.bfloat16)[6].float()).any())
    for t in (0, 1, 2, 4, 5, 7, 8, 9):
        assert torch.equal(ids[t], ids0[t])
        a, b = y.view(torch.bfloat16)[t].double(), clean.view(torch.bfloat16)[t].double()
        # (the same sums: which column of the products a token sits in does not change them)
        assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-6).all())


def test_corrupt_offsets_and_bases_are_flagged(s12):
    """Escape offsets that point outside and a base above 241: read in bounds, and the word says so."""
    L = Layer(s12, 2, 256, 128, 23, outliers=0.01)
    x = L.tokens(4, 1)
    v = L.views[0]
    host = blob_to_host(L.blobs[0]).copy()
    off = int(v.esc_off) - int(v.container)
    words = host[off:off + 4 * int(v.n_tiles)].view(np.uint32)
    words[3::5] = 0xFFFFFFF0
    bad = blob_to_dev(host)
    flag = new_flag()
    s12.s12_moe(s12.s12_open(bad), L.views[1], 2, x, L.router, 2, err_flag=flag)
    assert int(flag.item()) & (s12.S12_FLAG_ESC_COUNT | s12.S12_FLAG_ESC_RANGE)
    host = blob_to_host(L.blobs[0]).copy()
    base = int(v.base) - int(v.container)
    host[base:base + int(v.n_tiles)] = 250
    flag = new_flag()
    s12.s12_moe(s12.s12_open(blob_to_dev(host)), L.views[1], 2, x, L.router, 2, err_flag=flag)
    assert int(flag.item()) & s12.S12_FLAG_BASE


def test_other_stream_two_workspaces_and_replayed_graph(s12):
    L = Layer(s12, 8, 512, 384, 29)
    x = L.tokens(12, 1)
    ref = s12.s12_moe(*L.views, 8, x, L.router, 2)
    torch.cuda.synchronize()
    # two calls at once, each with its own workspace
    out, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        ws = s12.moe_workspace(*L.views, 8, 12, 2)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(3):
                out.append(s12.s12_moe(*L.views, 8, x, L.router, 2, ws=ws))
    torch.cuda.synchronize()
    for got in out:
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    # two graphs that share a workspace, replayed in turn
    ws = s12.moe_workspace(*L.views, 8, 12, 2)
    xs, graphs, outs = x.clone(), [], []
    for T in (12, 5):
        io = (torch.empty(T, L.H, dtype=torch.int16, device="cuda"),
              torch.empty(T, 2, dtype=torch.int32, device="cuda"), torch.empty(T, 2, device="cuda"))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s12.s12_moe(*L.views, 8, xs[:T], L.router, 2, y=io[0], ids=io[1], weights=io[2], ws=ws)
        graphs.append(graph)
        outs.append(io)
    for seed in (3, 4):
        xs.copy_(L.tokens(12, seed))
        for graph, io in zip(graphs, outs):
            graph.replay()
            T = io[0].shape[0]
            want = s12.s12_moe(*L.views, 8, xs[:T], L.router, 2)
            assert all(torch.equal(a, b) for a, b in zip(io, want))


def test_no_tokens_and_binding_refusals(s12):
    L = Layer(s12, 4, 256, 128, 31)
    x = L.tokens(3, 1)
    y, ids, w = s12.s12_moe(*L.views, 4, x[:0], L.router, 2)
    assert y.shape == (0, 256) and ids.shape == (0, 2)
    with pytest.raises(s12.S12Error):
        s12.s12_moe(*L.views, 4, x, L.router, 5)
    with pytest.raises(s12.S12Error):
        s12.s12_moe(L.views[1], L.views[1], 4, x, L.router, 2)
    with pytest.raises(s12.S12Error):
        s12.s12_moe(*L.views, 4, x, L.router, 2, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        s12.s12_moe(*L.views, 4, x[:, :128], L.router, 2)
    with pytest.raises(ValueError):
        s12.s12_moe(*L.views, 4, x, L.router[:3], 2)
    with pytest.raises(ValueError):
        s12.s12_moe(*L.views, 4, x.float(), L.router, 2)
    with pytest.raises(ValueError):
        s12.s12_moe_routed(*L.views, 4, x, torch.zeros(3, 2, dtype=torch.int64, device="cuda"),
                           torch.zeros(3, 2, device="cuda"))
    with pytest.raises(ValueError):
        s12.s12_moe_routed(*L.views, 4, x, torch.zeros(3, 2, dtype=torch.int32, device="cuda"),
                           torch.zeros(3, 3, device="cuda"))


@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 4096, 14336), (64, 8, 2, 4096, 14336), (64, 32, 4, 2176, 1408),
                                       (9, 32, 4, 2176, 1408), (40, 64, 8, 2048, 1024)])
def test_moe_full_size_block(s12, T, E, k, H, F):
    """The 8-expert block of the benchmark, top 2; many smaller experts, whose last rows leave warps without a row
    group while column ranges of one stage follow one another."""
    L = Layer(s12, E, H, F, 37, outliers=0.0005)
    x, flag = L.tokens(T, 1), new_flag()
    y, ids, w = s12.s12_moe(*L.views, E, x, L.router, k, err_flag=flag)
    want, weights = choose(L, x, k, True)
    assert np.array_equal(ids.cpu().numpy(), want)
    check(y, *reference(L, x, want, weights))
    assert int(flag.item()) == 0
