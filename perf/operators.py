"""Cases for the operators that surround the fused decode products: the RMS norm with the residual's
addition (BF16 or 8-bit output), the row quantiser, the 8-bit integer product with a scale for each
token and channel, and the whole mixture-of-experts layer over Split12 experts.

`own` selects what `run` computes: False, the operators in plain torch operations in 32 bits (64 where a
choice hangs on them); True, the calls of decode_split12_b200.s12.  The expert weights are BF16 matrices
in the plain form and the containers encoded from them in the other, which is what each program keeps.
8-bit outputs come back as the values they stand for (integer times scale, as BF16).
"""
import math

import torch

own = False


def _lib():
    from decode_split12_b200 import s12  # only where own is true
    return s12


# ---- cases -----------------------------------------------------------------------------------------

# share of the weights that are much larger than the rest
OUTLIERS = 0.0005
# bytes of a container per weight: 12 bits, a base and an offset for each 128, and its rare escapes
CONTAINER = 1.5 + 5 / 128 + 2 * OUTLIERS

# the largest listed sizes, which drawn cases stay below
MOST = {"norm": 4096 * 8192, "quant": 28672 * 8192, "i8": 4096 * 14336 * 4096, "moe": 3 * 8 * 14336 * 4096}


def listed():
    return [
        # one decode step of one sequence: the norm before a layer's first product
        {"name": "norm_decode_1x4096", "op": "norm", "rows": 1, "cols": 4096, "f32": False, "eight": False},
        # a batch of sequences, 32-bit sums from the GEMV and a 32-bit residual, in front of an 8-bit product;
        # a hidden size that fills no power of two
        {"name": "norm_batch_33x2056_i8", "op": "norm", "rows": 33, "cols": 2056, "f32": True, "eight": True},
        # a prompt through a 70B-style layer, in front of an 8-bit product
        {"name": "norm_prompt_4096x8192_i8", "op": "norm", "rows": 4096, "cols": 8192, "f32": False, "eight": True},
        # hidden activations of a few tokens made 8-bit for the down projection
        {"name": "quant_hidden_7x14336", "op": "quant", "rows": 7, "cols": 14336, "f32": True},
        # a 70B-style weight matrix made 8-bit when a model is loaded
        {"name": "quant_weight_28672x8192", "op": "quant", "rows": 28672, "cols": 8192, "f32": False},
        # the down projection of one decoded token
        {"name": "i8_decode_1x4096x14336", "op": "i8", "M": 1, "N": 4096, "K": 14336, "f32": True},
        # a ragged batch against a matrix whose sizes fill no tile
        {"name": "i8_batch_19x5000x2064", "op": "i8", "M": 19, "N": 5000, "K": 2064, "f32": False},
        # a large decode batch through a 70B-style up projection
        {"name": "i8_batch_256x28672x8192", "op": "i8", "M": 256, "N": 28672, "K": 8192, "f32": False},
        # a prompt through an 8B-style up projection
        {"name": "i8_prompt_4096x14336x4096", "op": "i8", "M": 4096, "N": 14336, "K": 4096, "f32": False},
        # the 8-expert block, top 2, one decoded token
        {"name": "moe_1_of_8x14336x4096", "op": "moe", "T": 1, "E": 8, "k": 2, "H": 4096, "F": 14336,
         "routed": False},
        # many small experts whose sizes are odd numbers of tiles, routed by the caller, some slots dropped
        {"name": "moe_9_of_32x1408x2176_routed", "op": "moe", "T": 9, "E": 32, "k": 4, "H": 2176, "F": 1408,
         "routed": True},
        # the 8-expert block, top 2, a batch of 64
        {"name": "moe_64_of_8x14336x4096", "op": "moe", "T": 64, "E": 8, "k": 2, "H": 4096, "F": 14336,
         "routed": False},
    ]


def _size(rng, low, high, step=1):
    """A multiple of `step` between low and high, even over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high // step, max(-(-low // step), round(v / step))) * step


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "i8", "i8", "moe", "moe"])
    f32 = rng.random() < 0.4
    if op in ("norm", "quant"):
        cols = _size(rng, 64, 28672, 8)
        c = {"op": op, "rows": _size(rng, 1, min(28672, MOST[op] // cols // 2)), "cols": cols, "f32": f32}
        return {**c, "eight": rng.random() < 0.5} if op == "norm" else c
    if op == "i8":
        N, K = _size(rng, 16, 28672), _size(rng, 16, 14336, 16)
        return {"op": op, "M": _size(rng, 1, min(4096, max(1, MOST[op] // (N * K)))), "N": N, "K": K, "f32": f32}
    E, H = _size(rng, 2, 64), _size(rng, 256, 4096, 128)
    F = _size(rng, 128, max(128, min(14336, MOST[op] // (3 * E * H))), 128)
    return {"op": op, "T": _size(rng, 1, 64), "E": E, "k": rng.randint(1, min(8, E)), "H": H, "F": F,
            "routed": rng.random() < 0.3}


def work(case):
    op = case["op"]
    if op in ("norm", "quant"):
        n, wide = case["rows"] * case["cols"], 4 if case["f32"] else 2
        if op == "quant":
            return {"bytes": n * (wide + 1) + 4 * case["rows"], "flops": 3 * n}
        out = 1 if case["eight"] else 2
        return {"bytes": n * (3 * wide + out) + 2 * case["cols"] + 4 * case["rows"] * case["eight"], "flops": 6 * n}
    if op == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * (4 if case["f32"] else 2), "flops": 2 * M * N * K}
    T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
    met = E * (1 - (1 - k / E) ** T)  # experts that some token is sent to, on average
    router = 0 if case["routed"] else E * H
    return {"bytes": met * 3 * F * H * CONTAINER + 2 * router + T * (4 * H + 8 * k),
            "flops": 2 * T * (k * 3 * F * H + router)}


# ---- inputs ----------------------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _weights(gen, rows, cols):
    """N(0, 1/sqrt(cols)) with 0.05 % of the values 10 to 100 times as large, BF16."""
    w = _normal(gen, rows, cols).mul_(1 / math.sqrt(cols))
    u = torch.rand((rows, cols), generator=gen, device="cuda")
    return w.mul_(torch.where(u < OUTLIERS, 10 + u * (90 / OUTLIERS), 1.0)).to(torch.bfloat16)


def _eights(gen, rows, cols):
    return (_normal(gen, rows, cols) * 36).round_().clamp_(-127, 127).to(torch.int8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] in ("norm", "quant"):
        wide = torch.float32 if case["f32"] else torch.bfloat16
        rows, cols = case["rows"], case["cols"]
        if case["op"] == "quant":
            s["x"] = _normal(gen, rows, cols).mul_(1 / math.sqrt(cols)).to(wide)
        else:
            # a residual stream has a few channels that are much larger than the rest
            loud = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.002, 30.0, 1.0)
            s["x"] = _normal(gen, rows, cols).to(wide)
            s["residual"] = (_normal(gen, rows, cols) * loud * 4).to(wide)
            s["weight"] = (1 + 0.2 * _normal(gen, cols)).to(torch.bfloat16)
            s["residual_out"] = torch.empty_like(s["residual"])
        s["values"] = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"], s["w"] = _eights(gen, M, K), _eights(gen, N, K)
        s["x_scale"] = torch.rand(M, generator=gen, device="cuda") * 0.05 + 0.01
        s["w_scale"] = (torch.rand(N, generator=gen, device="cuda") * 0.05 + 0.01) / math.sqrt(K)
        if own:
            s["ws"] = _lib().gemm_i8_workspace(M, N, K)
    else:
        T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
        # each expert's gate and up rows in alternate blocks of eight, expert after expert
        up, down = _weights(gen, E * 2 * F, H), _weights(gen, E * H, F)
        s["x"] = _normal(gen, T, H).to(torch.bfloat16)
        if case["routed"]:
            ids = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :k].to(torch.int32)
            drop = torch.rand((T, k), generator=gen, device="cuda") < 0.1
            s["ids"] = torch.where(drop, -1, ids).to(torch.int32).contiguous()
            s["weights"] = torch.rand((T, k), generator=gen, device="cuda")
        else:
            s["router"] = (_normal(gen, E, H) / math.sqrt(H)).to(torch.bfloat16)
        if own:
            lib = _lib()
            s["up"], s["down"] = lib.Container(lib.s12_encode(up)).view, lib.Container(lib.s12_encode(down)).view
            s["ws"] = lib.moe_workspace(s["up"], s["down"], E, T, k)
        else:
            s["up"], s["down"] = up.view(E, 2 * F, H), down.view(E, H, F)
    return s


# ---- the operators ---------------------------------------------------------------------------------

EPS = 1e-6


def run(s):
    return {"norm": _norm, "quant": _quant, "i8": _i8, "moe": _moe}[s["op"]](s)


def _to_eight(v):
    """Integers of at most 127 and their scale, a row's largest magnitude over 127."""
    scale = v.abs().amax(1, keepdim=True) / 127
    return torch.round(v / scale), scale


def _norm(s):
    if own:
        y, q, scale, res = _lib().s12_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"],
                                              residual_out=s["residual_out"], bf16=not s["eight"], int8=s["eight"])
        if not s["eight"]:
            return {"y": y.view(torch.bfloat16), "residual": res}
        return {"values": torch.mul(q, scale[:, None], out=s["values"]), "scale": scale, "residual": res}
    r = s["x"].float() + s["residual"].float()
    v = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    res = r.to(s["residual"].dtype)
    if not s["eight"]:
        return {"y": v.to(torch.bfloat16), "residual": res}
    q, scale = _to_eight(v)
    return {"values": (q * scale).to(torch.bfloat16), "scale": scale[:, 0], "residual": res}


def _quant(s):
    if own:
        q, scale = _lib().s12_quant_i8(s["x"])
        return {"values": torch.mul(q, scale[:, None], out=s["values"]), "scale": scale}
    q, scale = _to_eight(s["x"].float())
    return {"values": (q * scale).to(torch.bfloat16), "scale": scale[:, 0]}


def _i8(s):
    if own:
        y = _lib().s12_gemm_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], ws=s["ws"], f32=s["f32"])
        return y if s["f32"] else y.view(torch.bfloat16)
    y = s["x"].float() @ s["w"].float().T * s["x_scale"][:, None] * s["w_scale"]
    return y if s["f32"] else y.to(torch.bfloat16)


def _moe(s):
    if own:
        if s["routed"]:
            y = _lib().s12_moe_routed(s["up"], s["down"], s["E"], s["x"], s["ids"], s["weights"], ws=s["ws"])
            return {"y": y.view(torch.bfloat16)}
        y, ids, weights = _lib().s12_moe(s["up"], s["down"], s["E"], s["x"], s["router"], s["k"], ws=s["ws"])
        return {"y": y.view(torch.bfloat16), "ids": ids, "weights": weights}
    T, E, k, F = s["T"], s["E"], s["k"], s["F"]
    x, said = s["x"].float(), {}
    if s["routed"]:
        ids, weights = s["ids"].long(), s["weights"] * (s["ids"] >= 0)
        ids = ids.clamp(min=0)
    else:
        # 64 bits: which experts are chosen hangs on the order of the scores
        scores = s["x"].double() @ s["router"].double().T
        top, ids = torch.sort(scores, dim=1, descending=True, stable=True)
        ids, weights = ids[:, :k], torch.exp(top[:, :k] - top[:, :1])
        weights = (weights / weights.sum(1, keepdim=True)).float()
        said = {"ids": ids.to(torch.int32), "weights": weights}
    if T * k <= E:  # the chosen experts alone, once for each slot
        at = ids.reshape(-1)
        gu = s["up"][at].float() @ x.repeat_interleave(k, 0)[:, :, None]
        d = s["down"][at].float() @ _gated(gu[:, :, 0], F)[:, :, None]
        y = (d.view(T, k, -1) * weights[:, :, None]).sum(1)
    else:  # every expert on every token
        d = _gated(x @ s["up"].float().transpose(1, 2), F) @ s["down"].float().transpose(1, 2)
        share = torch.zeros((T, E), device="cuda").scatter_add_(1, ids, weights)
        y = (d * share.T[:, :, None]).sum(0)
    return {"y": y.to(torch.bfloat16), **said}


def _gated(gu, F):
    gu = gu.unflatten(-1, (F // 8, 2, 8))
    g, u = gu[..., 0, :], gu[..., 1, :]
    return (g / (1 + torch.exp(-g)) * u).flatten(-2)


# ---- the definitions in 64 bits --------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64

    def eight(v):
        scale = v.abs().max(dim=1, keepdim=True).values / 127
        return {"values": torch.round(v / scale) * scale, "scale": scale[:, 0]}

    if case["op"] == "norm":
        r = s["residual"].to(f8).add_(s["x"])
        length = (r * r).sum(dim=1, keepdim=True) / case["cols"] + EPS
        v = r / length.sqrt() * s["weight"].to(f8)
        return {**(eight(v) if case["eight"] else {"y": v}), "residual": r}
    if case["op"] == "quant":
        return eight(s["x"].to(f8))
    if case["op"] == "i8":
        a, b = s["x"].to(f8) * s["x_scale"].to(f8)[:, None], s["w"].to(f8) * s["w_scale"].to(f8)[:, None]
        return torch.matmul(a, b.T)
    T, k, F = case["T"], case["k"], case["F"]
    x, said = s["x"].to(f8), {}
    if case["routed"]:
        ids, weights = s["ids"].tolist(), s["weights"].tolist()
    else:
        scores = (x @ s["router"].to(f8).T).tolist()
        ids = [sorted(range(len(row)), key=lambda e: (-row[e], e))[:k] for row in scores]
        terms = [[math.exp(row[e] - row[at[0]]) for e in at] for row, at in zip(scores, ids)]
        weights = [[v / sum(row) for v in row] for row in terms]
        said = {"ids": torch.tensor(ids, dtype=torch.int32), "weights": torch.tensor(weights, dtype=f8)}
    y = torch.zeros((T, case["H"]), dtype=f8, device="cuda")
    for e in range(case["E"]):
        sent = [(t, weights[t][j]) for t in range(T) for j in range(k) if ids[t][j] == e]
        if not sent:
            continue
        at = torch.tensor([t for t, _ in sent], device="cuda")
        share = torch.tensor([w for _, w in sent], dtype=f8, device="cuda")
        both = (x[at] @ s["up"][e].to(f8).T).reshape(len(sent), F // 8, 16)
        g, u = both[:, :, :8].reshape(len(sent), F), both[:, :, 8:].reshape(len(sent), F)
        y.index_add_(0, at, (g * torch.sigmoid(g) * u) @ s["down"][e].to(f8).T * share[:, None])
    return {"y": y, **said}
