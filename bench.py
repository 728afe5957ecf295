#!/usr/bin/env python
"""Benchmark of the Split12 fused decode-GEMV (and the other kernels).

Default workload (one JSON line on rank 0): one Llama-style 8B decoder layer
-- q, o 4096x4096; k, v 1024x4096; gate, up 14336x4096; down 4096x14336,
Student-t(5) weights scaled to std 1/sqrt(in) -- encoded once into Split12
containers resident in HBM.  A step is the seven fused decode-GEMVs of the
layer at batch 1 (the decode phase of one token).  The metric is effective
BF16 GB/s = 2 bytes x weights / time, with the fraction of the measured HBM
copy bandwidth achieved on the compressed bytes actually moved.

    python bench.py [--gpus N --steps K --warmup W] [--impl reference]
                    [--workload llama8b|single] [--batch B]
                    [--no-cpu-baseline] [--no-gemm] [--no-decode] [--no-stack]

The line's roofline.comparisons carry the uncompressed BF16 GEMV on the same
layer, the layer in 8 bits, the 4096 x 4096 single tensor, the layer from
version 2 containers and the encoder; `extra` the other batches, launch groupings, the SwiGLU
epilogue, the skinny GEMM, the standalone decode, the 32-layer stack (also
as an activation chain) and the MoE block.

Several GPUs run independent replicas (the path does not shard): every
rank times its own copy and rank 0 reports the sum of work over the max
time over ranks.
"""
from __future__ import annotations

import argparse
import json
import math
import os
import statistics
import sys
import threading
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from decode_split12_b200 import workloads as wl  # noqa: E402

HBM_FALLBACK_GBS = 6650.0
L2_BYTES_B200 = 126 * 1024 * 1024
METRIC = "fused decode-GEMV effective BF16 GB/s & % HBM roofline on compressed bytes"


# --------------------------------------------------------------------------- helpers

def load_peaks():
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        with open(path) as f:
            d = json.load(f)
        return float(d["hbm_gbs"]), float(d.get("bf16_tflops", 1590.0)), \
            float(d.get("bf16_tflops_sustained", 1400.0)), "measured"
    except Exception:
        return HBM_FALLBACK_GBS, 1590.0, 1400.0, "fallback"


class ClockSampler:
    """Samples SM clock and clock-event reasons through NVML while running."""

    REASONS = {0x1: "gpu_idle", 0x2: "applications_clocks_setting", 0x4: "sw_power_cap", 0x8: "hw_slowdown",
               0x10: "sync_boost", 0x20: "sw_thermal_slowdown", 0x40: "hw_thermal_slowdown",
               0x80: "hw_power_brake_slowdown", 0x100: "display_clock_setting"}

    def __init__(self, device_index: int, period_s: float = 0.0005):
        self.period = period_s
        self.samples = []
        self.t_start = self.t_end = None
        self.max_mhz = None
        self._stop = threading.Event()
        self._thr = None
        self.ok = False
        try:
            import pynvml
            pynvml.nvmlInit()
            self.nv = pynvml
            vis = os.environ.get("CUDA_VISIBLE_DEVICES")
            idx = device_index
            if vis:
                parts = [p for p in vis.split(",") if p.strip()]
                if device_index < len(parts) and parts[device_index].strip().isdigit():
                    idx = int(parts[device_index])
            self.h = pynvml.nvmlDeviceGetHandleByIndex(idx)
            self.max_mhz = pynvml.nvmlDeviceGetMaxClockInfo(self.h, pynvml.NVML_CLOCK_SM)
            self.ok = True
        except Exception:
            self.ok = False

    def _run(self):
        nv = self.nv
        while not self._stop.is_set():
            try:
                mhz = nv.nvmlDeviceGetClockInfo(self.h, nv.NVML_CLOCK_SM)
                try:
                    reasons = nv.nvmlDeviceGetCurrentClocksEventReasons(self.h)
                except Exception:
                    reasons = nv.nvmlDeviceGetCurrentClocksThrottleReasons(self.h)
                self.samples.append((mhz, int(reasons), time.perf_counter()))
            except Exception:
                pass
            time.sleep(self.period)

    def __enter__(self):
        if self.ok:
            self._thr = threading.Thread(target=self._run, daemon=True)
            self._thr.start()
        return self

    def __exit__(self, *a):
        self._stop.set()
        if self._thr:
            self._thr.join()

    def mark_start(self):
        self.t_start = time.perf_counter()

    def mark_end(self):
        self.t_end = time.perf_counter()

    def summary(self):
        """Median SM clock and the clock-event reasons over every sample taken
        while the GPU was under load (the pre-warm replays right before the
        timed region and the timed region itself); `samples_timed` counts
        those inside the timed region."""
        if not self.samples:
            return {"sm_mhz": None, "sm_max_mhz": self.max_mhz, "reasons": [], "samples": 0, "samples_timed": 0}
        mhz = [s[0] for s in self.samples]
        bits = 0
        for _, r, _ in self.samples:
            bits |= r
        reasons = [name for b, name in self.REASONS.items() if bits & b and name != "gpu_idle"]
        timed = [s for s in self.samples
                 if self.t_start is not None and self.t_end is not None and self.t_start <= s[2] <= self.t_end]
        out = {"sm_mhz": float(statistics.median(mhz)), "sm_max_mhz": self.max_mhz, "reasons": reasons,
               "samples": len(mhz), "samples_timed": len(timed),
               "window": "pre-warm replays (0.3 s) immediately before the timed region, and the timed region"}
        if timed:
            out["sm_mhz_timed"] = float(statistics.median([t[0] for t in timed]))
        return out


def dist_init():
    world = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    if world > 1:
        import datetime

        import torch.distributed as dist
        backend = os.environ.get("S12_BENCH_BACKEND", "nccl")
        dist.init_process_group(backend=backend, timeout=datetime.timedelta(seconds=120))
    return world, rank, local


def barrier(world):
    if world > 1:
        import torch.distributed as dist
        dist.barrier()


def max_over_ranks(value: float, world: int) -> float:
    if world == 1:
        return value
    import torch
    import torch.distributed as dist
    dev = "cuda" if dist.get_backend() == "nccl" else "cpu"
    t = torch.tensor([value], dtype=torch.float64, device=dev)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def sum_over_ranks(value: float, world: int) -> float:
    if world == 1:
        return value
    import torch
    import torch.distributed as dist
    dev = "cuda" if dist.get_backend() == "nccl" else "cpu"
    t = torch.tensor([value], dtype=torch.float64, device=dev)
    dist.all_reduce(t, op=dist.ReduceOp.SUM)
    return float(t.item())


def dev16(a: np.ndarray):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint16).view(np.int16)).cuda()


def time_graph(graph, steps: int, world: int, sampler=None):
    """Replays `graph` `steps` times between two events on the current
    stream, bracketed by a barrier and synchronisations; returns seconds
    (max over ranks)."""
    import torch
    start = torch.cuda.Event(enable_timing=True)
    end = torch.cuda.Event(enable_timing=True)
    barrier(world)
    torch.cuda.synchronize()
    ctx = sampler if sampler is not None else _Null()
    with ctx:
        start.record()
        for _ in range(steps):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
    barrier(world)
    sec = start.elapsed_time(end) / 1e3
    return max_over_ranks(sec, world)


class _Null:
    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


def capture(fn):
    import torch
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()  # first run outside capture (sets kernel attributes)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        fn()
    torch.cuda.synchronize()
    return g


def prewarm(graph, seconds: float = 0.3):
    """Untimed replays so clocks are at their working level."""
    import torch
    t0 = time.time()
    while time.time() - t0 < seconds:
        for _ in range(20):
            graph.replay()
        torch.cuda.synchronize()


def load_traffic(kernel: str, workload: str):
    """DRAM bytes per launch recorded from an ncu capture (profiles/), used
    only if the kernel source has not changed since."""
    path = os.path.join(ROOT, "profiles", "traffic.json")
    try:
        with open(path) as f:
            d = json.load(f)
        e = d[kernel][workload]
        import hashlib
        src = os.path.join(ROOT, "decode_split12_b200", "csrc", e["source"])
        h = hashlib.sha256(open(src, "rb").read()).hexdigest()[:16]
        if h != e["source_sha256_16"]:
            return None
        return e
    except Exception:
        return None


# --------------------------------------------------------------------------- llama8b (default)

class Llama8bLayer:
    def __init__(self, batch: int, seed: int = 0, need_bf16: bool = True):
        import torch

        from decode_split12_b200 import s12
        self.s12 = s12
        self.batch = batch
        mats, xs = wl.llama8b_layer(seed, batch)
        self.names = list(wl.LLAMA8B_SHAPES)
        self.weights = sum(r * c for r, c in wl.LLAMA8B_SHAPES.values())
        self.containers, self.views, self.x, self.y = {}, {}, {}, {}
        self.host_blobs = {}
        self.w_dev = {}
        self.x_host = {}
        for n in self.names:
            wd = dev16(mats[n])
            blob = s12.s12_encode(wd)
            self.containers[n] = blob
            self.views[n] = s12.s12_open(blob)
            if need_bf16:
                self.w_dev[n] = wd
            else:
                del wd
            self.x[n] = dev16(xs[n])
            self.x_host[n] = xs[n]
            self.y[n] = torch.empty((batch, mats[n].shape[0]), dtype=torch.float32, device="cuda")
        self.mats = mats
        # one zero-filled GEMV workspace, large enough for every matrix; the
        # calls run one after another on one stream and leave it zeroed
        self.ws = torch.zeros(s12.s12_gemv_multi_ws_bytes([self.views[n] for n in self.names], 8),
                              dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        self.compressed = sum(int(v.container_bytes) for v in self.views.values())
        self.read_bytes = sum(self._alg_bytes(n) for n in self.names)

    def _alg_bytes(self, n):
        v = self.views[n]
        r, c = int(v.rows), int(v.cols)
        # every plane is read once (payload, per-tile base + offsets, escapes),
        # x is read, y is written
        return (r * c * 3 // 2 + int(v.n_tiles) * 5 + 4 + 2 * int(v.n_esc) + self.batch * c * 2 +
                self.batch * r * 4)

    def set_batch_x(self, batch, seed=0):
        import torch
        self.batch = batch
        for i, n in enumerate(self.names):
            c = wl.LLAMA8B_SHAPES[n][1]
            xs = wl.activations(batch, c, seed, 1000 + i)
            self.x[n] = dev16(xs)
            self.x_host[n] = xs
            self.y[n] = torch.empty((batch, wl.LLAMA8B_SHAPES[n][0]), dtype=torch.float32, device="cuda")
        self.read_bytes = sum(self._alg_bytes(n) for n in self.names)

    def step(self):
        """One grouped launch: all seven independent GEMVs of the layer."""
        self._multi(self.names)

    def _multi(self, names):
        self.s12.s12_gemv_multi([self.views[n] for n in names], [self.x[n] for n in names],
                                [self.y[n] for n in names], ws=self.ws)

    def step_dependency_groups(self):
        """Four launches, grouped as a decoder layer's data flow allows:
        {q, k, v} share an input, o follows attention, {gate, up} share an
        input, down follows the activation."""
        for grp in (("q", "k", "v"), ("o",), ("gate", "up"), ("down",)):
            self._multi(grp)

    def step_separate(self):
        """Seven launches, one s12_gemv per matrix."""
        for n in self.names:
            self.s12.s12_gemv(self.views[n], self.x[n], self.y[n], ws=self.ws)

    def step_bf16_own(self):
        for n in self.names:
            self.s12.s12_bf16_gemv(self.w_dev[n], self.x[n], self.y[n])

    def step_bf16_torch(self):
        import torch
        for n in self.names:
            torch.nn.functional.linear(self.x[n].view(torch.bfloat16), self.w_dev[n].view(torch.bfloat16))


def e2e_llama(layer: Llama8bLayer, steps: int, warmup: int, world: int):
    """Same metric through the public API with host buffers.  The seven
    inputs sit in one pinned host buffer and the seven outputs in one device
    buffer (each matrix's x and y are views into them, 16-byte aligned).
    Every step copies its x from pinned host memory, runs one s12_gemv_multi
    over the seven matrices and copies its y back to pinned host memory.
    The copies run on a second stream, double-buffered, so a step's input
    copy and the previous step's output copy overlap the GEMV between them
    (a graph holds two steps; its end waits for the last output copy)."""
    import torch

    from decode_split12_b200 import s12
    names = layer.names
    xs = [layer.x[n] for n in names]
    ys = [layer.y[n] for n in names]
    xh = torch.cat([torch.from_numpy(layer.x_host[n].view(np.int16)).reshape(-1) for n in names]).pin_memory()
    xd = [torch.empty_like(xh, device="cuda") for _ in range(2)]
    n_y = sum(y.numel() for y in ys)
    yd = [torch.empty(n_y, dtype=torch.float32, device="cuda") for _ in range(2)]
    yh = [torch.empty(n_y, dtype=torch.float32).pin_memory() for _ in range(2)]
    xv, yv = [[], []], [[], []]
    for k in range(2):
        ox = oy = 0
        for x, y in zip(xs, ys):
            xv[k].append(xd[k][ox:ox + x.numel()].view(x.shape))
            yv[k].append(yd[k][oy:oy + y.numel()].view(y.shape))
            ox += x.numel()
            oy += y.numel()
    views = [layer.views[n] for n in names]
    h2d = xh.numel() * 2
    d2h = n_y * 4
    s_copy = torch.cuda.Stream()
    ev_x1 = torch.cuda.Event()

    def two_steps():
        main = torch.cuda.current_stream()
        s_copy.wait_stream(main)
        with torch.cuda.stream(s_copy):
            xd[1].copy_(xh, non_blocking=True)          # step 1's input, during step 0
            ev_x1.record()
        s12.s12_gemv_multi(views, xv[0], yv[0], ws=layer.ws)
        s_copy.wait_stream(main)
        with torch.cuda.stream(s_copy):
            yh[0].copy_(yd[0], non_blocking=True)       # step 0's result, during step 1
            xd[0].copy_(xh, non_blocking=True)          # the next step 0's input
        main.wait_event(ev_x1)
        s12.s12_gemv_multi(views, xv[1], yv[1], ws=layer.ws)
        s_copy.wait_stream(main)
        with torch.cuda.stream(s_copy):
            yh[1].copy_(yd[1], non_blocking=True)
        main.wait_stream(s_copy)

    xd[0].copy_(xh)
    g = capture(two_steps)
    for _ in range(max(warmup, 3)):
        g.replay()
    torch.cuda.synchronize()
    pairs = max(1, steps // 2)
    sec = time_graph(g, pairs, world)
    # the copies carried the real results: both host outputs equal the
    # device step's y (same inputs, a deterministic kernel)
    ref = [torch.empty_like(y) for y in ys]
    s12.s12_gemv_multi(views, xs, ref, ws=layer.ws)
    dev_y = torch.cat([y.reshape(-1) for y in ref]).cpu()
    e2e_llama.matches = bool(torch.equal(yh[0], dev_y) and torch.equal(yh[1], dev_y))
    return sec / (2 * pairs), h2d, d2h, g


def cpu_baseline_llama(target_s: float = 12.0):
    """The oracle as it stands (single-threaded C, FP64) on a bounded sample:
    a fraction of the rows of each of the seven matrices, B = 1, scaled so the
    timed oracle work takes about `target_s` seconds (whole passes over the
    layer when one pass is shorter).  Only the GEMV calls are timed; the
    oracle's encoding of the sample is not."""
    from oracle.oracle import Oracle
    orc = Oracle()
    mats, xs = wl.llama8b_layer(0, 1)
    g = wl.rng_for(99, 0)

    def sample(frac):
        blobs, weights = {}, 0
        for n in wl.LLAMA8B_SHAPES:
            r, c = wl.LLAMA8B_SHAPES[n]
            k = max(1, int(round(frac * r)))
            rows = np.sort(g.choice(r, k, replace=False)) if k < r else np.arange(r)
            blobs[n] = orc.encode(mats[n][rows])
            weights += k * c
        return blobs, weights

    def timed(blobs):
        t0 = time.perf_counter()
        for n, b in blobs.items():
            orc.gemv_f64(b, xs[n])
        return time.perf_counter() - t0

    b1, w1 = sample(0.002)
    s1 = timed(b1)
    frac = min(1.0, 0.002 * target_s / max(s1, 1e-6))
    blobs, w_pass = sample(frac)
    secs, passes = timed(blobs), 1
    while secs < 0.75 * target_s and passes < 30:
        secs += timed(blobs)
        passes += 1
    weights = w_pass * passes
    return {"value": round(2 * weights / secs / 1e9, 4), "unit": "GB/s", "cores": 1, "kind": "oracle",
            "sample": f"{frac * 100:.2f}% of the rows of each of the 7 matrices, {passes} pass(es) "
                      f"(decode + FP64 GEMV, B=1): {weights} weights in {secs:.1f} s on 1 of {os.cpu_count()} "
                      f"host cores"}


def llama_config(batch: int, world: int = 1) -> dict:
    """The workload both arms (library and oracle) report, identically."""
    return {"workload": f"llama8b-layer decode GEMV, B={batch}: q,o 4096x4096; k,v 1024x4096; "
                        f"gate,up 14336x4096; down 4096x14336 (Student-t(5)/sqrt(in), Split12)",
            "batch": batch,
            "weights_per_step": sum(r * c for r, c in wl.LLAMA8B_SHAPES.values()),
            "grouping": "the seven independent GEMVs of the layer in one s12_gemv_multi launch",
            "l2": "inputs larger than L2: about 336 MB of containers per step vs 126 MiB L2",
            "parallelism": "replicas" if world > 1 else "single GPU"}


def single_c1(world, steps: int = 200):
    """The 4096 x 4096 single tensor (N(0, 0.02), 0.1 % outliers x U(10, 100)),
    B = 1.  The container (25.8 MB) fits in L2, so the timed loop walks a ring
    of distinct encoded copies totalling more than 3x the L2 size; one call =
    one GEMV.  The same ring for the BF16 baselines."""
    import torch

    from decode_split12_b200 import s12
    hbm, _, _, _ = load_peaks()
    w, x = wl.single_tensor(0)
    wd = dev16(w)
    blob0 = s12.s12_encode(wd)
    n_copies = max(2, math.ceil(3 * L2_BYTES_B200 / blob0.numel()))
    blobs = [blob0] + [blob0.clone() for _ in range(n_copies - 1)]
    views = [s12.s12_open(b) for b in blobs]
    xd = dev16(x)
    y = torch.empty((1, w.shape[0]), dtype=torch.float32, device="cuda")
    v0 = views[0]
    alg = int(v0.rows * v0.cols * 3 // 2 + v0.n_tiles * 5 + 4 + 2 * v0.n_esc + v0.cols * 2 + v0.rows * 4)
    ws = s12.gemv_workspace(v0)
    g = capture(lambda: [s12.s12_gemv(v, xd, y, ws=ws) for v in views])
    for _ in range(3):
        g.replay()
    passes = max(2, steps // n_copies)
    t = time_graph(g, passes, world) / (passes * n_copies)
    out = {"us": round(t * 1e6, 3), "effective_bf16_GBs": round(2 * w.size / t / 1e9, 1),
           "hbm_frac": round(alg / t / 1e9 / hbm, 4), "algorithmic_bytes": alg,
           "container_bytes": int(v0.container_bytes), "n_esc": int(v0.n_esc),
           "l2": f"ring of {n_copies} distinct containers ({n_copies * blob0.numel() / 1e6:.0f} MB), > 3x L2"}
    del g
    wb = [wd] + [wd.clone() for _ in range(max(2, math.ceil(3 * L2_BYTES_B200 / (wd.numel() * 2))) - 1)]
    for name, fn in (("bf16_own_gemv_us", lambda: [s12.s12_bf16_gemv(m, xd, y) for m in wb]),
                     ("cublas_bf16_us", lambda: [torch.nn.functional.linear(xd.view(torch.bfloat16),
                                                                            m.view(torch.bfloat16)) for m in wb])):
        gb = capture(fn)
        for _ in range(3):
            gb.replay()
        nb = max(2, passes)
        out[name] = round(time_graph(gb, nb, world) / (nb * len(wb)) * 1e6, 3)
        del gb
    del blobs, views, wb
    torch.cuda.empty_cache()
    return out


def v2_layer(layer, world, steps: int):
    """The same layer as container version 2 (compact tile header: one u16 of
    base | escape count per tile, one u32 escape offset per row), converted
    on the host from the version 1 containers, in the same grouped launch."""
    import torch

    from decode_split12_b200 import s12
    hbm, _, _, _ = load_peaks()
    blobs = [torch.from_numpy(s12.to_v2_host(layer.containers[n])).cuda() for n in layer.names]
    views = [s12.s12_open(b) for b in blobs]
    xs = [layer.x[n] for n in layer.names]
    ys = [layer.y[n] for n in layer.names]
    g = capture(lambda: s12.s12_gemv_multi(views, xs, ys, ws=layer.ws))
    for _ in range(3):
        g.replay()
    t = time_graph(g, steps, world) / steps
    alg = sum(int(v.rows * v.cols * 3 // 2) + 2 * int(v.n_tiles) + 4 * (int(v.rows) + 1) + 2 * int(v.n_esc) +
              layer.batch * int(v.cols) * 2 + layer.batch * int(v.rows) * 4 for v in views)
    cbytes = sum(int(v.container_bytes) for v in views)
    del g, blobs, views
    torch.cuda.empty_cache()
    return {"us": round(t * 1e6, 2), "effective_bf16_GBs": round(2 * layer.weights / t / 1e9, 1),
            "hbm_frac": round(alg / t / 1e9 / hbm, 4), "algorithmic_bytes": alg, "container_bytes": cbytes,
            "container_bytes_v1": layer.compressed}


def encode_llama(layer, world):
    """The encoder (s12_encode: tile windows and escape counts, one
    synchronisation, packing; one library call per matrix) on the seven
    matrices of the layer, timed with CUDA events around each whole call.  Algorithmic bytes: read the BF16 matrix once (2 B/weight), write
    the container (1.5 B/weight + 5 B/tile + 2 B/escape + the header)."""
    import torch

    from decode_split12_b200 import s12
    hbm, _, _, _ = load_peaks()
    total_t, total_b, weights = 0.0, 0, 0
    ws = torch.empty(max(s12.lib().s12_encode_ws_bytes(*wl.LLAMA8B_SHAPES[n]) for n in layer.names),
                     dtype=torch.uint8, device="cuda")
    for n in layer.names:
        wd = layer.w_dev[n]
        s12.s12_encode(wd, ws=ws)  # warm
        torch.cuda.synchronize()
        best = None
        for _ in range(3):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            blob = s12.s12_encode(wd, ws=ws)
            e1.record()
            torch.cuda.synchronize()
            t = e0.elapsed_time(e1) / 1e3
            best = t if best is None else min(best, t)
        total_t += best
        total_b += wd.numel() * 2 + blob.numel()
        weights += wd.numel()
        del blob
    return {"ms_layer": round(total_t * 1e3, 3), "GBs": round(total_b / total_t / 1e9, 1),
            "hbm_frac": round(total_b / total_t / 1e9 / hbm, 4), "weights": weights,
            "timing": "CUDA events around each whole s12_encode call (windows and counts, host sync, "
                      "packing), best of 3 per matrix"}


def int8_layer(layer, world, steps: int, fused_us: float):
    """The same seven matrices in 8 bits (s12_quant_i8 once, a scale per row),
    the lossy form that lossless 12 bits are compared with: each x quantised
    and multiplied by s12_gemm_i8, fourteen launches, against the fused GEMV
    as seven.  The error is that of y against the fused GEMV's y, relative in
    the root mean square over the layer."""
    import torch

    from decode_split12_b200 import s12
    ws = s12.gemm_i8_workspace(layer.batch, device="cuda")
    w = {n: s12.s12_quant_i8(layer.w_dev[n].view(torch.bfloat16)) for n in layer.names}
    x = {n: layer.x[n].view(torch.bfloat16).reshape(layer.batch, -1) for n in layer.names}
    xq = {n: s12.s12_quant_i8(x[n]) for n in layer.names}
    y = {n: torch.empty_like(layer.y[n]) for n in layer.names}

    def step():
        for n in layer.names:
            s12.s12_quant_i8(x[n], *xq[n])
            s12.s12_gemm_i8(*xq[n], *w[n], y[n], ws)

    g = capture(step)
    for _ in range(3):
        g.replay()
    t = time_graph(g, steps, world) / steps
    layer.step_separate()
    torch.cuda.synchronize()
    off = sum(float((y[n] - layer.y[n]).double().square().sum()) for n in layer.names)
    size = sum(float(layer.y[n].double().square().sum()) for n in layer.names)
    del g
    return {"us_14_launches": round(t * 1e6, 2), "fused_us_7_launches": fused_us,
            "weight_bytes": sum(q.numel() + 4 * c.numel() for q, c in w.values()),
            "container_bytes": layer.compressed, "rel_rms_error_vs_fused": round(math.sqrt(off / size), 6)}


def run_llama8b(args, world, rank):
    import torch
    hbm, _, _, peak_kind = load_peaks()
    layer = Llama8bLayer(args.batch)
    g = capture(layer.step)
    for _ in range(max(args.warmup, 3)):
        g.replay()
    torch.cuda.synchronize()
    sampler = ClockSampler(torch.cuda.current_device())
    with sampler:
        prewarm(g)  # untimed replays so the clocks are at their working level
        sampler.mark_start()
        sec = time_graph(g, args.steps, world)
        sampler.mark_end()
    ms = sec / args.steps * 1e3
    t_step = sec / args.steps
    value_rank = 2 * layer.weights / t_step / 1e9
    value = value_rank * world  # all ranks processed the same amount; time is the max
    achieved = layer.read_bytes / t_step / 1e9
    extra = {}
    # batch 4 and 8 on the same containers
    for b in (4, 8):
        if b == args.batch:
            continue
        layer.set_batch_x(b)
        gb = capture(layer.step)
        for _ in range(3):
            gb.replay()
        sb = time_graph(gb, max(20, args.steps // 4), world) / max(20, args.steps // 4)
        extra[f"B{b}"] = {"us_per_layer": round(sb * 1e6, 2), "effective_bf16_GBs": round(2 * layer.weights / sb / 1e9, 1),
                          "hbm_frac": round(layer.read_bytes / sb / 1e9 / hbm, 4)}
        del gb
    layer.set_batch_x(args.batch)
    # the same seven GEMVs in fewer-fused launch patterns
    for name, fn, nl in (("dependency_groups_4_launches", layer.step_dependency_groups, 4),
                         ("separate_7_launches", layer.step_separate, 7)):
        gb = capture(fn)
        for _ in range(3):
            gb.replay()
        nb = max(20, args.steps // 2)
        sb = time_graph(gb, nb, world) / nb
        extra[name] = {"us_per_layer": round(sb * 1e6, 2), "effective_bf16_GBs": round(2 * layer.weights / sb / 1e9, 1),
                       "hbm_frac": round(layer.read_bytes / sb / 1e9 / hbm, 4), "launches": nl}
        del gb
    # uncompressed BF16 baselines at the same batch: own kernel and cuBLAS
    for name, fn in (("bf16_own_gemv", layer.step_bf16_own), ("bf16_torch_linear", layer.step_bf16_torch)):
        gb = capture(fn)
        for _ in range(3):
            gb.replay()
        nb = max(20, args.steps // 2)
        sb = time_graph(gb, nb, world) / nb
        extra[name] = {"us_per_layer": round(sb * 1e6, 2), "GBs": round(2 * layer.weights / sb / 1e9, 1),
                       "hbm_frac": round(2 * layer.weights / sb / 1e9 / hbm, 4)}
        del gb
    comparisons = {}
    if layer.w_dev:
        extra["mlp_swiglu_epilogue"] = mlp_swiglu_extras(layer, world, max(20, args.steps // 4))
        fast_bf16 = min(extra["bf16_own_gemv"]["us_per_layer"], extra["bf16_torch_linear"]["us_per_layer"])
        comparisons["bf16_gemv_same_layer"] = {
            "fused_us": round(ms * 1e3, 2), "bf16_own_gemv_us": extra["bf16_own_gemv"]["us_per_layer"],
            "cublas_bf16_us": extra["bf16_torch_linear"]["us_per_layer"],
            "fused_speedup_vs_faster_bf16": round(fast_bf16 / (ms * 1e3), 4)}
        comparisons["int8_same_layer"] = int8_layer(layer, world, max(20, args.steps // 2),
                                                    extra["separate_7_launches"]["us_per_layer"])
        comparisons["encode_llama8b_layer"] = encode_llama(layer, world)
    comparisons["container_v2_same_layer"] = v2_layer(layer, world, max(20, args.steps // 2))
    comparisons["single_4096_b1"] = single_c1(world)
    e2e_t, h2d, d2h, ge = e2e_llama(layer, max(20, args.steps // 2), args.warmup, world)
    if not args.no_gemm:
        del layer.w_dev
        torch.cuda.empty_cache()
        extra["gemm_70b_mlp_tcgen05"] = gemm_extras(world)
    if not args.no_decode:
        extra["decode_escape_stress"] = decode_extras(world)
    if not args.no_stack:
        extra["whole_stack"] = stack_extras(world)
    del ge
    traffic = load_traffic("gemv_kernel", f"llama8b_b{args.batch}")
    out = {
        "metric": METRIC,
        "value": round(value, 2),
        "unit": "GB/s",
        "n_gpus": world,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32",
        "data": "synthetic",
        "config": llama_config(args.batch, world),
        "roofline": {
            "bound": "hbm",
            "achieved": round(achieved, 1),
            "peak": hbm,
            "unit": "GB/s",
            "frac": round(achieved / hbm, 4),
            "traffic": (traffic or {}).get("dram_bytes_per_step"),
            "peak_kind": peak_kind,
            "kernel": "gemv_kernel",
            "algorithmic_bytes_per_launch": layer.read_bytes,
            "compressed_bytes_per_step": layer.compressed,
            "launches_per_step": 1,
            # measured in the same run, on the same GPU
            "comparisons": comparisons,
        },
        "clocks": sampler.summary(),
        "e2e": {"value": round(2 * layer.weights / e2e_t / 1e9 * world, 2), "unit": "GB/s",
                "h2d_bytes_per_step": h2d, "d2h_bytes_per_step": d2h,
                "copies": "pinned host buffers, on a second stream, double-buffered: a step's input "
                          "and the previous step's output copy overlap the GEMV",
                "host_result_equals_device_step": getattr(e2e_llama, "matches", None)},
        "gpu_launches": args.steps,
        "extra": extra,
    }
    if rank == 0 and world == 1 and not args.no_cpu_baseline:
        out["cpu_baseline"] = cpu_baseline_llama()
    return out


def gemm_extras(world, steps: int = 40):
    """The 70B-style MLP decode-phase skinny GEMM: W 28672x8192 and
    8192x28672 (N(0, 1/sqrt(in)) with 0.05 % outliers x U(10, 100)), X bf16
    N(0, 1) at M = 16..256, on the tcgen05 fused decode-GEMM, next to cuBLAS
    (torch.matmul) on the uncompressed BF16 weights.  Each container (361 MB)
    is larger than L2, so back-to-back calls stream it from HBM."""
    import torch

    from decode_split12_b200 import s12
    hbm, tf_burst, tf_sust, _ = load_peaks()
    out = {}
    for name in wl.MLP70B_SHAPES:
        w = wl.mlp70b(name, 0)
        wd = dev16(w)
        del w
        blob = s12.s12_encode(wd)
        view = s12.s12_open(blob)
        n, k = int(view.rows), int(view.cols)
        cbytes = int(view.container_bytes)
        res = {}
        for m in (16, 32, 64, 128, 256):
            x = dev16(wl.activations(m, k, m))
            y = torch.empty((m, n), dtype=torch.float32, device="cuda")
            ws = torch.zeros(s12.s12_gemm_ws_bytes(view, m), dtype=torch.uint8, device="cuda")
            g = capture(lambda: s12.s12_gemm_skinny(view, x, y, ws=ws))
            for _ in range(3):
                g.replay()
            t = time_graph(g, steps, world) / steps
            gb = capture(lambda: torch.matmul(x.view(torch.bfloat16), wd.view(torch.bfloat16).t()))
            for _ in range(3):
                gb.replay()
            tb = time_graph(gb, steps, world) / steps
            alg = n * k * 3 // 2 + (n * k // 128) * 5 + 2 * int(view.n_esc) + m * k * 2 + m * n * 4
            flops = 2.0 * m * n * k
            res[f"M{m}"] = {"us": round(t * 1e6, 2), "hbm_GBs": round(alg / t / 1e9, 1),
                            "hbm_frac": round(alg / t / 1e9 / hbm, 4), "TFLOPs": round(flops / t / 1e12, 1),
                            "tensor_frac_sustained": round(flops / t / 1e12 / tf_sust, 4),
                            "cublas_bf16_us": round(tb * 1e6, 2)}
            del g, gb
        out[f"{name}_{n}x{k}"] = {"container_bytes": cbytes, **res}
        del wd, blob
        torch.cuda.empty_cache()
    return out


def decode_extras(world, steps: int = 30):
    """Standalone decode on the escape-rate stress tensors (8192 x 8192,
    exactly 0.03 %, 0.23 %, 2 % and 10 % escapes at uniform positions):
    throughput and a bit-exact check of the whole output against the source
    tensor on the device."""
    import torch

    from decode_split12_b200 import s12
    hbm, _, _, _ = load_peaks()
    out = {}
    for rate in wl.ESCAPE_RATES:
        w, n_planted = wl.escape_stress(rate, 0)
        wd = dev16(w)
        del w
        blob = s12.s12_encode(wd)
        view = s12.s12_open(blob)
        dst = torch.empty_like(wd)
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        g = capture(lambda: s12.s12_decode(view, dst, err_flag=flag))
        for _ in range(3):
            g.replay()
        t = time_graph(g, steps, world) / steps
        exact = bool(torch.equal(dst, wd)) and int(flag.item()) == 0
        n, nt = int(view.rows * view.cols), int(view.n_tiles)
        alg = n * 3 // 2 + nt * 5 + 4 + 2 * int(view.n_esc) + 2 * n
        out[f"{rate * 100:g}%"] = {"n_esc": int(view.n_esc), "planted": n_planted, "bit_exact": exact,
                                   "us": round(t * 1e6, 2), "hbm_GBs": round(alg / t / 1e9, 1),
                                   "hbm_frac": round(alg / t / 1e9 / hbm, 4),
                                   "bf16_out_GBs": round(2 * n / t / 1e9, 1)}
        del g, wd, blob, dst
        torch.cuda.empty_cache()
    return out


def _student_t_gpu(rows: int, cols: int, gen):
    """Student-t(5) scaled to std 1/sqrt(cols), drawn on the device: t = z /
    sqrt(chi2_5 / 5) with chi2_5 = 2 * Gamma(2.5); rounded to BF16."""
    import torch
    z = torch.randn(rows, cols, generator=gen, device="cuda")
    gam = torch._standard_gamma(torch.full((rows, cols), 2.5, device="cuda"), generator=gen)
    t = z / torch.sqrt(2.0 * gam / 5.0)
    del z, gam
    return (t * (1.0 / math.sqrt(5.0 / 3.0) / math.sqrt(cols))).to(torch.bfloat16).view(torch.int16)


def mlp_swiglu_extras(layer, world, steps: int):
    """The layer's MLP at its batch: h = silu(gate x) * (up x), then down h.
    Fused: one s12_gemv_swiglu over the interleaved gate/up container (h
    written once, as BF16) and one s12_gemv for down.  Unfused: the gate and
    up GEMVs in one grouped launch (FP32 outputs), torch's silu, multiply and
    BF16 cast, then the down GEMV."""
    import torch

    from decode_split12_b200 import s12
    hbm, _, _, _ = load_peaks()
    B = layer.x["gate"].shape[0]
    wi = s12.interleave_gate_up(layer.w_dev["gate"], layer.w_dev["up"])
    blob = s12.s12_encode(wi)
    del wi
    gu = s12.s12_open(blob)
    F = layer.views["gate"].rows
    h = torch.empty((B, F), dtype=torch.int16, device="cuda")
    yd = torch.empty((B, layer.views["down"].rows), dtype=torch.float32, device="cuda")
    xg = layer.x["gate"]
    yg = torch.empty((B, F), dtype=torch.float32, device="cuda")
    yu = torch.empty((B, F), dtype=torch.float32, device="cuda")

    def fused():
        s12.s12_gemv_swiglu(gu, xg, h, ws=layer.ws)
        s12.s12_gemv(layer.views["down"], h, yd, ws=layer.ws)

    def unfused():
        s12.s12_gemv_multi([layer.views["gate"], layer.views["up"]], [xg, xg], [yg, yu], ws=layer.ws)
        hh = (torch.nn.functional.silu(yg) * yu).to(torch.bfloat16).view(torch.int16)
        s12.s12_gemv(layer.views["down"], hh, yd, ws=layer.ws)

    out = {"batch": B}
    cbytes = int(gu.container_bytes) + int(layer.views["down"].container_bytes)
    for name, fn in (("fused", fused), ("unfused", unfused)):
        g = capture(fn)
        for _ in range(3):
            g.replay()
        t = time_graph(g, steps, world) / steps
        out[name] = {"us": round(t * 1e6, 2), "hbm_frac": round(cbytes / t / 1e9 / hbm, 4)}
        del g
    del blob, gu
    return out


def stack_extras(world, layers: int = 32, steps: int = 10):
    """Whole-stack weight streaming: `layers` independent 8B-style layers
    (layer l drawn with seed l) resident as Split12 containers (gate and up
    as one interleaved container), one pass = all layers; B = 1 and 8.
    Two forms: one grouped launch per layer over its six containers (pure
    weight streaming), and the activation chain, where the layer's down
    output (BF16) feeds the next layer: per layer q, k, v, o in one grouped
    launch (attention is outside the path: o reads the layer input in its
    place), gate/up with the SwiGLU epilogue, down with a BF16 output, then
    the RMS norm (s12_rmsnorm), so the activations neither vanish nor blow
    up over the layers.
    Plus an 8-expert MoE block (gate, up 14336x4096, down 4096x14336 per
    expert) with top-2 routing of 64 tokens: experts with >= 9 tokens use the
    skinny GEMM (rows padded to 16), the rest the GEMV.  And the same block as
    whole layers (s12_moe: routing, SwiGLU and weighted sum included) for 1, 8
    and 64 tokens."""
    import torch

    from decode_split12_b200 import s12
    hbm, _, _, _ = load_peaks()
    # containers per layer: q, k, v, o, gate/up interleaved, down
    names = ["q", "k", "v", "o", "gate_up", "down"]
    shapes = {n: wl.LLAMA8B_SHAPES[n] for n in ("q", "k", "v", "o", "down")}
    F, Dm = wl.LLAMA8B_SHAPES["gate"]
    shapes["gate_up"] = (2 * F, Dm)
    blobs, views = [], []
    for layer in range(layers):
        gen = torch.Generator(device="cuda").manual_seed(layer)
        lv = []
        for n in names:
            if n == "gate_up":
                wg = _student_t_gpu(F, Dm, gen)
                wu = _student_t_gpu(F, Dm, gen)
                wd = s12.interleave_gate_up(wg, wu)
                del wg, wu
            else:
                wd = _student_t_gpu(*shapes[n], gen)
            b = s12.s12_encode(wd)
            del wd
            blobs.append(b)
            lv.append(s12.s12_open(b))
        views.append(lv)
    torch.cuda.empty_cache()
    weights = layers * sum(r * c for r, c in wl.LLAMA8B_SHAPES.values())
    cbytes = sum(int(v.container_bytes) for lv in views for v in lv)
    ws = torch.zeros(s12.s12_gemv_multi_ws_bytes(views[0], 8), dtype=torch.uint8, device="cuda")
    out = {"layers": layers, "weights": weights, "container_bytes": cbytes}
    for B in (1, 8):
        xs = [dev16(wl.activations(B, shapes[n][1], B, 3000 + i)) for i, n in enumerate(names)]
        ys = [torch.empty((B, shapes[n][0]), dtype=torch.float32, device="cuda") for n in names]

        def step():
            for lv in views:
                s12.s12_gemv_multi(lv, xs, ys, ws=ws)

        g = capture(step)
        for _ in range(3):
            g.replay()
        t = time_graph(g, steps, world) / steps
        out[f"B{B}"] = {"ms_per_pass": round(t * 1e3, 3), "ms_per_token": round(t * 1e3 / B, 3),
                        "effective_bf16_GBs": round(2 * weights / t / 1e9, 1),
                        "hbm_frac": round(cbytes / t / 1e9 / hbm, 4), "launches_per_pass": layers}
        del g
    # the activation chain (each layer's GEMVs depend on the previous layer)
    for B in (1, 8):
        h0 = dev16(wl.activations(B, Dm, B, 5000))
        hs = [h0] + [torch.empty((B, Dm), dtype=torch.int16, device="cuda") for _ in range(layers)]
        hid = torch.empty((B, F), dtype=torch.int16, device="cuda")
        yd = torch.empty((B, Dm), dtype=torch.int16, device="cuda")
        yp = [torch.empty((B, shapes[n][0]), dtype=torch.float32, device="cuda") for n in ("q", "k", "v", "o")]

        def chain():
            for l, lv in enumerate(views):
                h = hs[l]
                s12.s12_gemv_multi(lv[:4], [h] * 4, yp, ws=ws)
                s12.s12_gemv_swiglu(lv[4], h, hid, ws=ws)
                s12.s12_gemv_bf16(lv[5], hid, yd, ws=ws)
                s12.s12_rmsnorm(yd, eps=1e-6, y=hs[l + 1])

        g = capture(chain)
        for _ in range(3):
            g.replay()
        t = time_graph(g, steps, world) / steps
        last = hs[layers].view(torch.bfloat16).float()
        out[f"chain_B{B}"] = {"ms_per_pass": round(t * 1e3, 3), "ms_per_token": round(t * 1e3 / B, 3),
                              "effective_bf16_GBs": round(2 * weights / t / 1e9, 1),
                              "hbm_frac": round(cbytes / t / 1e9 / hbm, 4), "launches_per_pass": 4 * layers,
                              "norm": "s12_rmsnorm after each layer, in the timed graph",
                              "output_finite": bool(torch.isfinite(last).all()),
                              "output_rms": float(last.pow(2).mean().sqrt())}
        del g
    del blobs, views
    torch.cuda.empty_cache()
    # MoE block
    route = wl.moe_routing(64, 8, 2, 0)
    experts = []
    gen = torch.Generator(device="cuda").manual_seed(1000)
    for e in range(8):
        ev = {}
        for n, (r, c) in wl.MOE_SHAPES.items():
            wd = _student_t_gpu(r, c, gen)
            b = s12.s12_encode(wd)
            del wd
            ev[n] = (b, s12.s12_open(b))
        experts.append(ev)
    counts = [int((route == e).any(axis=1).sum()) for e in range(8)]
    calls = []
    for e, m in enumerate(counts):
        if m == 0:
            continue
        for n, (r, c) in wl.MOE_SHAPES.items():
            v = experts[e][n][1]
            if m >= 9:
                mp = max(16, m)
                x = dev16(wl.activations(mp, c, e, 4000 + 10 * e + len(calls)))
                y = torch.empty((mp, r), dtype=torch.float32, device="cuda")
                gws = torch.zeros(s12.s12_gemm_ws_bytes(v, mp), dtype=torch.uint8, device="cuda")
                calls.append(("gemm", v, x, y, gws, n))
            else:
                x = dev16(wl.activations(m, c, e, 4000 + 10 * e + len(calls)))
                y = torch.empty((m, r), dtype=torch.float32, device="cuda")
                gws = torch.zeros(s12.s12_gemv_ws_bytes(v, m), dtype=torch.uint8, device="cuda")
                calls.append(("gemv", v, x, y, gws, n))

    def moe():
        for kind, v, x, y, gws, _ in calls:
            if kind == "gemm":
                s12.s12_gemm_skinny(v, x, y, ws=gws)
            else:
                s12.s12_gemv(v, x, y, ws=gws)

    g = capture(moe)
    for _ in range(3):
        g.replay()
    t = time_graph(g, steps, world) / steps
    moe_bytes = sum(int(experts[e][n][1].container_bytes) for e in range(8) if counts[e] for n in wl.MOE_SHAPES)
    out["moe_8x_top2_64_tokens"] = {"tokens_per_expert": counts, "us": round(t * 1e6, 2),
                                    "us_per_token": round(t * 1e6 / 64, 3),
                                    "hbm_frac": round(moe_bytes / t / 1e9 / hbm, 4),
                                    "calls": [c[0] for c in calls]}
    del g
    # the same block as grouped launches, in the order its data flow allows:
    # every expert's gate and up in one launch, every expert's down in another
    # (experts with fewer than 9 tokens, if any, as grouped GEMVs beside them)
    stages = []
    for names in (("gate", "up"), ("down",)):
        gv, gx, gy, vv, vx, vy = [], [], [], [], [], []
        for kind, v, x, y, _, n in calls:
            if n not in names:
                continue
            if kind == "gemm":
                gv.append(v), gx.append(x), gy.append(y)
            else:
                vv.append(v), vx.append(x), vy.append(y)
        gws = torch.zeros(max(256, s12.s12_gemm_multi_ws_bytes(gv, [x.shape[0] for x in gx])) if gv else 256,
                          dtype=torch.uint8, device="cuda")
        vws = [torch.zeros(max(256, s12.s12_gemv_multi_ws_bytes([v], x.shape[0])), dtype=torch.uint8,
                           device="cuda") for v, x in zip(vv, vx)]
        stages.append((gv, gx, gy, gws, vv, vx, vy, vws))

    def moe_grouped():
        for gv, gx, gy, gws, vv, vx, vy, vws in stages:
            if gv:
                s12.s12_gemm_skinny_multi(gv, gx, gy, ws=gws)
            for v, x, y, w_ in zip(vv, vx, vy, vws):
                s12.s12_gemv(v, x, y, ws=w_)

    g = capture(moe_grouped)
    for _ in range(3):
        g.replay()
    t = time_graph(g, steps, world) / steps
    out["moe_8x_top2_64_tokens_grouped"] = {
        "us": round(t * 1e6, 2), "us_per_token": round(t * 1e6 / 64, 3),
        "hbm_frac": round(moe_bytes / t / 1e9 / hbm, 4),
        "launches": sum((1 if st[0] else 0) + len(st[4]) for st in stages),
        "grouping": "one s12_gemm_skinny_multi over all experts' gate and up, one over all experts' down"}
    del g, experts, calls, stages
    torch.cuda.empty_cache()
    out["moe_layer_8x_top2"] = moe_layer_extras(world, steps)
    return out


def moe_layer_extras(world, steps: int):
    """The 8-expert block as whole layers (s12_moe), gate/up and down of all
    experts stacked in two containers: one launch, for 1, 8 and 64 tokens."""
    import torch

    from decode_split12_b200 import s12
    hbm, _, _, _ = load_peaks()
    E, k = 8, 2
    F, Dm = wl.MOE_SHAPES["gate"]
    gen = torch.Generator(device="cuda").manual_seed(2000)
    gate_up = s12.s12_open(s12.s12_encode(s12.interleave_gate_up(_student_t_gpu(E * F, Dm, gen),
                                                                 _student_t_gpu(E * F, Dm, gen))))
    down = s12.s12_open(s12.s12_encode(_student_t_gpu(E * Dm, F, gen)))
    torch.cuda.empty_cache()
    router = (torch.randn(E, Dm, generator=gen, device="cuda") / math.sqrt(Dm)).to(torch.bfloat16)
    ws = s12.moe_workspace(gate_up, down, E, 64, k)
    out = {}
    for T in (1, 8, 64):
        x = dev16(wl.activations(T, Dm, T, 6000))
        y, ids, weights = s12.s12_moe(gate_up, down, E, x, router, k, ws=ws)
        met = int(ids.unique().numel())
        g = capture(lambda: s12.s12_moe(gate_up, down, E, x, router, k, y=y, ids=ids, weights=weights, ws=ws))
        for _ in range(3):
            g.replay()
        t = time_graph(g, steps, world) / steps
        nbytes = (int(gate_up.container_bytes) + int(down.container_bytes)) * met / E
        out[f"T{T}"] = {"experts_met": met, "us": round(t * 1e6, 2), "hbm_frac": round(nbytes / t / 1e9 / hbm, 4)}
        del g
    return out


def run_reference(args, world, rank):
    """Reference arm: the CPU oracle, as it stands, on the same workload and
    metric; each step is a bounded sample (1 % of the rows of each matrix)."""
    if rank != 0:
        return None
    from oracle.oracle import Oracle
    orc = Oracle()
    mats, xs = wl.llama8b_layer(0, args.batch)
    g = wl.rng_for(98, 0)
    subs = {}
    weights = 0
    for n in wl.LLAMA8B_SHAPES:
        r, c = wl.LLAMA8B_SHAPES[n]
        k = max(1, int(round(0.01 * r)))
        rows = np.sort(g.choice(r, k, replace=False))
        subs[n] = orc.encode(mats[n][rows])
        weights += k * c

    def step():
        for n in subs:
            orc.gemv_f64(subs[n], xs[n])

    for _ in range(args.warmup):
        step()
    t0 = time.perf_counter()
    for _ in range(args.steps):
        step()
    sec = time.perf_counter() - t0
    t_step = sec / args.steps
    value = 2 * weights / t_step / 1e9
    cb = {"value": round(value, 4), "unit": "GB/s", "cores": 1, "kind": "oracle",
          "sample": f"1% of the rows of each of the 7 llama8b-layer matrices per step ({weights} weights), "
                    f"B={args.batch}, decode + FP64 GEMV, 1 of {os.cpu_count()} host cores"}
    return {"metric": METRIC, "value": round(value, 4), "unit": "GB/s", "n_gpus": world, "steps": args.steps,
            "warmup": args.warmup, "ms_per_step": round(t_step * 1e3, 3), "higher_is_better": True,
            "scaling": "weak", "vs_baseline": None, "dtype": "f64", "data": "synthetic",
            "config": llama_config(args.batch, world),
            "impl": "reference", "cpu_baseline": cb,
            "e2e": {"value": round(value, 4), "unit": "GB/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
            "gpu_launches": 0}


# --------------------------------------------------------------------------- single tensor

def run_single(args, world, rank):
    """4096 x 4096 N(0, 0.02) tensor with 0.1 % outliers, B = 1.  The whole
    container (25.8 MB) fits in L2, so the timed loop walks a ring of distinct
    encoded copies totalling more than 3x the L2 size; one step = one GEMV."""
    import torch

    from decode_split12_b200 import s12
    hbm, _, _, peak_kind = load_peaks()
    w, x = wl.single_tensor(0)
    wd = dev16(w)
    blob0 = s12.s12_encode(wd)
    n_copies = max(2, math.ceil(3 * L2_BYTES_B200 / blob0.numel()))
    blobs = [blob0] + [blob0.clone() for _ in range(n_copies - 1)]
    views = [s12.s12_open(b) for b in blobs]
    xd = dev16(x)
    y = torch.empty((1, w.shape[0]), dtype=torch.float32, device="cuda")
    v0 = views[0]
    alg = int(v0.rows * v0.cols * 3 // 2 + v0.n_tiles * 5 + 4 + 2 * v0.n_esc + v0.cols * 2 + v0.rows * 4)

    ws = s12.gemv_workspace(v0)

    def ring():
        for v in views:
            s12.s12_gemv(v, xd, y, ws=ws)

    g = capture(ring)
    for _ in range(max(args.warmup, 3)):
        g.replay()
    torch.cuda.synchronize()
    passes = max(1, args.steps // n_copies)
    if passes * n_copies >= 50:
        prewarm(g)
    sampler = ClockSampler(torch.cuda.current_device())
    sec = time_graph(g, passes, world, sampler)
    steps = passes * n_copies
    t = sec / steps
    extra = {}
    wb = [wd] + [wd.clone() for _ in range(max(2, math.ceil(3 * L2_BYTES_B200 / (wd.numel() * 2))) - 1)]
    for name, fn in (("bf16_own_gemv", lambda: [s12.s12_bf16_gemv(m, xd, y) for m in wb]),
                     ("bf16_torch_linear", lambda: [torch.nn.functional.linear(xd.view(torch.bfloat16),
                                                                               m.view(torch.bfloat16)) for m in wb])):
        gb = capture(fn)
        for _ in range(3):
            gb.replay()
        nb = max(2, passes)
        sb = time_graph(gb, nb, world) / (nb * len(wb))
        extra[name] = {"us": round(sb * 1e6, 3), "GBs": round(2 * w.size / sb / 1e9, 1)}
        del gb
    return {
        "metric": METRIC, "value": round(2 * w.size / t / 1e9 * world, 2), "unit": "GB/s", "n_gpus": world,
        "steps": steps, "warmup": args.warmup, "ms_per_step": round(t * 1e3, 5), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "f32", "data": "synthetic",
        "config": {"workload": "single 4096x4096 N(0,0.02) + 0.1% outliers x U(10,100), GEMV B=1",
                   "batch": 1, "container_bytes": int(v0.container_bytes), "n_esc": int(v0.n_esc),
                   "l2": f"ring of {n_copies} distinct containers ({n_copies * blob0.numel() / 1e6:.0f} MB) "
                         f"walked in order, > 3x L2"},
        "roofline": {"bound": "hbm", "achieved": round(alg / t / 1e9, 1), "peak": hbm, "unit": "GB/s",
                     "frac": round(alg / t / 1e9 / hbm, 4), "traffic": None, "peak_kind": peak_kind,
                     "kernel": "gemv_kernel"},
        "clocks": sampler.summary(),
        "gpu_launches": steps,
        "extra": extra,
    }


# --------------------------------------------------------------------------- main

def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=2000)
    ap.add_argument("--warmup", type=int, default=20)
    ap.add_argument("--impl", choices=["split12", "reference"], default="split12")
    ap.add_argument("--workload", choices=["llama8b", "single"], default="llama8b")
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-gemm", action="store_true", help="skip the skinny-GEMM extras")
    ap.add_argument("--no-decode", action="store_true", help="skip the standalone-decode extras")
    ap.add_argument("--no-stack", action="store_true", help="skip the whole-stack extras")
    args = ap.parse_args(argv)
    if args.warmup < 3:
        args.warmup = 3
    world, rank, local = dist_init()
    if args.impl == "reference":
        out = run_reference(args, world, rank)
        if out is not None:
            print(json.dumps(out), flush=True)
        return 0
    import torch
    torch.cuda.set_device(local)
    from decode_split12_b200 import s12
    s12.device_check()
    out = run_single(args, world, rank) if args.workload == "single" else run_llama8b(args, world, rank)
    if rank == 0:
        print(json.dumps(out), flush=True)
    if world > 1:
        import torch.distributed as dist
        dist.destroy_process_group()
    return 0


if __name__ == "__main__":
    sys.exit(main())
