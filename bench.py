#!/usr/bin/env python
"""Benchmark of the BitLinear W1.58A8 hot path on GB300.

Headline workload (BitNet-3B decode, M = 1 token): one step is the FFN's three
BitLinear calls of one token, exactly as a decode step runs them:
    act_quant(x [1, 2560])                     (shared by gate and up)
    g = forward(gate 2560 -> 10240), u = forward(up 2560 -> 10240)
    act_quant(h = ReLU^2(g) * u [1, 10240])
    forward(down 10240 -> 2560)
i.e. 19,660,800 packed weight bytes per step.  Inputs are seeded synthetic
tensors (weights ~ N(0, 0.02), activations ~ N(0, 1) with 1% of channels x20).
Each step uses the next of R copies of the packed weights (R * 19.7 MB > 4x
L2), so every weight byte comes from HBM.  Steps run as CUDA graphs with
programmatic dependent launch between kernels.  By default a step is two
bitlinear_linear calls (act_quant fused into the decode kernel; gate and up in
one launch whose epilogue writes h); --separate times the five separate
act_quant / forward calls.  The oracle arms (CPU baseline, --impl reference)
quantise a synthetic [1, 10240] row pair with the same gating prologue for the
down call: the oracle's work does not depend on the values, and a step split
over host cores by output rows cannot chain the full h.

Metric: packed-weight GB/s (1e9 B/s) over the whole job.  One JSON line on
rank 0.  `--impl reference` times the CPU oracle on the same workload instead.
Multi-GPU (torchrun): independent replicas, one per GPU (weak scaling).
"""
from __future__ import annotations

import argparse
import hashlib
import json
import os
import statistics
import subprocess
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

METRIC = "W1.58A8 BitLinear: packed-weight GB/s at M=1 (%HBM peak); int8 TOPS at M=2048"
UNIT = "GB/s"
WORKLOAD = "bitnet3b_ffn_decode_m1"
L2_BYTES = 129 * 1024 * 1024
FALLBACK_HBM_GBS = 6800.0


def parse_args():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=200000)
    ap.add_argument("--warmup", type=int, default=2000)
    ap.add_argument("--impl", choices=["ours", "reference"], default="ours")
    ap.add_argument("--cpu-seconds", type=float, default=10.0,
                    help="bound of the oracle CPU-baseline sample")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--e2e-steps", type=int, default=2000)
    ap.add_argument("--no-pdl", action="store_true")
    ap.add_argument("--no-prefill", action="store_true", help="skip the M=2048 prefill measurement")
    ap.add_argument("--no-weight-set", action="store_true",
                    help="skip the full BitNet-3B weight-set measurement (M = 1, 8, 32, 64)")
    ap.add_argument("--attention", type=int, default=0, metavar="TOKENS",
                    help="also measure the full weight set's step with every layer attending to so many cached tokens")
    ap.add_argument("--separate", action="store_true",
                    help="time separate act_quant + forward calls instead of bitlinear_linear")
    return ap.parse_args()


# ---------------------------------------------------------------------------
# Workload definition (shapes and seeds of the BitNet-3B decode GEMV)
# ---------------------------------------------------------------------------
def workload_inputs():
    from bitlinear_w1_a8_gb300 import synth
    s = synth.SEEDS["decode"]
    D, F = synth.DIM_3B, synth.FFN_3B
    W_up_shape = synth.weight(F, D, s["W_up_shape"])       # gate and up: 2560 -> 10240
    W_down_shape = synth.weight(D, F, s["W_down_shape"])   # down: 10240 -> 2560
    x_a = synth.activations(1, D, s["x"], outlier_seed=s["outliers"])
    x_b = synth.activations(1, F, s["x"], outlier_seed=s["outliers"])
    u_b = synth.activations(1, F, s["x"] + 1)   # the oracle arms' stand-in for the up output
    return dict(D=D, F=F, W_up_shape=W_up_shape, W_down_shape=W_down_shape, x_a=x_a, x_b=x_b, u_b=u_b)


def step_packed_bytes(D, F):
    return 3 * (D * F // 4)


# ---------------------------------------------------------------------------
# Reference arm and CPU baseline: the oracle, as it stands, on host cores.
# ---------------------------------------------------------------------------
class OracleStep:
    """One decode step computed by the CPU oracle (single-threaded C)."""

    def __init__(self, inp, row_fraction: float = 1.0):
        import oracle
        self.o = oracle
        D, F = inp["D"], inp["F"]
        Wq_u, self.sw_u, _ = oracle.weight_quant(inp["W_up_shape"].numpy())
        Wq_d, self.sw_d, _ = oracle.weight_quant(inp["W_down_shape"].numpy())
        # a step may process a leading fraction of the output rows (bounded sample)
        self.nu = max(1, int(F * row_fraction))
        self.nd = max(1, int(D * row_fraction))
        self.p_u = oracle.pack(Wq_u[: self.nu])
        self.p_d = oracle.pack(Wq_d[: self.nd])
        self.x_a, self.x_b, self.u_b = inp["x_a"].numpy(), inp["x_b"].numpy(), inp["u_b"].numpy()
        self.D, self.F = D, F
        self.bytes = 2 * self.p_u.size + self.p_d.size

    def run(self):
        o = self.o
        xq, sx = o.act_quant(self.x_a)
        o.forward(xq, sx, self.p_u, self.sw_u, self.nu, self.D)   # gate
        o.forward(xq, sx, self.p_u, self.sw_u, self.nu, self.D)   # up
        xq, sx = o.act_quant(self.x_b, mul=self.u_b)           # the gating prologue
        o.forward(xq, sx, self.p_d, self.sw_d, self.nd, self.F)   # down


def host_cores() -> int:
    try:
        return len(os.sched_getaffinity(0))
    except AttributeError:  # pragma: no cover
        return os.cpu_count() or 1


def _oracle_worker(jobs, results):
    """Process of OraclePool: runs oracle decode steps (or a prefill row slice)
    over the row slices it was given, as the parent asks."""
    import oracle
    while True:
        job = jobs.get()
        if job is None:
            return
        kind, payload = job
        t0 = time.perf_counter()
        if kind == "decode":
            x_a, x_b, u_b, parts, steps = payload
            for _ in range(steps):
                xq, sx = oracle.act_quant(x_a)
                for p_u, sw_u, nu, D in parts["up"]:
                    oracle.forward(xq, sx, p_u, sw_u, nu, D)   # gate
                    oracle.forward(xq, sx, p_u, sw_u, nu, D)   # up
                xq, sx = oracle.act_quant(x_b, mul=u_b)
                for p_d, sw_d, nd, F in parts["down"]:
                    oracle.forward(xq, sx, p_d, sw_d, nd, F)
        else:  # "prefill": a slice of output columns for a block of token rows
            xq, sx, p, sw, n, k = payload
            oracle.forward(xq, sx, p, sw, n, k)
        results.put(time.perf_counter() - t0)


class OraclePool:
    """The oracle on every host core: one spawned process per core, each over a
    disjoint slice of the output rows (processes are started with `spawn`, so
    none is forked from a process that has used the GPU)."""

    def __init__(self, inp, row_fraction: float = 1.0, cores: int | None = None):
        import multiprocessing as mp
        import oracle
        self.cores = cores or host_cores()
        D, F = inp["D"], inp["F"]
        Wq_u, sw_u, _ = oracle.weight_quant(inp["W_up_shape"].numpy())
        Wq_d, sw_d, _ = oracle.weight_quant(inp["W_down_shape"].numpy())
        nu = max(1, int(F * row_fraction))
        nd = max(1, int(D * row_fraction))
        self.bytes = 2 * oracle.packed_bytes(nu, D) + oracle.packed_bytes(nd, F)
        self.x_a, self.x_b, self.u_b = inp["x_a"].numpy(), inp["x_b"].numpy(), inp["u_b"].numpy()
        self.parts = []
        for c in range(self.cores):
            u0, u1 = nu * c // self.cores, nu * (c + 1) // self.cores
            d0, d1 = nd * c // self.cores, nd * (c + 1) // self.cores
            self.parts.append({
                "up": [(oracle.pack(Wq_u[u0:u1]), sw_u, u1 - u0, D)] if u1 > u0 else [],
                "down": [(oracle.pack(Wq_d[d0:d1]), sw_d, d1 - d0, F)] if d1 > d0 else []})
        self.row_fraction = row_fraction
        ctx = mp.get_context("spawn")
        self.jobs = [ctx.Queue() for _ in range(self.cores)]
        self.results = ctx.Queue()
        self.procs = [ctx.Process(target=_oracle_worker, args=(self.jobs[c], self.results), daemon=True)
                      for c in range(self.cores)]
        for p in self.procs:
            p.start()
        self.run_decode(1)  # every worker has imported the oracle and touched its slice

    def _gather(self, n, timeout_s: float = 900.0):
        """n results from the workers; raises if a worker died or time ran out."""
        import queue
        out, t_end = [], time.monotonic() + timeout_s
        while len(out) < n:
            try:
                out.append(self.results.get(timeout=1.0))
            except queue.Empty:
                dead = [p.exitcode for p in self.procs if not p.is_alive()]
                if dead or time.monotonic() > t_end:
                    self.close()
                    raise RuntimeError(f"oracle pool: worker exit codes {dead}, "
                                       f"{len(out)} of {n} results")
        return out

    def run_decode(self, steps: int) -> float:
        """Wall seconds for `steps` decode steps over all cores."""
        t0 = time.perf_counter()
        for c in range(self.cores):
            self.jobs[c].put(("decode", (self.x_a, self.x_b, self.u_b, self.parts[c], steps)))
        self._gather(self.cores)
        return time.perf_counter() - t0

    def run_prefill_slice(self, xq, sx, Wq, sw) -> float:
        """Wall seconds for the forward of token rows xq against every row of Wq,
        the output columns split over the cores."""
        import oracle
        N, K = Wq.shape
        jobs = []
        for c in range(self.cores):
            n0, n1 = N * c // self.cores, N * (c + 1) // self.cores
            if n1 > n0:
                jobs.append((c, (xq, sx, oracle.pack(Wq[n0:n1]), sw, n1 - n0, K)))
        t0 = time.perf_counter()
        for c, payload in jobs:
            self.jobs[c].put(("prefill", payload))
        self._gather(len(jobs))
        return time.perf_counter() - t0

    def close(self):
        for q in self.jobs:
            q.put(None)
        for p in self.procs:
            p.join(timeout=10)
            if p.is_alive():
                p.terminate()


def cpu_baseline(inp, seconds: float):
    """The oracle as it stands on the host: every core (the reported value),
    one core beside it, and a 64-token slice of the M = 2048 prefill shapes on
    every core, extrapolated to 2048 tokens."""
    import oracle
    from bitlinear_w1_a8_gb300 import synth
    step = OracleStep(inp)
    n1 = 0
    t0 = time.perf_counter()
    while True:
        step.run()
        n1 += 1
        el1 = time.perf_counter() - t0
        if el1 >= seconds / 2 or n1 >= 10000:
            break
    one_core = step.bytes * n1 / el1 / 1e9
    pool = OraclePool(inp)
    try:
        steps = max(3, int(seconds / 2 * n1 / el1 * pool.cores * 0.8))
        el = pool.run_decode(steps)
        value = step.bytes * steps / el / 1e9
        # prefill: 64 of the 2048 token rows, both FFN shapes, all cores
        s = synth.SEEDS["prefill"]
        D, F = synth.DIM_3B, synth.FFN_3B
        rows, M = 64, 2048
        x = synth.activations(rows, F, s["x"]).numpy()
        pre = {}
        for name, N, K, seed in (("up_shape", F, D, s["W_up_shape"]), ("down_shape", D, F, s["W_down_shape"])):
            Wq, sw, _ = oracle.weight_quant(synth.weight(N, K, seed).numpy())
            xq, sx = oracle.act_quant(np.ascontiguousarray(x[:, :K]))
            t_slice = pool.run_prefill_slice(xq, sx, Wq, sw)
            pre[name] = {"tokens_timed": rows, "seconds": round(t_slice, 3),
                         "tops_extrapolated": round(2.0 * rows * N * K / t_slice / 1e12, 6),
                         "seconds_for_2048_extrapolated": round(t_slice * M / rows, 2)}
    finally:
        pool.close()
    return {"value": round(value, 6), "unit": UNIT, "cores": pool.cores, "kind": "oracle",
            "sample": f"{steps} full decode steps (act_quant x2 + gate/up/down forwards over {step.bytes} "
                      f"packed bytes each) in {el:.1f} s on {pool.cores} host cores, one process per core "
                      f"over disjoint output rows",
            "one_core": {"value": round(one_core, 6), "unit": UNIT, "cores": 1,
                         "sample": f"{n1} full decode steps in {el1:.1f} s, single-threaded"},
            "prefill_m2048_slice": dict(pre, note="64 of 2048 tokens on every core; the per-token work is "
                                                  "the same for every token, so 2048 tokens take 32x as long "
                                                  "(extrapolated, not run)")}


def run_reference(args, rank, world):
    """The oracle, as it stands, timed on every host core (rank 0 only).  Each
    step is a bounded sample of the decode step: both act_quant calls and the
    three forwards over the leading fraction of the output rows (split over the
    cores), the fraction chosen so that the whole run takes about a minute
    whatever --steps is."""
    if rank != 0:
        return 0
    inp = workload_inputs()
    probe = OracleStep(inp, row_fraction=1.0 / 64)
    t0 = time.perf_counter()
    probe.run()
    t_probe = max(time.perf_counter() - t0, 1e-6)
    cores = host_cores()
    warm = min(max(args.warmup, 0), 3)
    budget = 60.0 / max(1, args.steps + warm)
    frac = min(1.0, max(1.0 / inp["F"], budget * cores / (t_probe * 64)))
    pool = OraclePool(inp, row_fraction=frac, cores=cores)
    try:
        if warm:
            pool.run_decode(warm)
        el = pool.run_decode(args.steps)
    finally:
        pool.close()
    value = pool.bytes * args.steps / el / 1e9
    sample = (f"{args.steps} steps, each act_quant x2 + gate/up/down over the first {frac:.4%} of output "
              f"rows ({pool.bytes} packed bytes), the C oracle on {cores} host cores (one process per core "
              f"over disjoint rows)")
    line = {
        "impl": "reference", "metric": METRIC, "value": round(value, 6), "unit": UNIT,
        "n_gpus": args.gpus, "steps": args.steps, "warmup": warm,
        "ms_per_step": round(el / args.steps * 1e3, 4), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "int8", "data": "synthetic",
        "config": {"workload": WORKLOAD, "M": 1, "sample_row_fraction": round(frac, 6)},
        "cpu_baseline": {"value": round(value, 6), "unit": UNIT, "cores": cores, "kind": "oracle",
                         "sample": sample},
        "e2e": {"value": round(value, 6), "unit": UNIT, "h2d_bytes_per_step": 0,
                "d2h_bytes_per_step": 0},
    }
    print(json.dumps(line), flush=True)
    return 0


# ---------------------------------------------------------------------------
# Clock sampling during the timed region
# ---------------------------------------------------------------------------
class ClockSampler:
    FIELDS = ("timestamp,index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, gpu_index: int):
        self.gpu_index = gpu_index
        self.proc = None
        self.lines = []

    def start(self):
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", f"--query-gpu={self.FIELDS}", "--format=csv,noheader,nounits",
                 "-lms", "100", "-i", str(self.gpu_index)],
                stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
        except OSError:
            self.proc = None
        time.sleep(0.3)

    def stop(self):
        if self.proc is None:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["nvidia-smi unavailable"]}
        time.sleep(0.15)
        self.proc.terminate()
        out, _ = self.proc.communicate(timeout=10)
        sm, mx, reasons = [], [], set()
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for line in out.strip().splitlines():
            parts = [p.strip() for p in line.split(",")]
            if len(parts) < 10:
                continue
            try:
                sm.append(float(parts[2]))
                mx.append(float(parts[3]))
            except ValueError:
                continue
            for name, val in zip(names, parts[6:10]):
                if val.lower().startswith("active"):
                    reasons.add(name)
        return {"sm_mhz": statistics.median(sm) if sm else None,
                "sm_max_mhz": max(mx) if mx else None,
                "reasons": sorted(reasons), "samples": len(sm)}


# ---------------------------------------------------------------------------
# Whole-job aggregation over ranks (replicas): max time, summed work
# ---------------------------------------------------------------------------
def reduce_max_ms(ms: float, dist=None, device=None) -> float:
    """The slowest rank's time (every rank must call it when dist is given)."""
    if dist is None:
        return float(ms)
    import torch
    t = torch.tensor([ms], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def device_lead(stream, us: float = 100.0):
    """Queue a short device-side spin on `stream` ahead of a start event, so the
    host's submission of the timed work overlaps it and the events bracket
    device execution only (the spin itself lies before the start event)."""
    import torch
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(us * 2000))  # ~us microseconds at ~2 GHz


def whole_job_gbs(bytes_per_rank: int, world: int, ms_max: float) -> float:
    """Aggregate throughput: every rank's bytes over the slowest rank's time."""
    return bytes_per_rank * world / (ms_max * 1e-3) / 1e9


# ---------------------------------------------------------------------------
# Our arm
# ---------------------------------------------------------------------------
def measured_peak_hbm():
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        with open(path) as f:
            return float(json.load(f)["hbm_gbs"]), "measured (MEASURED_PEAKS.json hbm_gbs, copy)"
    except (OSError, KeyError, ValueError):
        return FALLBACK_HBM_GBS, "fallback"


def ncu_traffic(kernel_sources, profile_name):
    """DRAM bytes per launch from the committed ncu summary, or None if the
    kernel source changed since it was captured."""
    path = os.path.join(ROOT, "profiles", profile_name)
    h = hashlib.sha256()
    for src in kernel_sources:
        with open(os.path.join(ROOT, src), "rb") as f:
            h.update(f.read())
    digest = h.hexdigest()
    try:
        kv = {}
        with open(path) as f:
            for line in f:
                if ":" in line and not line.startswith("#"):
                    k, v = line.split(":", 1)
                    kv[k.strip()] = v.strip()
        if kv.get("source_sha256") != digest:
            return None
        return float(kv["dram_bytes_per_launch"])
    except (OSError, KeyError, ValueError):
        return None


DECODE_SOURCES = ["bitlinear_w1_a8_gb300/csrc/decode.cu", "bitlinear_w1_a8_gb300/csrc/quant_row.cuh",
                  "bitlinear_w1_a8_gb300/csrc/common.cuh"]


def measured_peak_tensor():
    """Dense fp16/bf16 tensor peak (the prefill kernel runs kind::f16 MMAs)."""
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        with open(path) as f:
            return float(json.load(f)["bf16_tflops"]), "measured (MEASURED_PEAKS.json bf16_tflops, burst)"
    except (OSError, KeyError, ValueError):
        return 1900.0, "fallback"


def measure_int8_peak(dev, n: int = 8192, reps: int = 10):
    """Dense int8 tensor throughput as a library GEMM sees it on this GPU:
    torch._int_mm (int8 x int8 -> int32, cuBLASLt) on n^3, best of `reps`
    launches timed with CUDA events (the way the pool's bf16 peak is taken
    with torch.matmul)."""
    import torch
    try:
        a = torch.randint(-127, 128, (n, n), dtype=torch.int8, device=dev)
        b = torch.randint(-127, 128, (n, n), dtype=torch.int8, device=dev).t()
        torch._int_mm(a, b)
        torch.cuda.synchronize(dev)
        best = None
        for _ in range(reps):
            e0 = torch.cuda.Event(enable_timing=True)
            e1 = torch.cuda.Event(enable_timing=True)
            e0.record()
            torch._int_mm(a, b)
            e1.record()
            torch.cuda.synchronize(dev)
            ms = e0.elapsed_time(e1)
            best = ms if best is None else min(best, ms)
        del a, b
        return {"tops": round(2.0 * n ** 3 / (best * 1e-3) / 1e12, 2),
                "method": f"torch._int_mm int8 x int8 -> int32 (cuBLASLt), {n}^3, best of {reps}, CUDA events"}
    except Exception as e:  # an int8 GEMM the library does not offer on this GPU
        return {"tops": None, "method": f"torch._int_mm unavailable: {type(e).__name__}: {e}"[:200]}


PREFILL_SOURCES = ["bitlinear_w1_a8_gb300/csrc/prefill.cu", "bitlinear_w1_a8_gb300/csrc/tc_util.cuh",
                   "bitlinear_w1_a8_gb300/csrc/common.cuh"]


def measure_prefill(bl, dev, stream, dist, M=2048, launches=30):
    """BitNet-3B prefill GEMM, M = 2048 tokens, both FFN shapes, on the tensor-core
    kernels: TOPS = 2*M*N*K / launch time, back-to-back calls in a CUDA graph over
    rotating copies of inputs and outputs (working set > L2).  The headline is
    bitlinear_forward's AUTO path (the kernel with 128-token tiles); "wide" is
    bitlinear_forward_ws with BITLINEAR_ALGO_WIDE (the activations widened once
    into the workspace, then the contraction kernel; both launches timed)."""
    import torch
    from bitlinear_w1_a8_gb300 import synth
    s = synth.SEEDS["prefill"]
    D, F = synth.DIM_3B, synth.FFN_3B
    x = synth.activations(M, F, s["x"])  # K = 10240 for down; the first D columns for up
    out = {}
    peak, peak_src = measured_peak_tensor()
    for name, N, K, seed in (("up_shape", F, D, s["W_up_shape"]), ("down_shape", D, F, s["W_down_shape"])):
        W = synth.weight(N, K, seed).to(dev)
        nb = bl.bitlinear_packed_bytes(N, K)
        per_copy = nb + M * K + 4 * M * N
        copies = max(2, -(-2 * L2_BYTES // per_copy))
        packed = [torch.empty(nb, dtype=torch.uint8, device=dev) for _ in range(copies)]
        sw = torch.empty(1, dtype=torch.float32, device=dev)
        ws = torch.empty(bl.bitlinear_quantize_weights_workspace(N, K), dtype=torch.uint8, device=dev)
        bl.bitlinear_quantize_weights(W, packed[0], sw, ws)
        for p in packed[1:]:
            p.copy_(packed[0])
        xd = x[:, :K].contiguous().to(dev)
        xq = [torch.empty(M, K, dtype=torch.int8, device=dev) for _ in range(copies)]
        sx = torch.empty(M, dtype=torch.float32, device=dev)
        for q in xq:
            bl.bitlinear_quant_act(xd, q, sx)
        ys = [torch.empty(M, N, dtype=torch.float32, device=dev) for _ in range(copies)]
        fws = torch.empty(bl.bitlinear_forward_workspace(M, K), dtype=torch.uint8, device=dev)
        del W, xd

        def time_path(body):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.stream(stream):
                body(0, stream)
                torch.cuda.synchronize(dev)
                with torch.cuda.graph(g, stream=stream):
                    for i in range(launches):
                        body(i, stream)
                g.replay()
                torch.cuda.synchronize(dev)
                e0 = torch.cuda.Event(enable_timing=True)
                e1 = torch.cuda.Event(enable_timing=True)
                device_lead(stream)
                e0.record(stream)
                g.replay()
                e1.record(stream)
            torch.cuda.synchronize(dev)
            ms = reduce_max_ms(e0.elapsed_time(e1), dist, dev) / launches
            tops = 2.0 * M * N * K / (ms * 1e-3) / 1e12
            return {"us_per_launch": round(ms * 1e3, 3), "tops": round(tops, 2),
                    "frac_of_fp16_peak": round(tops / peak, 4)}

        def wide(i, st):
            j = i % copies
            bl.bitlinear_forward_ws(xq[j], sx, packed[j], sw, N, ys[j], workspace=fws, algo=bl.ALGO_WIDE,
                                    flags=bl.FLAG_PDL, stream=st)

        def tiles128(i, st):
            j = i % copies
            bl.bitlinear_forward_ex(xq[j], sx, packed[j], sw, N, ys[j], algo=bl.ALGO_PREFILL, stream=st)

        r = {"M": M, "N": N, "K": K, "rotating_copies": copies}
        r.update(time_path(tiles128))
        r["path"] = "bitlinear_forward (AUTO: 128-token tiles)"
        r["wide"] = time_path(wide)
        r["wide"]["path"] = "bitlinear_forward_ws, BITLINEAR_ALGO_WIDE (widen pre-pass + contraction, both timed)"
        out[name] = r
        del packed, xq, ys, fws
        torch.cuda.empty_cache()
    tot_ops = sum(2.0 * v["M"] * v["N"] * v["K"] for v in out.values())
    tot_us = sum(v["us_per_launch"] for v in out.values())
    achieved = tot_ops / (tot_us * 1e-6) / 1e12
    int8 = measure_int8_peak(dev)
    out["roofline"] = {"kernel": "prefill_kernel (tcgen05 kind::f16, exact int8 x ternary)",
                       "bound": "tensor", "achieved": round(achieved, 2), "peak": peak,
                       "unit": "TFLOP/s", "frac": round(achieved / peak, 4), "peak_source": peak_src,
                       "traffic": ncu_traffic(PREFILL_SOURCES, "prefill_m2048_bitnet3b_ncu.txt"),
                       "note": "int8-equivalent ops (2*M*N*K) per launch / launch time; no int8 "
                               "tcgen05 MMA exists on sm_103a (ptxas rejects kind::i8), so the kernel "
                               "runs exact kind::f16 MMAs and the dense fp16 peak is the roofline",
                       "int8_peak": dict(int8, frac=(round(achieved / int8["tops"], 4) if int8["tops"] else None),
                                         note="the dense int8 rate a library GEMM reaches on this GPU; "
                                              "frac = this kernel's int8-equivalent rate over it")}
    return out


def measure_weight_set(bl, dev, stream, dist, Ms=(1, 8, 32, 64), reps=10, attention=0):
    """BitNet-3B full per-token weight set: 32 layers x (q, k, v, o 2560x2560;
    gate, up 2560->10240; down 10240->2560) plus the LM head 2560->50000, every
    matrix independently seeded N(0, 0.02) and quantised once (870,860,800
    packed bytes, > 4x L2).  One step = every BitLinear call of one decode step
    of M tokens in block order -- [q||k||v], [o], [gate||up], [down] per layer,
    then the LM head and the greedy token (bitlinear_argmax, 4 bytes a token)
    -- each a bitlinear_linear_ws call (one shared workspace) on seeded synthetic inputs
    (attention and residuals are not part of this path), replayed as one CUDA
    graph with PDL.  With attention = n > 0 each layer also rotates and caches
    its new tokens (bitlinear_kv_append, an int8 cache of its own) and attends
    to n tokens a sequence (bitlinear_attention) between q||k||v and o, which
    then reads the attention's output."""
    import torch
    from bitlinear_w1_a8_gb300 import synth
    D, F, V, L = synth.DIM_3B, synth.FFN_3B, synth.VOCAB, synth.LAYERS_3B
    shapes = [(D, D), (D, D), (D, D), (D, D), (F, D), (F, D), (D, F)]  # q k v o gate up down: (N, K)
    ws = torch.empty(bl.bitlinear_quantize_weights_workspace(F, D), dtype=torch.uint8, device=dev)
    layers = []
    total_bytes = 0
    for layer in range(L):
        mats = []
        for proj, (N, K) in enumerate(shapes):
            W = synth.normal_cuda((N, K), synth.WEIGHT_STD, synth.weight_set_seed(layer, proj), dev)
            pk = torch.empty(bl.bitlinear_packed_bytes(N, K), dtype=torch.uint8, device=dev)
            sc = torch.empty(1, dtype=torch.float32, device=dev)
            bl.bitlinear_quantize_weights(W, pk, sc, ws)
            mats.append((pk, sc, N))
            total_bytes += pk.numel()
        layers.append(mats)
    W = synth.normal_cuda((V, D), synth.WEIGHT_STD, synth.SEEDS["weight_set"]["lm_head"], dev)
    head_pk = torch.empty(bl.bitlinear_packed_bytes(V, D), dtype=torch.uint8, device=dev)
    head_sc = torch.empty(1, dtype=torch.float32, device=dev)
    bl.bitlinear_quantize_weights(W, head_pk, head_sc, ws)
    total_bytes += head_pk.numel()
    del W
    weights_n = sum(N * K for N, K in shapes) * L + V * D
    out = {"packed_bytes_per_step": total_bytes, "weights": weights_n, "launch_calls_per_step": (6 if attention else 4) * L + 2}
    for M in Ms:
        xa = synth.activations(M, D, synth.SEEDS["weight_set"]["x"]).to(dev)
        xb = synth.activations(M, F, synth.SEEDS["weight_set"]["x"] + 1).to(dev)
        xq_a = torch.empty(M, D, dtype=torch.int8, device=dev)
        xq_b = torch.empty(M, F, dtype=torch.int8, device=dev)
        sx_a = torch.empty(M, dtype=torch.float32, device=dev)
        sx_b = torch.empty(M, dtype=torch.float32, device=dev)
        ys = {n: torch.empty(M, n, dtype=torch.float32, device=dev) for n in (D, F, V)}
        yq, yk, yv = (torch.empty(M, D, dtype=torch.float32, device=dev) for _ in range(3))
        yu = torch.empty(M, F, dtype=torch.float32, device=dev)
        token = torch.empty(M, dtype=torch.int32, device=dev)
        fws = torch.empty(bl.bitlinear_forward_workspace(M, F), dtype=torch.uint8, device=dev)
        attend = layer_attention(bl, dev, M, D, L, attention, (yq, yk, yv)) if attention else None
        xo = attend.out.view(M, D) if attention else xa

        def step(s):
            for layer, mats in enumerate(layers):
                (q, sq, _), (k, sk, _), (v, sv, _), (o, so, _), (g, sg, _), (u, su, _), (d, sd, _) = mats
                bl.bitlinear_linear_ws(xa, [(q, sq, yq), (k, sk, yk), (v, sv, yv)], xq_a, sx_a, fws,
                                       flags=bl.FLAG_PDL, stream=s)
                if attention:
                    attend(layer, s)
                bl.bitlinear_linear_ws(xo, [(o, so, ys[D])], xq_a, sx_a, fws, flags=bl.FLAG_PDL, stream=s)
                bl.bitlinear_linear_ws(xa, [(g, sg, ys[F]), (u, su, yu)], xq_a, sx_a, fws, flags=bl.FLAG_PDL,
                                       stream=s)
                bl.bitlinear_linear_ws(xb, [(d, sd, ys[D])], xq_b, sx_b, fws, flags=bl.FLAG_PDL, stream=s)
            bl.bitlinear_linear_ws(xa, [(head_pk, head_sc, ys[V])], xq_a, sx_a, fws, flags=bl.FLAG_PDL, stream=s)
            bl.bitlinear_argmax(ys[V], token, stream=s)

        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            step(stream)
            torch.cuda.synchronize(dev)
            with torch.cuda.graph(g, stream=stream):
                step(stream)
            for _ in range(3):
                g.replay()
            torch.cuda.synchronize(dev)
            e0 = torch.cuda.Event(enable_timing=True)
            e1 = torch.cuda.Event(enable_timing=True)
            device_lead(stream)
            e0.record(stream)
            for _ in range(reps):
                g.replay()
            e1.record(stream)
        torch.cuda.synchronize(dev)
        ms = reduce_max_ms(e0.elapsed_time(e1), dist, dev) / reps
        out[f"M{M}"] = {"us_per_step": round(ms * 1e3, 2),
                        "packed_GBps": round(total_bytes / (ms * 1e-3) / 1e9, 1),
                        "tops": round(2.0 * M * weights_n / (ms * 1e-3) / 1e12, 2),
                        "us_per_token": round(ms * 1e3 / M, 3)}
        del g, attend
    if attention:
        out["attention_tokens"] = attention
        out["cache_bytes_per_token_and_layer"] = 2 * D + 2 * synth.HEADS_3B * 4
    return out


def layer_attention(bl, dev, M, D, layers, tokens, qkv):
    """A callable (layer, stream) that caches the new tokens of q, k, v [M, D] in the layer's own
    paged int8 cache, `tokens` long, and attends to it; its `out` is [M, heads, head_dim]."""
    import torch
    from bitlinear_w1_a8_gb300 import synth
    H, page = synth.HEADS_3B, 64
    hd, width = D // H, -(-tokens // page)
    g = torch.Generator(device=dev)
    g.manual_seed(synth.SEEDS["weight_set"]["x"])
    shape = (M * width, H, page, hd)
    caches = []
    for _ in range(layers):
        codes = [torch.randint(-127, 128, shape, generator=g, dtype=torch.int8, device=dev) for _ in "kv"]
        caches.append((*codes, *(torch.full(shape[:3], 1 / 64, device=dev) for _ in "kv")))
    table = torch.randperm(M * width, generator=g, device=dev).to(torch.int32).view(M, width)
    lengths = torch.full((M,), tokens, dtype=torch.int32, device=dev)
    positions = lengths - 1
    rope = (bl.bitlinear_rope_frequencies(hd).to(dev), bl.ROPE_HALF)
    q, k, v = (t.view(M, H, hd) for t in qkv)
    out = torch.empty(M, H, hd, dtype=torch.float32, device=dev)
    need = bl.bitlinear_attention_workspace(M, H, H, hd)
    space = torch.empty(need, dtype=torch.uint8, device=dev) if need else None

    def attend(layer, stream):
        bl.bitlinear_kv_append(k, v, caches[layer], positions, table, q=q, q_out=q, rope=rope, flags=bl.FLAG_PDL,
                               stream=stream)
        bl.bitlinear_attention(q, caches[layer], table, lengths, out, workspace=space, flags=bl.FLAG_PDL, stream=stream)

    attend.out = out
    return attend


def measure_ffn_1b3(bl, dev, stream, dist, Ms=(1, 512), reps=50):
    """BitNet-1.3B FFN sub-block (dim 2048, ffn 8192): RMSNorm -> act_quant ->
    gate || up -> ReLU^2(gate) * up -> sub-norm -> act_quant -> down, as two
    bitlinear_linear_ws calls (the prologues fused, and at M <= 8 the gating in
    the gate || up launch's epilogue; with a workspace, so the WIDE kernel
    takes the matrices its AUTO rule gives it), seeded as in the
    parity test; one CUDA graph of `reps` sub-blocks over rotating weight
    copies (> 4x L2)."""
    import torch
    from bitlinear_w1_a8_gb300 import synth
    s = synth.SEEDS["ffn_1b3"]
    D, F = synth.DIM_1B3, synth.FFN_1B3
    gamma = synth.uniform((D,), 0.5, 1.5, s["norm"]).to(dev)
    gamma_sub = synth.uniform((F,), 0.5, 1.5, s["subnorm"]).to(dev)
    ws = torch.empty(bl.bitlinear_quantize_weights_workspace(F, D), dtype=torch.uint8, device=dev)
    base = []
    for name, (N, K) in (("gate", (F, D)), ("up", (F, D)), ("down", (D, F))):
        pk = torch.empty(bl.bitlinear_packed_bytes(N, K), dtype=torch.uint8, device=dev)
        sc = torch.empty(1, dtype=torch.float32, device=dev)
        bl.bitlinear_quantize_weights(synth.weight(N, K, s[name]).to(dev), pk, sc, ws)
        base.append((pk, sc))
    per = sum(p.numel() for p, _ in base)
    copies = max(2, -(-4 * L2_BYTES // per))
    sets = [base] + [[(p.clone(), sc) for p, sc in base] for _ in range(copies - 1)]
    out = {"packed_bytes_per_block": per, "weight_copies": copies}
    for M in Ms:
        x = synth.activations(M, D, s["x"]).to(dev)
        xq = torch.empty(M, D, dtype=torch.int8, device=dev)
        sx = torch.empty(M, dtype=torch.float32, device=dev)
        hq = torch.empty(M, F, dtype=torch.int8, device=dev)
        hsx = torch.empty(M, dtype=torch.float32, device=dev)
        yg = torch.empty(M, F, dtype=torch.float32, device=dev)
        yu = torch.empty(M, F, dtype=torch.float32, device=dev)
        yd = torch.empty(M, D, dtype=torch.float32, device=dev)
        fws = torch.empty(bl.bitlinear_forward_workspace(M, F), dtype=torch.uint8, device=dev)

        # At decode sizes the gate || up launch writes ReLU^2(gate) * up from its
        # epilogue; above them the down call's prologue applies the gating.
        gated = M <= 8

        def block(i, st):
            (g, sg), (u, su), (d, sd) = sets[i % copies]
            bl.bitlinear_linear_ws(x, [(g, sg, yg), (u, su, yu)], xq, sx, fws, rms_weight=gamma, rms_eps=1e-6,
                                   flags=bl.FLAG_PDL | (bl.FLAG_GATED if gated else 0), stream=st)
            bl.bitlinear_linear_ws(yg, [(d, sd, yd)], hq, hsx, fws, mul=None if gated else yu,
                                   rms_weight=gamma_sub, rms_eps=1e-6, flags=bl.FLAG_PDL, stream=st)

        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            block(0, stream)
            torch.cuda.synchronize(dev)
            with torch.cuda.graph(g, stream=stream):
                for i in range(reps):
                    block(i, stream)
            for _ in range(3):
                g.replay()
            torch.cuda.synchronize(dev)
            e0 = torch.cuda.Event(enable_timing=True)
            e1 = torch.cuda.Event(enable_timing=True)
            device_lead(stream)
            e0.record(stream)
            g.replay()
            e1.record(stream)
        torch.cuda.synchronize(dev)
        us = reduce_max_ms(e0.elapsed_time(e1), dist, dev) / reps * 1e3
        out[f"M{M}"] = {"us_per_block": round(us, 2), "packed_GBps": round(per / (us * 1e-6) / 1e9, 1),
                        "tops": round(2.0 * M * (2 * F * D + D * F) / (us * 1e-6) / 1e12, 2)}
        del g
    return out


def run_ours(args, rank, world, local_rank):
    import torch
    import bitlinear_w1_a8_gb300 as bl
    from bitlinear_w1_a8_gb300 import build as blbuild

    if not os.path.exists(bl.library_path()):
        blbuild.build()
    bl.load_library()
    torch.cuda.set_device(local_rank)
    dev = torch.device("cuda", local_rank)
    dist = None
    if world > 1:
        import torch.distributed as dist
        dist.init_process_group("nccl", device_id=dev)

    inp = workload_inputs()
    D, F = inp["D"], inp["F"]
    bytes_u = bl.bitlinear_packed_bytes(F, D)
    bytes_d = bl.bitlinear_packed_bytes(D, F)
    per_step = 2 * bytes_u + bytes_d
    R = max(8, -(-4 * L2_BYTES // per_step))          # copies so that R * step > 4x L2
    R = 1 << (R - 1).bit_length()                       # 32 for the 3B shapes

    # Quantise once, then replicate the packed bytes into R slots (distinct memory).
    pu = torch.empty(bytes_u, dtype=torch.uint8, device=dev)
    pd = torch.empty(bytes_d, dtype=torch.uint8, device=dev)
    sw = torch.empty(2, dtype=torch.float32, device=dev)
    ws = torch.empty(bl.bitlinear_quantize_weights_workspace(F, D), dtype=torch.uint8, device=dev)
    bl.bitlinear_quantize_weights(inp["W_up_shape"].to(dev), pu, sw[0:1], ws)
    bl.bitlinear_quantize_weights(inp["W_down_shape"].to(dev), pd, sw[1:2], ws)
    slots = []
    for _ in range(R):
        slots.append((pu.clone(), pu.clone(), pd.clone()))
    sw_u, sw_d = sw[0:1], sw[1:2]
    x_a = inp["x_a"].to(dev)
    xq_a = torch.empty(1, D, dtype=torch.int8, device=dev)
    xq_b = torch.empty(1, F, dtype=torch.int8, device=dev)
    sx_a = torch.empty(1, dtype=torch.float32, device=dev)
    sx_b = torch.empty(1, dtype=torch.float32, device=dev)
    y_g = torch.empty(1, F, dtype=torch.float32, device=dev)
    y_u = torch.empty(1, F, dtype=torch.float32, device=dev)
    y_d = torch.empty(1, D, dtype=torch.float32, device=dev)
    flags = 0 if args.no_pdl else bl.FLAG_PDL

    # One step is the FFN of one decode token: down(ReLU^2(gate(x)) * up(x)).
    def step_separate(i, stream):
        # act_quant and forward as separate calls (5 launches per step); the
        # second act_quant applies the gating prologue to the gate and up outputs
        g, u, d = slots[i % R]
        bl.bitlinear_quant_act(x_a, xq_a, sx_a, stream=stream)
        bl.bitlinear_forward_ex(xq_a, sx_a, g, sw_u, F, y_g, flags=flags, stream=stream)
        bl.bitlinear_forward_ex(xq_a, sx_a, u, sw_u, F, y_u, flags=flags, stream=stream)
        bl.bitlinear_quant_act(y_g, xq_b, sx_b, mul=y_u, stream=stream)
        bl.bitlinear_forward_ex(xq_b, sx_b, d, sw_d, D, y_d, flags=flags, stream=stream)

    def step_linear(i, stream):
        # bitlinear_linear: act_quant fused into the decode kernel; gate || up in
        # one launch whose epilogue writes h = ReLU^2(gate) * up; down on h
        g, u, d = slots[i % R]
        bl.bitlinear_linear(x_a, [(g, sw_u, y_g), (u, sw_u, y_u)], xq_a, sx_a, flags=flags | bl.FLAG_GATED,
                            stream=stream)
        bl.bitlinear_linear(y_g, [(d, sw_d, y_d)], xq_b, sx_b, flags=flags, stream=stream)

    step = step_separate if args.separate else step_linear
    kernels_per_step = 5 if args.separate else 2
    stream = torch.cuda.Stream(device=dev)

    def capture(fn, n):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            fn(0, stream)  # settle any lazy initialisation outside the capture
            torch.cuda.synchronize(dev)
            with torch.cuda.graph(g, stream=stream):
                for i in range(n):
                    fn(i, stream)
        return g

    # One graph = one full rotation of R steps; K steps = K // R launches + a remainder graph.
    g_full = capture(step, R)
    rem = args.steps % R
    g_rem = capture(step, rem) if rem else None

    def run_steps(k):
        with torch.cuda.stream(stream):
            for _ in range(k // R):
                g_full.replay()
            if k % R:
                if k % R == rem and g_rem is not None:
                    g_rem.replay()
                else:
                    for i in range(k % R):
                        step(i, stream)

    # warm-up: every graph the timed region replays is replayed (and so
    # uploaded) here first, then the requested warm-up steps run
    with torch.cuda.stream(stream):
        g_full.replay()
        if g_rem is not None:
            g_rem.replay()
    run_steps(max(3, args.warmup))
    torch.cuda.synchronize(dev)

    # timed region
    visible = os.environ.get("CUDA_VISIBLE_DEVICES", "")
    ids = [v.strip() for v in visible.split(",") if v.strip()]
    smi_id = ids[local_rank] if local_rank < len(ids) else str(local_rank)
    sampler = ClockSampler(smi_id) if rank == 0 else None
    if sampler:
        sampler.start()
    if dist:
        dist.barrier()
    torch.cuda.synchronize(dev)
    ev0 = torch.cuda.Event(enable_timing=True)
    ev1 = torch.cuda.Event(enable_timing=True)
    device_lead(stream)
    ev0.record(stream)
    run_steps(args.steps)
    ev1.record(stream)
    torch.cuda.synchronize(dev)
    if dist:
        dist.barrier()
    clocks = sampler.stop() if sampler else None
    ms_max = reduce_max_ms(ev0.elapsed_time(ev1), dist, dev)
    value = whole_job_gbs(per_step * args.steps, world, ms_max)

    # The other path, for comparison (same rotation, same timing method).
    alt = step_linear if args.separate else step_separate
    g_alt = capture(alt, R)
    alt_reps = max(3, min(2000, args.steps // R))
    with torch.cuda.stream(stream):
        g_alt.replay()
    torch.cuda.synchronize(dev)
    a0 = torch.cuda.Event(enable_timing=True)
    a1 = torch.cuda.Event(enable_timing=True)
    device_lead(stream)
    a0.record(stream)
    with torch.cuda.stream(stream):
        for _ in range(alt_reps):
            g_alt.replay()
    a1.record(stream)
    torch.cuda.synchronize(dev)
    alt_ms = a0.elapsed_time(a1) / (alt_reps * R)
    alt_line = {"path": "separate act_quant + forward calls (5 launches)" if not args.separate
                else "bitlinear_linear (2 launches)",
                "ms_per_step": round(alt_ms, 6), "value": round(per_step / (alt_ms * 1e-3) / 1e9, 3)}

    # Dominant kernel alone: back-to-back launches of the decode kernel over the rotation.
    def fwd_only(i, s):
        g, u, d = slots[i % R]
        if args.separate:
            bl.bitlinear_forward_ex(xq_a, sx_a, g, sw_u, F, y_g, flags=flags, stream=s)
            bl.bitlinear_forward_ex(xq_a, sx_a, u, sw_u, F, y_u, flags=flags, stream=s)
            bl.bitlinear_forward_ex(xq_b, sx_b, d, sw_d, D, y_d, flags=flags, stream=s)
        else:
            step_linear(i, s)

    g_fwd = capture(fwd_only, R)
    reps = max(3, min(200, args.steps // R))
    with torch.cuda.stream(stream):
        for _ in range(3):
            g_fwd.replay()
    torch.cuda.synchronize(dev)
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    device_lead(stream)
    e0.record(stream)
    with torch.cuda.stream(stream):
        for _ in range(reps):
            g_fwd.replay()
    e1.record(stream)
    torch.cuda.synchronize(dev)
    launches_per_rot = 3 if args.separate else 2
    fwd_launches = reps * launches_per_rot * R
    fwd_ms = e0.elapsed_time(e1) / fwd_launches
    if args.separate:
        # per forward launch: packed weights + int8 activations + one fp32 scale + fp32 outputs
        alg_bytes = (2 * (bytes_u + D + 4 + 4 * F) + (bytes_d + F + 4 + 4 * D)) / 3.0
    else:
        # per fused launch: packed weights + fp32 input + int8 codes and scale written + fp32 outputs
        alg_bytes = ((2 * bytes_u + 4 * D + D + 4 + 2 * 4 * F) + (bytes_d + 4 * F + F + 4 + 4 * D)) / 2.0
    peak, peak_src = measured_peak_hbm()
    achieved = alg_bytes / (fwd_ms * 1e-3) / 1e9

    # End to end through the public API: pinned host inputs in, host outputs out
    # (one copy each way: the step's inputs and outputs sit in one buffer each).
    # The step's input is the token row x, its result the down projection.
    e2e_steps = max(10, min(args.e2e_steps, args.steps))
    h_in = inp["x_a"].reshape(-1).clone().pin_memory()
    h_out = torch.empty(D, dtype=torch.float32).pin_memory()
    e_xa = torch.empty(1, D, dtype=torch.float32, device=dev)
    e_yg = torch.empty(1, F, dtype=torch.float32, device=dev)
    e_yu = torch.empty(1, F, dtype=torch.float32, device=dev)
    e_yd = torch.empty(1, D, dtype=torch.float32, device=dev)
    e2e_h2d, e2e_d2h = 4 * D, 4 * D
    e_xa_flat, e_yd_flat = e_xa.view(-1), e_yd.view(-1)

    def e2e_step(i):
        g, u, d = slots[i % R]
        e_xa_flat.copy_(h_in, non_blocking=True)
        if args.separate:
            bl.bitlinear_quant_act(e_xa, xq_a, sx_a, stream=stream)
            bl.bitlinear_forward_ex(xq_a, sx_a, g, sw_u, F, e_yg, flags=flags, stream=stream)
            bl.bitlinear_forward_ex(xq_a, sx_a, u, sw_u, F, e_yu, flags=flags, stream=stream)
            bl.bitlinear_quant_act(e_yg, xq_b, sx_b, mul=e_yu, stream=stream)
            bl.bitlinear_forward_ex(xq_b, sx_b, d, sw_d, D, e_yd, flags=flags, stream=stream)
        else:
            bl.bitlinear_linear(e_xa, [(g, sw_u, e_yg), (u, sw_u, e_yu)], xq_a, sx_a, flags=flags | bl.FLAG_GATED,
                                stream=stream)
            bl.bitlinear_linear(e_yg, [(d, sw_d, e_yd)], xq_b, sx_b, flags=flags, stream=stream)
        h_out.copy_(e_yd_flat, non_blocking=True)

    with torch.cuda.stream(stream):
        for i in range(20):
            e2e_step(i)
        torch.cuda.synchronize(dev)
        if dist:
            dist.barrier()
        q0 = torch.cuda.Event(enable_timing=True)
        q1 = torch.cuda.Event(enable_timing=True)
        q0.record(stream)
        for i in range(e2e_steps):
            e2e_step(i)
        q1.record(stream)
        torch.cuda.synchronize(dev)
    e2e_value = whole_job_gbs(per_step * e2e_steps, world, reduce_max_ms(q0.elapsed_time(q1), dist, dev))
    # The same calls captured once into a CUDA graph (one step per weight copy)
    # and replayed: every step still copies its inputs in and its outputs out,
    # but no Python runs per step.
    g_e2e = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(g_e2e, stream=stream):
            for i in range(R):
                e2e_step(i)
        for _ in range(3):
            g_e2e.replay()
        torch.cuda.synchronize(dev)
        if dist:
            dist.barrier()
        e2e_reps = max(1, e2e_steps // R)
        device_lead(stream)
        q2 = torch.cuda.Event(enable_timing=True)
        q3 = torch.cuda.Event(enable_timing=True)
        q2.record(stream)
        for _ in range(e2e_reps):
            g_e2e.replay()
        q3.record(stream)
        torch.cuda.synchronize(dev)
    e2e_graph_value = whole_job_gbs(per_step * R * e2e_reps, world, reduce_max_ms(q2.elapsed_time(q3), dist, dev))

    prefill = None if args.no_prefill else measure_prefill(bl, dev, stream, dist)
    weight_set = None if args.no_weight_set else measure_weight_set(bl, dev, stream, dist)
    with_attention = measure_weight_set(bl, dev, stream, dist, attention=args.attention) if args.attention > 0 else None
    ffn_1b3 = None if args.no_weight_set else measure_ffn_1b3(bl, dev, stream, dist)

    cpu = None
    if rank == 0 and world == 1 and not args.no_cpu_baseline:
        cpu = cpu_baseline(inp, args.cpu_seconds)

    if rank == 0:
        line = {
            "metric": METRIC, "value": round(value, 3), "unit": UNIT, "n_gpus": world,
            "steps": args.steps, "warmup": max(3, args.warmup),
            "ms_per_step": round(ms_max / args.steps, 6), "higher_is_better": True,
            "scaling": "weak", "vs_baseline": None, "dtype": "int8", "data": "synthetic",
            "config": {
                "workload": WORKLOAD, "M": 1,
                "matrices_per_step": {"gate": [F, D], "up": [F, D], "down": [D, F]},
                "packed_bytes_per_step": per_step, "weight_copies": R,
                "l2": f"inputs larger than L2: {R} rotating weight copies, "
                      f"{R * per_step / 1e6:.0f} MB > 4x {L2_BYTES / 1e6:.0f} MB",
                "cuda_graph": True, "pdl": not args.no_pdl, "parallelism": f"replicas{world}",
                "path": ("separate bitlinear_quant_act + bitlinear_forward_ex calls" if args.separate else
                         "bitlinear_linear: gate||up in one launch (its epilogue writes ReLU^2(gate)*up), "
                         "down on that product in one launch, act_quant fused in both"),
            },
            "other_path": alt_line,
            "roofline": {
                "kernel": ("decode_kernel<1> (bitlinear_forward, M=1)" if args.separate else
                           "decode_kernel<1> (bitlinear_linear: act_quant fused, M=1)"), "bound": "hbm",
                "achieved": round(achieved, 3), "peak": peak, "unit": "GB/s",
                "frac": round(achieved / peak, 4),
                "traffic": ncu_traffic(DECODE_SOURCES, "decode_m1_bitnet3b_ncu.txt"),
                "peak_source": peak_src,
                "algorithmic_bytes_per_launch": round(alg_bytes, 1),
                "avg_launch_us": round(fwd_ms * 1e3, 4),
                "timing": f"{fwd_launches} back-to-back launches in CUDA graphs (PDL), CUDA events",
            },
            "e2e": {"value": round(e2e_value, 3), "unit": UNIT,
                    "h2d_bytes_per_step": e2e_h2d, "d2h_bytes_per_step": e2e_d2h,
                    "steps": e2e_steps,
                    "note": "eager calls through the Python binding of the C ABI (FLAG_PDL); the "
                            "token row copied in from pinned host memory and the down output "
                            "copied out every step"},
            "e2e_graph": {"value": round(e2e_graph_value, 3), "unit": UNIT,
                          "h2d_bytes_per_step": e2e_h2d, "d2h_bytes_per_step": e2e_d2h,
                          "steps": R * e2e_reps,
                          "note": f"the same calls captured once into a CUDA graph of {R} steps and "
                                  "replayed: the host copies in and out still run every step"},
            "gpu_launches": kernels_per_step * args.steps,
            "clocks": clocks,
        }
        if prefill:
            line["prefill_m2048"] = prefill
        if weight_set:
            line["weight_set_3b"] = weight_set
        if with_attention:
            line["weight_set_3b_attention"] = with_attention
        if ffn_1b3:
            line["ffn_1b3"] = ffn_1b3
        if cpu:
            line["cpu_baseline"] = cpu
        print(json.dumps(line), flush=True)
    if dist:
        dist.barrier()
        dist.destroy_process_group()
    return 0


def main():
    args = parse_args()
    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    local_rank = int(os.environ.get("LOCAL_RANK", "0"))
    if args.impl == "reference":
        return run_reference(args, rank, world)
    return run_ours(args, rank, world, local_rank)


if __name__ == "__main__":
    sys.exit(main())
