"""Benchmark of the ragged MoE grouped GEMM on B200.

One step = one pass of the whole hot path over one batch of synthetic input:
forward, dgrad and wgrad of the large grouped GEMM (E=16, T=262144 rows, K=6144, N=4096,
bf16, the TileOPs issue 1566 "GLM-up" shape) plus the masked forward of the sglang PR 32385
shape (E=8, mmax=128, K=768, N=2048). The metric is grouped GEMM bf16 TFLOP/s with
algorithmic flops 2*T*K*N per pass (T counts real rows only).

    python bench.py [--gpus N] [--steps K] [--warmup W] [--impl ours|reference]

Under torchrun (N > 1) every rank runs its own copy of the per-GPU workload (expert
parallelism: each GPU owns its experts; no collective on the data path), the timed region
is bracketed by barriers, and rank 0 prints the max-over-ranks time. ``--impl reference``
times the CPU oracle on a bounded sample of the same workload (rank 0 only).
"""
from __future__ import annotations

import argparse
import hashlib
import json
import os
import statistics
import subprocess
import threading
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

METRIC = "grouped GEMM BF16 TFLOP/s (fwd/dgrad/wgrad) and % of B200 dense BF16 peak"
UNIT = "TFLOP/s"

# DRAM bytes per launch (dram__bytes_read.sum + dram__bytes_write.sum) of the dominant kernel,
# keyed by pass and workload, valid only for the kernel sources whose hash is recorded with
# them (a changed kernel reports null until it is captured again). The figures come from one
# capture of the second launch of each pass (-k regex:grouped_gemm -s 3 -c 3) with only these
# counters, which ncu collects in a single pass (nothing saved or restored); a launch list over
# many kernels collects gpu__time_duration.sum alone.
NCU_TRAFFIC = {
    ("forward", "large"): 11.899e9,
    ("dgrad", "large"): 12.970e9,
    ("wgrad", "large"): 16.147e9,
}
NCU_TRAFFIC_SRC_HASH = "034efc478728fc44"


GEMM_SOURCES = ("gg_kernel.cuh", "ptx.cuh", "gg_api.cu", "gg_masked.cuh")  # kernels + launch


def kernel_source_hash() -> str:
    """Hash of the sources of the grouped GEMM kernels: the stored ncu traffic is reported
    only while it matches (a changed kernel invalidates the counters)."""
    h = hashlib.sha256()
    for f in GEMM_SOURCES:
        h.update(open(os.path.join(ROOT, "moe_grouped_gemm_ragged_b200", "csrc", f), "rb").read())
    return h.hexdigest()[:16]


def load_peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        d = json.load(open(p))
        return d, "measured"
    return {"hbm_gbs": 6650.0, "bf16_tflops": 1590.0, "bf16_tflops_sustained": 1400.0}, \
        "fallback"


class ClockSampler:
    """nvidia-smi clock/throttle sampling during the timed region."""

    FIELDS = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, device_index: int):
        self.proc = None
        self.lines = []
        sel = str(device_index)
        try:
            uuid = str(torch.cuda.get_device_properties(device_index).uuid)
            sel = uuid if uuid.startswith("GPU-") else "GPU-" + uuid
        except Exception:
            pass
        self.sel = sel

    def start(self):
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", "-i", self.sel, f"--query-gpu={self.FIELDS}",
                 "--format=csv,noheader,nounits", "-lms", "100"],
                stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
        except OSError:
            self.proc = None

    def stop(self, window=None):
        if self.proc is None:
            return None
        self.proc.terminate()
        try:
            out, _ = self.proc.communicate(timeout=5)
        except subprocess.TimeoutExpired:
            self.proc.kill()
            out, _ = self.proc.communicate()
        return self.parse(out)

    @staticmethod
    def parse(out: str):
        """Summary of `nvidia-smi --format=csv,noheader,nounits` lines of FIELDS."""
        rows = []
        for line in out.strip().splitlines():
            parts = [x.strip() for x in line.split(",")]
            if len(parts) >= 9:
                rows.append(parts)
        if not rows:
            return None
        sm = [float(r[1]) for r in rows if r[1].replace(".", "").isdigit()]
        mx = [float(r[2]) for r in rows if r[2].replace(".", "").isdigit()]
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        reasons = sorted({names[i] for r in rows for i in range(4) if r[5 + i] == "Active"})
        loaded = [s for s in sm if mx and s > 0.5 * max(mx)] or sm
        return {"sm_mhz": statistics.median(loaded) if loaded else None,
                "sm_max_mhz": max(mx) if mx else None, "reasons": reasons,
                "samples": len(rows)}


class NvmlClockSampler:
    """SM clock and clock-event reasons sampled in-process through NVML every 10 ms during
    the timed region (nvidia-smi, started as a process, catches only a few samples of a
    region a few hundred milliseconds long). Same summary as ClockSampler.parse."""

    # NVML clock-event reason bits
    REASONS = {"sw_power_cap": 0x4, "hw_slowdown": 0x8, "sw_thermal_slowdown": 0x20,
               "hw_thermal_slowdown": 0x40}

    def __init__(self, device_index: int, period_s: float = 0.01):
        import pynvml
        self.nv = pynvml
        pynvml.nvmlInit()
        uuid = str(torch.cuda.get_device_properties(device_index).uuid)
        uuid = uuid if uuid.startswith("GPU-") else "GPU-" + uuid
        self.h = pynvml.nvmlDeviceGetHandleByUUID(uuid)
        self.max_mhz = pynvml.nvmlDeviceGetMaxClockInfo(self.h, pynvml.NVML_CLOCK_SM)
        self.period = period_s
        self.samples = []
        self.stop_flag = threading.Event()
        self.thread = None

    def _run(self):
        nv = self.nv
        get_reasons = getattr(nv, "nvmlDeviceGetCurrentClocksEventReasons", None) or \
            nv.nvmlDeviceGetCurrentClocksThrottleReasons
        while not self.stop_flag.is_set():
            try:
                self.samples.append((time.perf_counter(),
                                     nv.nvmlDeviceGetClockInfo(self.h, nv.NVML_CLOCK_SM),
                                     int(get_reasons(self.h))))
            except Exception:
                pass
            self.stop_flag.wait(self.period)

    def start(self):
        self.thread = threading.Thread(target=self._run, daemon=True)
        self.thread.start()

    def stop(self, window=None):
        """Summary of the samples taken inside `window` (perf_counter start, end), or of all."""
        self.stop_flag.set()
        if self.thread is not None:
            self.thread.join(timeout=5)
        samples = [x for x in self.samples
                   if window is None or window[0] <= x[0] <= window[1]]
        if not samples:
            return None
        sm = [float(c) for _, c, _ in samples]
        reasons = sorted({name for _, _, bits in samples
                          for name, bit in self.REASONS.items() if bits & bit})
        return {"sm_mhz": statistics.median(sm), "sm_max_mhz": float(self.max_mhz),
                "reasons": reasons, "samples": len(sm), "source": "nvml, 10 ms"}


def make_clock_sampler(device_index: int):
    try:
        return NvmlClockSampler(device_index)
    except Exception:
        return ClockSampler(device_index)


def clocked(fn, device_index: int):
    """Runs fn() with the SM clock sampled meanwhile: (fn's result, median SM MHz or None).
    Kernels that are latency-bound (the masked forward, the small configs) scale with it."""
    sampler = make_clock_sampler(device_index)
    sampler.start()
    res = fn()
    c = sampler.stop()
    return res, (c or {}).get("sm_mhz")


def reduce_max(value: float, device) -> float:
    """Max of `value` over all ranks (identity without a process group)."""
    if not (torch.distributed.is_available() and torch.distributed.is_initialized()):
        return float(value)
    t = torch.tensor([float(value)], dtype=torch.float64, device=device)
    torch.distributed.all_reduce(t, op=torch.distributed.ReduceOp.MAX)
    return float(t.item())


def dist_env():
    ws = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    return ws, rank, local


def workload_desc(name, r, m) -> str:
    return (f"{name}: E={r.E} T={r.T} K={r.K} N={r.N} bf16 (fwd+dgrad+wgrad) + masked "
            f"E={m.E} mmax={m.mmax} K={m.K} N={m.N} fwd")


def make_inputs(workload: str, device):
    import workloads
    r = workloads.make_ragged(workload, tail=0, device=device)
    m = workloads.make_masked(device=device)
    return r, m


def oracle_sample_step(r, m, host, rows_per_group: int, k_per_expert: int, threads: int):
    """One bounded oracle step: forward/dgrad on sampled rows, wgrad on sampled K rows,
    masked forward on all its rows. Returns (flops, seconds)."""
    import oracle
    A, W, dY = host["A"], host["W"], host["dY"]
    rng = np.random.default_rng(0)
    starts, ends, _ = oracle.group_bounds(r.offs, r.rows_alloc)
    rows = np.concatenate([rng.integers(s, t, rows_per_group) for s, t in zip(starts, ends)
                           if t > s]).astype(np.int64)
    ks = np.sort(rng.choice(r.K, k_per_expert, replace=False)).astype(np.int64)
    t0 = time.perf_counter()
    oracle.forward(A, W, r.offs, rows=rows, threads=threads)
    oracle.dgrad(dY, W, r.offs, rows=rows, threads=threads)
    oracle.wgrad(A, dY, r.offs, ks=ks, threads=threads)
    oracle.masked_forward(host["mA"], host["mW"], m.masked_m, threads=threads)
    dt = time.perf_counter() - t0
    flops = (2 * 2 * len(rows) * r.K * r.N + 2 * int(r.sizes.sum()) * len(ks) * r.N
             + m.flops)
    sample = (f"forward+dgrad on {rows_per_group} random rows per group, wgrad on "
              f"{k_per_expert} random K rows of every expert, full masked forward")
    return flops, dt, sample


def host_copies(r, m):
    import oracle
    return {"A": oracle.as_u16(r.A), "W": oracle.as_u16(r.W), "dY": oracle.as_u16(r.dY),
            "mA": oracle.as_u16(m.A), "mW": oracle.as_u16(m.W)}


def run_reference(args):
    ws, rank, _ = dist_env()
    if rank != 0:
        return 0
    import oracle
    threads = oracle.default_threads()
    r, m = make_inputs(args.workload, "cpu")
    host = host_copies(r, m)
    for _ in range(args.warmup):
        oracle_sample_step(r, m, host, 16, 8, threads)
    flops = secs = 0.0
    sample = ""
    for _ in range(args.steps):
        f, dt, sample = oracle_sample_step(r, m, host, 16, 8, threads)
        flops += f
        secs += dt
    value = flops / secs / 1e12
    line = {
        "impl": "reference", "metric": METRIC, "value": value, "unit": UNIT,
        "n_gpus": ws, "steps": args.steps, "warmup": args.warmup,
        "ms_per_step": 1e3 * secs / max(args.steps, 1), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "f64", "data": "synthetic",
        "config": {"workload": workload_desc(args.workload, r, m), "parallelism": "cpu oracle"},
        "cpu_baseline": {"value": value, "unit": UNIT, "cores": threads, "kind": "oracle",
                         "sample": sample},
        "e2e": {"value": value, "unit": UNIT, "h2d_bytes_per_step": 0,
                "d2h_bytes_per_step": 0},
    }
    print(json.dumps(line), flush=True)
    return 0


def run_ours(args):
    import moe_grouped_gemm_ragged_b200 as gg

    ws, rank, local = dist_env()
    if not torch.cuda.is_available():
        raise SystemExit("bench.py needs a CUDA device (there is no CPU implementation)")
    torch.cuda.set_device(local)
    dev = torch.device("cuda", local)
    if ws > 1:
        import datetime
        torch.distributed.init_process_group("nccl", timeout=datetime.timedelta(seconds=120),
                                             device_id=dev)

    def barrier():
        if ws > 1:
            torch.distributed.barrier()

    gg.testing_force_variant(args.variant)
    r, m = make_inputs(args.workload, dev)
    rows, K, N, E = r.rows_alloc, r.K, r.N, r.E
    offs = torch.from_numpy(r.offs).to(dev)
    mm = torch.from_numpy(m.masked_m).to(dev)
    out = torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
    dX = torch.empty((rows, K), dtype=torch.bfloat16, device=dev)
    dW = torch.empty((E, K, N), dtype=torch.bfloat16, device=dev)
    mout = torch.empty((m.E, m.mmax, m.N), dtype=torch.bfloat16, device=dev)
    status = torch.zeros(4, dtype=torch.int32, device=dev)
    stream = torch.cuda.current_stream(dev)

    passes = ["forward", "dgrad", "wgrad", "masked"]
    pass_flops = [r.flops, r.flops, r.flops, m.flops]
    step_flops = sum(pass_flops)

    def step(evs=None):
        if evs is not None:
            evs[0].record(stream)
        gg.forward(r.A, r.W, offs, out, status=status[0:1])
        if evs is not None:
            evs[1].record(stream)
        gg.dgrad(r.dY, r.W, offs, dX, status=status[1:2])
        if evs is not None:
            evs[2].record(stream)
        gg.wgrad(r.A, r.dY, offs, dW, status=status[2:3])
        if evs is not None:
            evs[3].record(stream)
        gg.masked_forward(m.A, m.W, mm, mout, status=status[3:4])
        if evs is not None:
            evs[4].record(stream)

    # NVML samples carry timestamps, so the sampler runs from before the warm-up and only the
    # samples inside the timed region are kept (no idle gap before the timed steps)
    sampler = make_clock_sampler(local)
    sampler.start()
    for _ in range(args.warmup):
        step()
    torch.cuda.synchronize()
    st = status.cpu().numpy()
    if np.any(st & gg.DEV_ERROR_MASK) or not np.all(st & gg.DEV_LAUNCHED):
        raise SystemExit(f"kernel status after warm-up: {[hex(x) for x in st]}")

    evs = [[torch.cuda.Event(enable_timing=True) for _ in range(5)] for _ in range(args.steps)]
    barrier()
    torch.cuda.synchronize()
    w0 = time.perf_counter()
    t_start = torch.cuda.Event(enable_timing=True)
    t_end = torch.cuda.Event(enable_timing=True)
    t_start.record(stream)
    for i in range(args.steps):
        step(evs[i])
    t_end.record(stream)
    torch.cuda.synchronize()
    w1 = time.perf_counter()
    barrier()
    clocks = sampler.stop(window=(w0, w1))
    total_ms = t_start.elapsed_time(t_end)
    per_pass_ms = [sum(evs[i][j].elapsed_time(evs[i][j + 1]) for i in range(args.steps))
                   / args.steps for j in range(4)]
    total_ms = reduce_max(total_ms, dev)
    ms_per_step = total_ms / args.steps
    value = ws * step_flops / (ms_per_step * 1e-3) / 1e12

    extras = None
    peaks, peak_src = load_peaks()
    if not args.no_extras:
        extras = run_extras(args, gg, r, dev, stream, offs, out, dW)
        extras["masked"] = masked_timings(gg, m, dev, peaks)
        extras["masked"]["ms_in_step"] = per_pass_ms[3]
        extras["tiny_forward_call"] = tiny_call_costs(gg, dev)
        if ws == 1:
            extras["configs"] = run_config_extras(gg, dev, stream, peaks,
                                                  reps=max(5, args.steps))

    # end to end through the public API: pinned host inputs -> device, all passes, results
    # back to pinned host memory, every step inside the timed region
    e2e = None
    if not args.no_e2e:
        e2e = run_e2e(args, gg, r, m, dev, stream, ws, barrier)

    dom = int(np.argmax(per_pass_ms[:3]))
    dom_tflops = pass_flops[dom] / (per_pass_ms[dom] * 1e-3) / 1e12
    peak_sus = peaks.get("bf16_tflops_sustained", peaks["bf16_tflops"])
    traffic = None
    if NCU_TRAFFIC_SRC_HASH == kernel_source_hash():
        traffic = NCU_TRAFFIC.get((passes[dom], args.workload))
    roofline = {"bound": "tensor", "kernel": f"grouped_gemm_kernel<{passes[dom]}>",
                "achieved": dom_tflops, "peak": peak_sus, "unit": "TFLOP/s",
                "frac": dom_tflops / peak_sus, "traffic": traffic,
                "peak_kind": f"bf16_tflops_sustained ({peak_src}): the kernel runs inside a "
                             "seconds-long back-to-back timed region",
                "frac_of_burst_peak": dom_tflops / peaks["bf16_tflops"],
                "frac_of_spec_2250": dom_tflops / 2250.0}

    cpu = None
    if rank == 0 and not args.no_cpu:
        import oracle
        threads = oracle.default_threads()
        host = host_copies(r, m)
        f, dt, sample = oracle_sample_step(r, m, host, 32, 16, threads)
        cpu = {"value": f / dt / 1e12, "unit": UNIT, "cores": threads, "kind": "oracle",
               "sample": sample, "seconds": dt}

    if rank == 0:
        line = {
            "metric": METRIC, "value": value, "unit": UNIT, "n_gpus": ws,
            "steps": args.steps, "warmup": args.warmup, "ms_per_step": ms_per_step,
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
            "dtype": "bf16", "data": "synthetic",
            "config": {
                "workload": workload_desc(args.workload, r, m),
                "group_sizes": f"min {int(r.sizes.min())} max {int(r.sizes.max())}",
                "l2": "inputs (>6 GB) exceed the 126 MB L2; no flush",
                "parallelism": f"ep{ws} (independent per-GPU experts)",
            },
            "passes": {p: {"ms": per_pass_ms[j],
                           "tflops": pass_flops[j] / (per_pass_ms[j] * 1e-3) / 1e12}
                       for j, p in enumerate(passes)},
            "roofline": roofline,
            "cpu_baseline": cpu,
            "e2e": e2e,
            "extras": extras,
            "gpu_launches": 4 * args.steps,
            "clocks": clocks,
        }
        print(json.dumps(line), flush=True)
    if ws > 1:
        torch.distributed.destroy_process_group()
    return 0


def run_extras(args, gg, r, dev, stream, offs, out, dW):
    """The further operations of the library on the same workload, each timed on its own
    (outside the step): fp32 wgrad accumulating into a main-grad buffer (beta=1), forward
    with per-expert bias and per-token bias scale, and forward with SiLU-and-mul."""
    reps = max(3, args.steps // 2)
    gen = torch.Generator(device=dev).manual_seed(11)
    bias = torch.randn(r.E, r.N, generator=gen, device=dev).to(torch.bfloat16)
    scale = torch.rand(r.rows_alloc, generator=gen, device=dev)
    dw32 = torch.zeros((r.E, r.K, r.N), dtype=torch.float32, device=dev)
    ops = {
        "wgrad_f32_accumulate": lambda: gg.wgrad_f32(r.A, r.dY, offs, dw32, alpha=1.0, beta=1.0),
        "forward_bias_scale": lambda: gg.forward_ex(r.A, r.W, offs, out, bias=bias,
                                                    bias_scale=scale),
    }
    if r.N % 256 == 0:
        act_out = torch.empty((r.rows_alloc, r.N // 2), dtype=torch.bfloat16, device=dev)
        ops["forward_silu_mul"] = lambda: gg.forward_ex(r.A, r.W, offs, act_out, bias=bias,
                                                        act=gg.ACT_SILU_MUL)
    # token routing that would produce this workload's packed rows: T/8 tokens, top-8
    tok = max(1, r.T // 8)
    ids_np, X = __import__("workloads").make_routing(tok, 8, r.E, r.K, seed=12, device=dev) \
        if tok <= 65536 else (None, None)
    route_bytes = None
    if ids_np is not None:
        ids = torch.from_numpy(ids_np).to(dev)
        a_packed = torch.empty((tok * 8, r.K), dtype=torch.bfloat16, device=dev)
        row_of = torch.empty(tok * 8, dtype=torch.int32, device=dev)
        roffs = torch.empty(r.E, dtype=torch.int32, device=dev)
        ws = torch.empty(max(4, gg.route_workspace_bytes(tok * 8, r.E)), dtype=torch.uint8,
                         device=dev)
        ops["route_tokens"] = lambda: gg.route(ids, X, r.E, A_packed=a_packed, row_of=row_of,
                                               offs=roffs, workspace=ws)
        # ids + X once + packed rows + row_of + offsets
        route_bytes = (ids.numel() * 4 + X.numel() * 2 + a_packed.numel() * 2
                       + row_of.numel() * 4 + r.E * 4)
    res = {}
    for name, fn in ops.items():
        fn()
        torch.cuda.synchronize()
        e0 = torch.cuda.Event(enable_timing=True)
        e1 = torch.cuda.Event(enable_timing=True)
        e0.record(stream)
        for _ in range(reps):
            fn()
        e1.record(stream)
        torch.cuda.synchronize()
        ms = e0.elapsed_time(e1) / reps
        if name == "route_tokens":
            res[name] = {"ms": ms, "gbs": route_bytes / (ms * 1e-3) / 1e9,
                         "tokens": tok, "topk": 8, "launches": 3 * reps}
        else:
            res[name] = {"ms": ms, "tflops": r.flops / (ms * 1e-3) / 1e12, "launches": reps}
    return res


def run_config_extras(gg, dev, stream, peaks, reps: int):
    """Forward, dgrad and wgrad of the other ragged configs (gate-up E=64 Zipf, down-proj E=32,
    the large shape with unaligned sizes), each pass timed on its own outside the step: median
    of per-call CUDA-event times of `reps` back-to-back calls after 3 warm-up calls."""
    import workloads
    res = {}
    for name in ("gateup", "downproj", "large_unaligned"):
        r = workloads.make_ragged(name, tail=0, device=dev)
        offs = torch.from_numpy(r.offs).to(dev)
        out = torch.empty((r.rows_alloc, r.N), dtype=torch.bfloat16, device=dev)
        dX = torch.empty((r.rows_alloc, r.K), dtype=torch.bfloat16, device=dev)
        dW = torch.empty((r.E, r.K, r.N), dtype=torch.bfloat16, device=dev)
        fns = {"forward": lambda: gg.forward(r.A, r.W, offs, out),
               "dgrad": lambda: gg.dgrad(r.dY, r.W, offs, dX),
               "wgrad": lambda: gg.wgrad(r.A, r.dY, offs, dW)}
        entry = {"E": r.E, "T": r.T, "K": r.K, "N": r.N, "flops_per_pass": r.flops,
                 "group_sizes": f"min {int(r.sizes.min())} max {int(r.sizes.max())}, "
                                f"{int((r.sizes == 0).sum())} empty"}
        for pas, fn in fns.items():
            ms, mhz = clocked(lambda: _median_call_ms(fn, stream, reps), dev.index)
            tf = r.flops / (ms * 1e-3) / 1e12
            entry[pas] = {"ms": ms, "tflops": tf, "frac_of_burst": tf / peaks["bf16_tflops"],
                          "sm_mhz": mhz}
        res[name] = entry
        del r, offs, out, dX, dW, fns
        torch.cuda.empty_cache()
    return res


def masked_timings(gg, m, dev, peaks, copies: int = 16, rounds: int = 12):
    """Per-call time of the masked forward replayed from a CUDA graph: `hot` calls reuse one
    set of inputs (the weights stay in L2), `cold` calls cycle through `copies` sets of inputs
    (copies x 25 MB, above the 126 MB L2), so every call reads its weights from HBM."""
    mm = torch.from_numpy(m.masked_m).to(dev)
    As = [m.A] + [m.A.clone() for _ in range(copies - 1)]
    Ws = [m.W] + [m.W.clone() for _ in range(copies - 1)]
    outs = [torch.empty((m.E, m.mmax, m.N), dtype=torch.bfloat16, device=dev)
            for _ in range(copies)]
    side = torch.cuda.Stream(device=dev)

    def per_call_us(seq):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for i in seq:
                gg.masked_forward(As[i], Ws[i], mm, outs[i])
        g.replay()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        cur = torch.cuda.current_stream(dev)
        a.record(cur)
        g.replay()
        b.record(cur)
        torch.cuda.synchronize()
        del g
        return a.elapsed_time(b) * 1e3 / len(seq)

    def single_after_us(dirty: bool, reps: int = 20):
        """One eager call (event to event) right after a 256 MB pass that leaves L2 full of
        clean lines (a read) or of dirty ones (a write, as the output stores of a preceding
        GEMM do): with dirty lines every line the call brings in first writes one back."""
        buf = torch.empty(256 << 20, dtype=torch.uint8, device=dev)
        acc = torch.empty((), dtype=torch.int64, device=dev)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        ts = []
        for r in range(reps):
            if dirty:
                buf.fill_(r & 0xFF)
            else:
                torch.sum(buf.view(torch.int64), dim=0, out=acc)
            i = r % copies
            a.record()
            gg.masked_forward(As[i], Ws[i], mm, outs[i])
            b.record()
            torch.cuda.synchronize()
            ts.append(a.elapsed_time(b) * 1e3)
        del buf
        return float(np.median(ts))

    gg.masked_forward(As[0], Ws[0], mm, outs[0])
    torch.cuda.synchronize()
    hot, hot_mhz = clocked(lambda: float(np.median([per_call_us([0] * 200)
                                                    for _ in range(3)])), dev.index)
    cold, cold_mhz = clocked(lambda: float(np.median([per_call_us(list(range(copies)) * rounds)
                                                      for _ in range(3)])), dev.index)
    after_clean = single_after_us(False)
    after_dirty = single_after_us(True)
    nbytes = masked_bytes(m)
    return {"algorithmic_bytes": nbytes, "hot_graph_us": hot, "cold_graph_us": cold,
            "cold_gbs": nbytes / (cold * 1e-6) / 1e9,
            "cold_frac_of_hbm": nbytes / (cold * 1e-6) / 1e9 / peaks["hbm_gbs"],
            "hot_gbs": nbytes / (hot * 1e-6) / 1e9,
            "hot_sm_mhz": hot_mhz, "cold_sm_mhz": cold_mhz,
            "single_after_clean_l2_us": after_clean,
            "single_after_dirty_l2_us": after_dirty,
            "kernel": "masked_forward_kernel (weight columns as the MMA's M)"}


def tiny_call_costs(gg, dev, calls: int = 2000):
    """Cost of one call of the tiny forward (4 experts, A[48, 8], offsets (8,16,32,40)), the
    shape where the host launch dominates: host time per call through the Python binding and
    through the C ABI alone (ctypes, arguments prepared once), CUDA-event time per call of
    back-to-back calls, and the per-call time of calls replayed from a CUDA graph."""
    import time as _t
    import workloads
    r = workloads.make_tiny((8, 16, 32, 40))
    A, W = r.A.to(dev), r.W.to(dev)
    offs = torch.from_numpy(np.ascontiguousarray(r.offs)).to(dev)
    out = torch.empty((r.rows_alloc, r.N), dtype=torch.bfloat16, device=dev)
    stream = torch.cuda.current_stream(dev)
    fn = lambda: gg.forward(A, W, offs, out)  # noqa: E731
    L = gg.lib()
    cargs = (A.data_ptr(), W.data_ptr(), offs.data_ptr(), out.data_ptr(), r.rows_alloc, r.K,
             r.N, r.E, None, stream.cuda_stream)
    cfn = L.gg_forward

    def host_us(f):
        for _ in range(50):
            f()
        torch.cuda.synchronize()
        t0 = _t.perf_counter()
        for _ in range(calls):
            f()
        t1 = _t.perf_counter()
        torch.cuda.synchronize()
        return (t1 - t0) * 1e6 / calls

    py = host_us(fn)
    cabi = host_us(lambda: cfn(*cargs))
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record(stream)
    for _ in range(calls):
        cfn(*cargs)
    e1.record(stream)
    torch.cuda.synchronize()
    return {"host_us_python_binding": py, "host_us_c_abi": cabi,
            "event_us_back_to_back_c_abi": e0.elapsed_time(e1) * 1e3 / calls,
            "graph_us": _graph_call_us(fn, stream, 200), "calls": calls}


def run_e2e(args, gg, r, m, dev, stream, ws, barrier):
    steps = max(1, min(args.steps, args.e2e_steps))
    hA = r.A.cpu().pin_memory()
    hW = r.W.cpu().pin_memory()
    hdY = r.dY.cpu().pin_memory()
    hoffs = torch.from_numpy(r.offs).pin_memory()
    hmA, hmW = m.A.cpu().pin_memory(), m.W.cpu().pin_memory()
    hmm = torch.from_numpy(m.masked_m).pin_memory()
    rows, K, N, E = r.rows_alloc, r.K, r.N, r.E
    dA = torch.empty_like(r.A)
    dWt = torch.empty_like(r.W)
    ddY = torch.empty_like(r.dY)
    doffs = torch.empty(E, dtype=torch.int32, device=dev)
    dmA, dmW = torch.empty_like(m.A), torch.empty_like(m.W)
    dmm = torch.empty(m.E, dtype=torch.int32, device=dev)
    out = torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
    dX = torch.empty((rows, K), dtype=torch.bfloat16, device=dev)
    dW = torch.empty((E, K, N), dtype=torch.bfloat16, device=dev)
    mout = torch.empty((m.E, m.mmax, m.N), dtype=torch.bfloat16, device=dev)
    hout = torch.empty(out.shape, dtype=out.dtype).pin_memory()
    hdX = torch.empty(dX.shape, dtype=dX.dtype).pin_memory()
    hdW = torch.empty(dW.shape, dtype=dW.dtype).pin_memory()
    hmout = torch.empty(mout.shape, dtype=mout.dtype).pin_memory()
    # bytes the step moves: the rows inside the groups (T of them), all of W and dW, offsets
    T = r.T
    nb = lambda t: t.numel() * t.element_size()
    h2d = (T * (K + N) * 2 + nb(hW) + nb(hoffs) + nb(hmA) + nb(hmW) + nb(hmm))
    d2h = T * (N + K) * 2 + nb(hdW) + nb(hmout)

    staging = {"A": dA, "W": dWt, "dY": ddY, "offs": doffs, "out": out, "dX": dX, "dW": dW}

    def step():
        # the ragged passes through the host-buffer entry point (expert chunks, copies both
        # ways overlapped with the GEMMs), then the masked call with its own copies
        gg.layer_step_host(hA, hW, hdY, hoffs, hout, hdX, hdW, staging, chunks=args.e2e_chunks)
        for d, h in ((dmA, hmA), (dmW, hmW), (dmm, hmm)):
            d.copy_(h, non_blocking=True)
        gg.masked_forward(dmA, dmW, dmm, mout)
        hmout.copy_(mout, non_blocking=True)

    step()
    torch.cuda.synchronize()
    barrier()
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    e0.record(stream)
    for _ in range(steps):
        step()
    e1.record(stream)
    torch.cuda.synchronize()
    barrier()
    ms = reduce_max(e0.elapsed_time(e1) / steps, dev)
    flops = 3 * r.flops + m.flops
    return {"value": ws * flops / (ms * 1e-3) / 1e12, "unit": UNIT, "ms_per_step": ms,
            "steps": steps, "h2d_bytes_per_step": h2d, "d2h_bytes_per_step": d2h,
            "api": "gg_layer_step_host + gg_masked_forward",
            "expert_chunks": args.e2e_chunks or 16}


def _median_call_ms(fn, stream, calls: int) -> float:
    """Median of per-call CUDA-event times on ``stream`` after 3 warm-up calls."""
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
          for _ in range(calls)]
    for a, b in ev:
        a.record(stream)
        fn()
        b.record(stream)
    torch.cuda.synchronize()
    return float(np.median([a.elapsed_time(b) for a, b in ev]))


def _graph_call_us(fn, stream, calls: int) -> float:
    """Per-call time of ``calls`` launches captured in one CUDA graph and replayed."""
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        for _ in range(calls):
            fn()
    g.replay()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    cur = torch.cuda.current_stream()
    a.record(cur)
    g.replay()
    b.record(cur)
    torch.cuda.synchronize()
    del g
    return a.elapsed_time(b) * 1e3 / calls


def masked_bytes(m) -> int:
    """Algorithmic bytes of the masked forward: active rows of A read once, W of the experts
    with at least one active row read once, active output rows written once."""
    act = np.clip(np.asarray(m.masked_m, np.int64), 0, m.mmax)
    return int(act.sum() * (m.K + m.N) * 2 + (act > 0).sum() * m.K * m.N * 2)


def run_table(args):
    """Per-config, per-pass measurement of every parity config: GPU time (median of 20
    calls; 200 for the tiny and masked shapes, which also report graph-replayed per-call
    time), TFLOP/s and algorithmic GB/s, and the oracle's time on the host cores (in full
    for tiny, masked and gate-up; on a row / K-row sample, extrapolated, for the others).
    One JSON line per (config, pass)."""
    import oracle
    import workloads
    import moe_grouped_gemm_ragged_b200 as gg
    if not torch.cuda.is_available():
        raise SystemExit("bench.py needs a CUDA device (there is no CPU implementation)")
    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream()
    peaks, _ = load_peaks()
    threads = oracle.default_threads()

    def emit(cfg, pas, flops, nbytes, ms, oracle_s, oracle_note, graph_us=None):
        line = {"config": cfg, "pass": pas, "flops": flops, "algorithmic_bytes": nbytes,
                "gpu_ms": ms, "tflops": flops / (ms * 1e-3) / 1e12,
                "frac_of_burst_peak": flops / (ms * 1e-3) / 1e12 / peaks["bf16_tflops"],
                "frac_of_spec_2250": flops / (ms * 1e-3) / 1e12 / 2250.0,
                "gbs": nbytes / (ms * 1e-3) / 1e9,
                "frac_of_hbm": nbytes / (ms * 1e-3) / 1e9 / peaks["hbm_gbs"],
                "graph_us_per_call": graph_us, "oracle_s": oracle_s,
                "oracle_note": oracle_note, "oracle_threads": threads}
        print(json.dumps(line), flush=True)

    def ragged_bytes(r, pas):
        T, K, N = r.T, r.K, r.N
        live = int((np.asarray(r.sizes) > 0).sum())
        w = live * K * N * 2
        if pas == "forward":
            return T * K * 2 + w + T * N * 2
        if pas == "dgrad":
            return T * N * 2 + w + T * K * 2
        return T * (K + N) * 2 + r.E * K * N * 2

    cases = [("tiny (8,16,32,40)", workloads.make_tiny((8, 16, 32, 40))),
             ("tiny (8,8,32,40)", workloads.make_tiny((8, 8, 32, 40)))]
    cases += [(n, None) for n in ("gateup", "downproj", "large", "large_unaligned")]
    for cfg, r in cases:
        if r is None:
            r = workloads.make_ragged(cfg, tail=0, device=dev)
        small = cfg.startswith("tiny")
        A, W, dY = (t.to(dev) for t in (r.A, r.W, r.dY))
        offs = torch.from_numpy(np.ascontiguousarray(r.offs)).to(dev)
        out = torch.empty((r.rows_alloc, r.N), dtype=torch.bfloat16, device=dev)
        dX = torch.empty((r.rows_alloc, r.K), dtype=torch.bfloat16, device=dev)
        dW = torch.empty((r.E, r.K, r.N), dtype=torch.bfloat16, device=dev)
        fns = {"forward": lambda: gg.forward(A, W, offs, out),
               "dgrad": lambda: gg.dgrad(dY, W, offs, dX),
               "wgrad": lambda: gg.wgrad(A, dY, offs, dW)}
        hA, hW, hdY = oracle.as_u16(A), oracle.as_u16(W), oracle.as_u16(dY)
        full = cfg.startswith("tiny") or cfg == "gateup"
        rng = np.random.default_rng(0)
        starts, ends, _ = oracle.group_bounds(r.offs, r.rows_alloc)
        rows = None if full else np.concatenate(
            [rng.integers(s, t, 16) for s, t in zip(starts, ends) if t > s]).astype(np.int64)
        ks = None if full else np.sort(rng.choice(r.K, 8, replace=False)).astype(np.int64)
        for pas, fn in fns.items():
            ms = _median_call_ms(fn, stream, 200 if small else 20)
            gus = _graph_call_us(fn, stream, 200) if small else None
            t0 = time.perf_counter()
            if pas == "forward":
                oracle.forward(hA, hW, r.offs, rows=rows, threads=threads)
            elif pas == "dgrad":
                oracle.dgrad(hdY, hW, r.offs, rows=rows, threads=threads)
            else:
                oracle.wgrad(hA, hdY, r.offs, ks=ks, threads=threads)
            osec = time.perf_counter() - t0
            note = "full pass"
            if not full:
                frac = (len(rows) / max(1, r.T)) if pas != "wgrad" else len(ks) / r.K
                osec /= frac
                note = (f"extrapolated from {len(rows)} sampled rows" if pas != "wgrad"
                        else f"extrapolated from {len(ks)} sampled K rows")
            emit(cfg, pas, r.flops, ragged_bytes(r, pas), ms, osec, note, gus)
        del A, W, dY, out, dX, dW
        torch.cuda.empty_cache()

    m = workloads.make_masked(device=dev)
    mA, mW = m.A.to(dev), m.W.to(dev)
    mm = torch.from_numpy(m.masked_m).to(dev)
    mout = torch.empty((m.E, m.mmax, m.N), dtype=torch.bfloat16, device=dev)
    fn = lambda: gg.masked_forward(mA, mW, mm, mout)  # noqa: E731
    ms = _median_call_ms(fn, stream, 200)
    mt = masked_timings(gg, m, dev, peaks)
    t0 = time.perf_counter()
    oracle.masked_forward(oracle.as_u16(mA), oracle.as_u16(mW), m.masked_m, threads=threads)
    osec = time.perf_counter() - t0
    # graph-replayed per call with the weights read from HBM (16 rotating input copies)
    emit("masked", "forward", m.flops, masked_bytes(m), ms, osec, "full pass",
         mt["cold_graph_us"])
    print(json.dumps({"config": "masked", "pass": "forward", "graph_timings": mt}), flush=True)
    print(json.dumps({"config": "tiny (8,16,32,40)", "pass": "forward",
                      "call_costs": tiny_call_costs(gg, dev)}), flush=True)
    return 0


def run_launch_only(args):
    """Launch the chosen passes of one workload `--reps` times each, in order, untimed: the
    command that `ncu` captures (select the launch with -k / -s / -c). Workloads: the ragged
    configs of --workload, or "tiny" (4 experts, offsets (8,16,32,40)), "masked" (the
    sglang shape) and "route" (the token routing of the large shape's rows: 32768 tokens,
    top-8 of 16 experts, K=6144; pass "route")."""
    import workloads
    import moe_grouped_gemm_ragged_b200 as gg
    if not torch.cuda.is_available():
        raise SystemExit("bench.py needs a CUDA device (there is no CPU implementation)")
    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    passes = args.passes.split(",")
    if args.workload == "masked":
        m = workloads.make_masked(device=dev)
        mm = torch.from_numpy(m.masked_m).to(dev)
        mout = torch.empty((m.E, m.mmax, m.N), dtype=torch.bfloat16, device=dev)
        fns = {"masked": lambda: gg.masked_forward(m.A, m.W, mm, mout)}
    elif args.workload == "route":
        tok, k, E, K = 32768, 8, 16, 6144
        ids_np, X = workloads.make_routing(tok, k, E, K, seed=12, device=dev)
        ids = torch.from_numpy(ids_np).to(dev)
        a_packed = torch.empty((tok * k, K), dtype=torch.bfloat16, device=dev)
        row_of = torch.empty(tok * k, dtype=torch.int32, device=dev)
        roffs = torch.empty(E, dtype=torch.int32, device=dev)
        wsp = torch.empty(max(4, gg.route_workspace_bytes(tok * k, E)), dtype=torch.uint8,
                          device=dev)
        fns = {"route": lambda: gg.route(ids, X, E, A_packed=a_packed, row_of=row_of,
                                         offs=roffs, workspace=wsp)}
    else:
        r = (workloads.make_tiny((8, 16, 32, 40)) if args.workload == "tiny"
             else workloads.make_ragged(args.workload, tail=0, device=dev))
        A, W, dY = (t.to(dev) for t in (r.A, r.W, r.dY))
        offs = torch.from_numpy(np.ascontiguousarray(r.offs)).to(dev)
        out = torch.empty((r.rows_alloc, r.N), dtype=torch.bfloat16, device=dev)
        dX = torch.empty((r.rows_alloc, r.K), dtype=torch.bfloat16, device=dev)
        dW = torch.empty((r.E, r.K, r.N), dtype=torch.bfloat16, device=dev)
        fns = {"forward": lambda: gg.forward(A, W, offs, out),
               "dgrad": lambda: gg.dgrad(dY, W, offs, dX),
               "wgrad": lambda: gg.wgrad(A, dY, offs, dW)}
    for p in passes:
        if p not in fns:
            raise SystemExit(f"pass {p!r} is not one of {sorted(fns)} for {args.workload}")
    torch.cuda.synchronize()
    for _ in range(args.reps):
        for p in passes:
            fns[p]()
    torch.cuda.synchronize()
    print(f"launched {args.reps} x {passes} on {args.workload}", flush=True)
    return 0


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--warmup", type=int, default=3)
    ap.add_argument("--impl", choices=["ours", "reference"], default="ours")
    ap.add_argument("--workload", default="large",
                    choices=["large", "large_unaligned", "gateup", "downproj", "large_e2",
                             "tiny", "masked", "route"],
                    help="tiny, masked and route: with --launch-only")
    ap.add_argument("--e2e-steps", type=int, default=3)
    ap.add_argument("--e2e-chunks", type=int, default=0,
                    help="expert chunks of the host-buffer pass (0: the library default)")
    ap.add_argument("--no-e2e", action="store_true")
    ap.add_argument("--no-cpu", action="store_true")
    ap.add_argument("--no-extras", action="store_true")
    ap.add_argument("--variant", type=int, default=0, choices=[0, 1, 2, 3],
                    help="launch shapes: 0 automatic, 1 single CTA, 2 CTA pair, 3 CTA pair with 256 x 512 wgrad tiles")
    ap.add_argument("--table", action="store_true",
                    help="per-config, per-pass table of every parity config (JSON lines)")
    ap.add_argument("--launch-only", action="store_true",
                    help="launch --passes of --workload --reps times, untimed (for ncu)")
    ap.add_argument("--passes", default="forward,dgrad,wgrad",
                    help="with --launch-only: forward, dgrad, wgrad (ragged) or masked")
    ap.add_argument("--reps", type=int, default=2, help="with --launch-only")
    args = ap.parse_args(argv)
    if args.launch_only:
        return run_launch_only(args)
    if args.workload in ("tiny", "masked", "route"):
        ap.error("--workload tiny/masked/route needs --launch-only")
    if args.table:
        return run_table(args)
    if args.warmup < 3:
        args.warmup = 3
    if args.impl == "reference":
        return run_reference(args)
    return run_ours(args)


if __name__ == "__main__":
    sys.exit(main())
