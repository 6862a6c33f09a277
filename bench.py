#!/usr/bin/env python
"""Benchmark of the Tail-Replay hot path on B200: rebuild every GDN layer's
state from the last R tokens of the matched prefix, then prefill the suffix.

    python bench.py [--gpus N --steps K --warmup W] [--impl ours|reference]
                    [--workload stack|sweep|varlen|decode|outputs|overlap|fused|hybrid]

One JSON line on stdout (rank 0).  Default workload: the 24-layer stack, 32
heads, d = 128, bf16, matched prefix L = 32768, replay R = 3277 (10%), suffix
N = 1024.  Following the 3:1 interleave (8 groups of 3 GDN layers after full
attention layers), a step runs 3 replay launches of 8 layers each, then 3
suffix-prefill launches of 8 layers.

`value` = replayed prefix tokens per second through the whole stack
(sum over requests of R / the device time of the state rebuild, summed over
ranks); `ms_per_step` is the whole step (rebuild + suffix prefill).  Under
torchrun every rank runs an independent replica ("scaling": "weak"); the only
cross-rank traffic is the timing barrier and the max over ranks.
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
import torch

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

from gated_deltanet_state_tail_b200 import inputs  # noqa: E402

L2_FLUSH_BYTES = 256 << 20
GROUPS, GDN_PER_GROUP = 8, 3     # 24 GDN layers = 8 groups x 3


# --------------------------------------------------------------------------
# distributed plumbing
# --------------------------------------------------------------------------
def dist_init(n_gpus, backend=None):
    """One process per GPU (torchrun env).  NCCL on GPUs; gloo covers the same host
    logic on CPU.  Returns (rank, world, local rank)."""
    world = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    if world > 1:
        import datetime
        if backend is None:
            backend = "nccl" if torch.cuda.is_available() else "gloo"
        if backend == "nccl":
            torch.cuda.set_device(local)
            torch.distributed.init_process_group("nccl", timeout=datetime.timedelta(seconds=120),
                                                 device_id=torch.device("cuda", local))
        else:
            torch.distributed.init_process_group(backend, timeout=datetime.timedelta(seconds=60))
    elif torch.cuda.is_available():
        torch.cuda.set_device(0)
    return rank, world, local


def barrier(world):
    if world > 1:
        torch.distributed.barrier()


def _reduce_device():
    return torch.device("cuda") if torch.distributed.get_backend() == "nccl" else torch.device("cpu")


def max_over_ranks(x, world):
    if world == 1:
        return x
    t = torch.tensor([x], dtype=torch.float64, device=_reduce_device())
    torch.distributed.all_reduce(t, op=torch.distributed.ReduceOp.MAX)
    return float(t.item())


def sum_over_ranks(x, world):
    if world == 1:
        return x
    t = torch.tensor([x], dtype=torch.float64, device=_reduce_device())
    torch.distributed.all_reduce(t, op=torch.distributed.ReduceOp.SUM)
    return float(t.item())


def replica_throughput(replayed_per_rank, world, t_rebuild_max_s):
    """Whole-job replayed tokens/s of `world` independent replicas (no exchange step):
    every rank replays the same count and the job lasts as long as its slowest rank."""
    return replayed_per_rank * world / t_rebuild_max_s


# --------------------------------------------------------------------------
# clocks sampled during the timed region
# --------------------------------------------------------------------------
# NVML clock-event reason bits (nvmlClocksEventReason*)
_REASON_BITS = {"sw_power_cap": 0x4, "hw_slowdown": 0x8, "sw_thermal_slowdown": 0x20,
                "hw_thermal_slowdown": 0x40, "hw_power_brake_slowdown": 0x80}


class ClockSampler:
    """Samples the SM clock and the clock-event reasons through NVML every few
    milliseconds while the timed region runs (a background thread)."""

    def __init__(self, device_index, period_s=0.005):
        self.dev = device_index
        self.period = period_s
        self.samples = []
        self.max_mhz = None
        self._stop = None

    def _handle(self, pynvml):
        try:
            props = torch.cuda.get_device_properties(self.dev)
            uuid = str(props.uuid)
            return pynvml.nvmlDeviceGetHandleByUUID(("GPU-" + uuid) if not uuid.startswith("GPU-") else uuid)
        except Exception:
            return pynvml.nvmlDeviceGetHandleByIndex(self.dev)

    def __enter__(self):
        import threading
        try:
            import pynvml
            pynvml.nvmlInit()
            h = self._handle(pynvml)
            self.max_mhz = float(pynvml.nvmlDeviceGetMaxClockInfo(h, pynvml.NVML_CLOCK_SM))
        except Exception:
            return self
        self._stop = threading.Event()

        def run():
            while not self._stop.is_set():
                try:
                    mhz = pynvml.nvmlDeviceGetClockInfo(h, pynvml.NVML_CLOCK_SM)
                    reasons = pynvml.nvmlDeviceGetCurrentClocksEventReasons(h)
                    self.samples.append((float(mhz), int(reasons)))
                except Exception:
                    pass
                self._stop.wait(self.period)

        self._thread = threading.Thread(target=run, daemon=True)
        self._thread.start()
        return self

    def __exit__(self, *exc):
        if self._stop is not None:
            self._stop.set()
            self._thread.join(timeout=2)

    def summary(self):
        sm = [m for m, _ in self.samples]
        reasons = sorted({name for _, r in self.samples for name, bit in _REASON_BITS.items() if r & bit})
        return {"sm_mhz": statistics.median(sm) if sm else None, "sm_max_mhz": self.max_mhz,
                "reasons": reasons, "samples": len(sm), "source": "NVML, 5 ms period"}


# --------------------------------------------------------------------------
# peaks and profile summaries
# --------------------------------------------------------------------------
def measured_peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        with open(p) as f:
            d = json.load(f)
        return {"hbm_gbs": d["hbm_gbs"], "bf16_tflops": d["bf16_tflops"],
                "bf16_tflops_sustained": d.get("bf16_tflops_sustained"), "source": "measured",
                "sm_max_mhz": d.get("sm_max_mhz", 1965.0)}
    return {"hbm_gbs": 6650.0, "bf16_tflops": 1590.0, "bf16_tflops_sustained": 1400.0,
            "source": "fallback", "sm_max_mhz": 1965.0}


REPLAY_KERNEL_SOURCES = ("gdn_replay.cu", "gdn_chunk_common.h", "gdn_sm100.h", "gdn_internal.h")
# the metric both arms report (ours and the oracle reference arm)
BENCH_METRIC = "GDN tail-replay tokens/s per GPU; state-rebuild latency at 32K prefix"


def kernel_source_sha():
    """Hash of the sources that define the replay kernel (its DRAM traffic record in
    profiles/traffic.txt is used only while this hash matches)."""
    h = hashlib.sha256()
    csrc = os.path.join(ROOT, "gated_deltanet_state_tail_b200", "csrc")
    for name in REPLAY_KERNEL_SOURCES:
        with open(os.path.join(csrc, name), "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


def profiled_traffic(kernel_name, launch_units):
    """DRAM bytes per launch from the committed ncu summary, if it was taken on
    the current kernel sources; scaled by work units if captured on a smaller case."""
    p = os.path.join(ROOT, "profiles", "traffic.txt")
    if not os.path.exists(p):
        return None
    rec = {}
    with open(p) as f:
        for line in f:
            if ":" in line and not line.lstrip().startswith("#"):
                key, val = line.split(":", 1)
                rec[key.strip()] = val.strip()
    if rec.get("kernel") != kernel_name or rec.get("source_sha") != kernel_source_sha():
        return None
    try:
        per_unit = float(rec["dram_bytes"]) / float(rec["units"])
    except (KeyError, ValueError, ZeroDivisionError):
        return None
    return per_unit * launch_units


# --------------------------------------------------------------------------
# workload construction (device-resident inputs)
# --------------------------------------------------------------------------
class StackData:
    """Per-layer buffers of prefix ++ suffix rows, laid out launch-major:
    buffer slot s = j * GROUPS + g holds GDN layer 3g + j (seed = layer id)."""

    def __init__(self, wl, device, compact=False):
        # compact: keep only the replay window and the suffix of each layer
        # (rows [L - R, L + N)); the replay reads exactly the same work, but
        # the full-prefill comparator needs the whole prefix.
        self.wl = wl
        self.layers = wl.layers
        L, N = wl.match_len[0], wl.suffix_len[0]
        if compact:
            L = wl.R[0]
        self.L, self.N, self.R = L, N, wl.R[0]
        self.seq = L + N
        rows = self.layers * self.seq
        H, dk, dv = wl.H, wl.dk, wl.dv
        td = torch.bfloat16 if wl.dtype == "bf16" else torch.float32
        self.q = torch.empty((rows, H, dk), dtype=td, device=device)
        self.k = torch.empty((rows, H, dk), dtype=td, device=device)
        self.v = torch.empty((rows, H, dv), dtype=td, device=device)
        self.alpha = torch.empty((rows, H), dtype=torch.float32, device=device)
        self.beta = torch.empty((rows, H), dtype=torch.float32, device=device)
        self.layer_of_slot = []
        per_launch = self.layers // GDN_PER_GROUP if self.layers % GDN_PER_GROUP == 0 else self.layers
        self.per_launch = per_launch
        for s in range(self.layers):
            j, g = divmod(s, per_launch)
            layer = GDN_PER_GROUP * g + j if per_launch != self.layers else s
            self.layer_of_slot.append(layer)
            t = inputs.draw_tensors(self.seq, H, dk, dv, wl.dtype, wl.alpha_lo, wl.alpha_hi,
                                    seed=wl.seeds[layer], device=device)
            sl = slice(s * self.seq, (s + 1) * self.seq)
            for name in ("q", "k", "v", "alpha", "beta"):
                getattr(self, name)[sl].copy_(t[name])
            del t
        # suffix rows as their own packed buffers (the new tokens of the request)
        idx = torch.cat([torch.arange(s * self.seq + L, (s + 1) * self.seq, device=device)
                         for s in range(self.layers)])
        self.sq, self.sk, self.sv = self.q[idx], self.k[idx], self.v[idx]
        self.sa, self.sb = self.alpha[idx], self.beta[idx]
        self.launches = [list(range(j * per_launch, (j + 1) * per_launch))
                         for j in range(self.layers // per_launch)]

    def replay_desc(self, slots):
        off = np.array([s * self.seq for s in slots] + [(slots[-1] + 1) * self.seq], np.int32)
        return off, np.full(len(slots), self.L, np.int32), np.full(len(slots), self.R, np.int32)

    def suffix_cu(self, slots):
        return np.array([s * self.N for s in slots] + [(slots[-1] + 1) * self.N], np.int32)


def build_stack_runner(data, kernel):
    """Plans and buffers for the cache-hit step of the layer stack."""
    import gated_deltanet_state_tail_b200 as gdn
    wl = data.wl
    H, dk, dv = wl.H, wl.dk, wl.dv
    rp, pp = [], []
    for slots in data.launches:
        off, ml, R = data.replay_desc(slots)
        rp.append(gdn.ReplayPlan(H, dk, dv, wl.dtype, off, ml, R, kernel))
        pp.append(gdn.PrefillPlan(H, dk, dv, wl.dtype, data.suffix_cu(slots), kernel))
    n_launch = len(data.launches)
    state = torch.empty((data.layers, H, dk, dv), dtype=torch.float32, device="cuda")
    o = torch.empty((data.layers * data.N, H, dv), dtype=data.k.dtype, device="cuda")
    st_out = torch.empty_like(state)
    return rp, pp, state, o, st_out, n_launch


def run_step(data, rp, pp, state, o, st_out, events=None, launch_events=None):
    """One cache-hit step: replay every layer's tail, then prefill every suffix."""
    per = data.per_launch
    if events:
        events[0].record()
    for j, plan in enumerate(rp):
        sl = slice(j * per, (j + 1) * per)
        if launch_events is not None:
            launch_events[j][0].record()
        plan.run(data.k, data.v, data.alpha, data.beta, state[sl])
        if launch_events is not None:
            launch_events[j][1].record()
    if events:
        events[1].record()
    for j, plan in enumerate(pp):
        sl = slice(j * per, (j + 1) * per)
        plan.run(data.sq, data.sk, data.sv, data.sa, data.sb, o, state_in=state[sl],
                 state_out=st_out[sl])
    if events:
        events[2].record()


# --------------------------------------------------------------------------
# the CPU oracle as a bounded baseline
# --------------------------------------------------------------------------
def oracle_replay_sample(wl, layers=1, min_seconds=0.0, max_reps=8):
    """Time the fp64 oracle's replay of `layers` of the stack's layers (all heads, R tokens
    each; one layer's inputs repeated, the oracle's cost does not depend on the values),
    repeated until `min_seconds` have passed.  Returns (replayed tokens/s through the
    whole stack, cores, sample text)."""
    import oracle
    R = wl.R[0]
    t = inputs.draw_tensors(R, wl.H, wl.dk, wl.dv, wl.dtype, wl.alpha_lo, wl.alpha_hi, 0,
                            device="cpu", with_q=False)

    def bits(x):
        return x.contiguous().view(torch.int16).numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.numpy()
    k = np.concatenate([bits(t["k"])] * layers)
    v = np.concatenate([bits(t["v"])] * layers)
    a = np.concatenate([t["alpha"].numpy()] * layers)
    b = np.concatenate([t["beta"].numpy()] * layers)
    off = (np.arange(layers + 1) * R).astype(np.int32)
    reps = 0
    t0 = time.perf_counter()
    while True:
        oracle.replay_state(k, v, a, b, off, [R] * layers, [R] * layers)
        reps += 1
        elapsed = time.perf_counter() - t0
        if elapsed >= min_seconds or reps >= max_reps:
            break
    per_stack = elapsed / (reps * layers) * wl.layers
    scaled = "" if layers == wl.layers else f", scaled x{wl.layers / layers:g} to the {wl.layers}-layer stack"
    return (R / per_stack, oracle.num_threads(),
            f"fp64 oracle replay of {layers} of {wl.layers} layers ({wl.H} heads x {R} tokens each), "
            f"{reps} run(s) in {elapsed:.1f} s{scaled}")


def _oracle_bits(x):
    """bf16 tensors as their raw bits (the oracle's bf16 input form); fp32 as numpy."""
    return x.contiguous().view(torch.int16).numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.numpy()


def oracle_throughput(kind, dtype, H, dk, dv, tokens, alpha_lo, alpha_hi, seed=3, min_seconds=1.0,
                      max_reps=20):
    """Token-heads/s of the fp64 oracle on a bounded sample: one sequence of `tokens` rows
    and `H` heads from a zero state, run until `min_seconds` have passed; kind "replay"
    (state only) or "prefill" (with outputs).  The oracle runs its (sequence, head) units
    in parallel, so H at least its thread count makes the figure stand for the whole
    host.  Returns (token-heads/s, seconds)."""
    import oracle
    t = inputs.draw_tensors(tokens, H, dk, dv, dtype, alpha_lo, alpha_hi, seed, device="cpu",
                            with_q=(kind == "prefill"))
    off = np.array([0, tokens], np.int32)
    k, v = _oracle_bits(t["k"]), _oracle_bits(t["v"])
    a, b = t["alpha"].numpy(), t["beta"].numpy()
    q = _oracle_bits(t["q"]) if kind == "prefill" else None
    reps = 0
    t0 = time.perf_counter()
    while True:
        if kind == "replay":
            oracle.replay_state(k, v, a, b, off, [tokens], [tokens])
        else:
            oracle.prefill(q, k, v, a, b, off)
        reps += 1
        dt = time.perf_counter() - t0
        if dt >= min_seconds or reps >= max_reps:
            break
    return reps * tokens * H / dt, dt


def cpu_full_prefill_sample(wl, sample_tokens=2048):
    """The fp64 oracle's full prefill (prefix ++ suffix from a zero state, with outputs) on
    a bounded sample (as many heads as the oracle has threads, `sample_tokens` rows),
    extrapolated by token-heads to the whole stack.  Returns (seconds per full prefill
    of the stack, sample text)."""
    import oracle
    th = max(1, oracle.num_threads())
    tps, dt = oracle_throughput("prefill", wl.dtype, th, wl.dk, wl.dv, sample_tokens, wl.alpha_lo,
                                wl.alpha_hi)
    full_tokens = wl.match_len[0] + wl.suffix_len[0]
    secs = full_tokens * wl.H * wl.layers / tps
    return secs, (f"fp64 oracle prefill with outputs of {th} heads x {sample_tokens} tokens (repeated for "
                  f"{dt:.1f} s), "
                  f"extrapolated by token-heads to {wl.layers} layers x {wl.H} heads x {full_tokens} tokens")


# --------------------------------------------------------------------------
# main benchmark (our kernels)
# --------------------------------------------------------------------------
def bench_ours(args, rank, world, local):
    import gated_deltanet_state_tail_b200 as gdn
    wl = inputs.stack_workload(args.layers)
    kernel = {"auto": gdn.GDN_KERNEL_AUTO, "recurrent": gdn.GDN_KERNEL_RECURRENT,
              "chunked": gdn.GDN_KERNEL_CHUNKED_TC}[args.kernel]
    data = StackData(wl, "cuda", compact=args.no_comparator)
    rp, pp, state, o, st_out, n_launch = build_stack_runner(data, kernel)
    kernel_used = rp[0].info["kernel"]
    kname = {1: "recurrent", 2: "chunked_tc"}[kernel_used]
    flush = torch.empty(L2_FLUSH_BYTES // 4, dtype=torch.float32, device="cuda")
    stream = torch.cuda.current_stream()

    for _ in range(args.warmup):
        run_step(data, rp, pp, state, o, st_out)
    torch.cuda.synchronize()
    for p in rp + pp:
        p.check()

    evs = [[torch.cuda.Event(enable_timing=True) for _ in range(3)] for _ in range(args.steps)]
    lev = [[[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in range(n_launch)]
           for _ in range(args.steps)]
    barrier(world)
    torch.cuda.synchronize()
    with ClockSampler(local) as clk:
        wall0 = time.perf_counter()
        for i in range(args.steps):
            flush.fill_(float(i))             # L2 flush between steps, outside the step events
            run_step(data, rp, pp, state, o, st_out, evs[i], lev[i])
        torch.cuda.synchronize()
        wall = time.perf_counter() - wall0
    barrier(world)
    for p in rp + pp:
        p.check()
    rebuild_ms = [e[0].elapsed_time(e[1]) for e in evs]
    suffix_ms = [e[1].elapsed_time(e[2]) for e in evs]
    step_ms = [e[0].elapsed_time(e[2]) for e in evs]
    launch_ms = [l[0].elapsed_time(l[1]) for step in lev for l in step]
    t_rebuild = max_over_ranks(sum(rebuild_ms) / 1e3, world)
    t_step = max_over_ranks(sum(step_ms) / 1e3, world)

    # one request's tail through all 24 layers, per step and per replica
    value = replica_throughput(data.R * args.steps, world, t_rebuild)

    # roofline of the dominant kernel (the replay launch)
    peaks = measured_peaks()
    units_per_launch = data.per_launch * wl.H
    launch_s = statistics.mean(launch_ms) / 1e3
    if kernel_used == gdn.GDN_KERNEL_CHUNKED_TC:
        alg_bytes = units_per_launch * (data.R * (2 * wl.dk * 2 + 8) + wl.dk * wl.dv * 4)
        achieved = alg_bytes / launch_s / 1e9
        roof = {"bound": "hbm", "achieved": achieved, "peak": peaks["hbm_gbs"], "unit": "GB/s",
                "frac": achieved / peaks["hbm_gbs"],
                "traffic": profiled_traffic(kname, units_per_launch),
                "peak_source": peaks["source"]}
    else:
        # fp32 CUDA-core recurrence: 4 d_k d_v flops per token-head (dot + rank-1 update)
        flops = units_per_launch * data.R * 4 * wl.dk * wl.dv
        achieved = flops / launch_s / 1e12
        fp32_peak = 148 * 128 * 2 * peaks["sm_max_mhz"] * 1e6 / 1e12
        roof = {"bound": "alu", "achieved": achieved, "peak": fp32_peak, "unit": "TFLOP/s",
                "frac": achieved / fp32_peak,
                "traffic": profiled_traffic(kname, units_per_launch),
                "peak_source": "148 SMs x 128 fp32 FMA/clk x 2 x max SM clock"}

    result = {
        "metric": BENCH_METRIC,
        "value": value, "unit": "replayed tokens/s", "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": t_step * 1e3 / args.steps,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
        "dtype": wl.dtype, "data": "synthetic (seeded q/k/v/alpha/beta; no datasets or weights)",
        "config": {"workload": wl.name, "layers": wl.layers, "heads": wl.H, "d_k": wl.dk,
                   "d_v": wl.dv, "matched_prefix": wl.match_len[0], "replay": data.R, "suffix": data.N,
                   "resident_prefix_rows": data.L,
                   "launches_per_phase": n_launch, "layers_per_launch": data.per_launch,
                   "kernel": kname, "l2": "inputs larger than L2 and a 256 MB flush between steps",
                   "parallelism": f"replicas x{world}"},
        "state_rebuild_latency_ms": t_rebuild * 1e3 / args.steps,
        "suffix_prefill_ms": statistics.mean(suffix_ms),
        "rebuild_ms_p50": statistics.median(rebuild_ms),
        "rebuild_ms_p90": float(np.percentile(rebuild_ms, 90)),
        "token_head_layers_per_s": value * wl.H * wl.layers,
        "gpu_launches": 2 * n_launch * args.steps,
        "roofline": roof,
        "wall_s_timed": wall,
    }
    result["clocks"] = clk.summary()
    # tensor side of the same replay launch: 6 C d + 4 d^2 flops per token-head (chunk GEMMs)
    flops_launch = units_per_launch * data.R * (6 * 64 * wl.dk + 4 * wl.dk * wl.dv)
    result["replay_tflops"] = flops_launch / launch_s / 1e12
    result["replay_tensor_frac"] = result["replay_tflops"] / peaks["bf16_tflops"]
    if kernel_used == gdn.GDN_KERNEL_CHUNKED_TC:
        result.update(launch_shapes(data, kernel))

    if not args.no_comparator:
        result.update(full_prefill_comparator(data, kernel, rp, pp, state, o, st_out))
        result["gdn_speedup_vs_full_prefill"] = result["full_prefill_ms"] / result["ms_per_step"]
        result["gdn_speedup_token_ratio"] = (wl.match_len[0] + data.N) / (data.R + data.N)
    if not args.no_e2e:
        result["e2e"] = e2e_host_buffers(data, kernel, args, world)
    R_stack, N_stack = data.R, data.N
    if world == 1 and not args.no_extras:
        # the other workloads of the hot path, one GPU: the single layer at 8K (5%), the
        # ragged 64-request batch and the replay-budget sweep
        for p_ in rp + pp:
            p_.close()
        del data, rp, pp, state, o, st_out
        torch.cuda.empty_cache()
        result["workloads"] = {"layer": workload_layer(flush, peaks), "varlen": workload_varlen(flush, peaks),
                               "sweep": workload_sweep(flush, peaks)}
    if rank == 0 and world == 1 and not args.no_cpu_baseline:
        v, cores, sample = oracle_replay_sample(wl, layers=wl.layers, min_seconds=10.0)
        result["cpu_baseline"] = {"value": v, "unit": "replayed tokens/s", "cores": cores,
                                  "kind": "oracle", "sample": sample}
        sv, ssample = cpu_suffix_sample(wl)
        result["cpu_suffix_prefill"] = {"value": sv, "unit": "suffix tokens/s", "cores": cores, "kind": "oracle",
                                        "sample": ssample}
        fs, fsample = cpu_full_prefill_sample(wl)
        result["cpu_full_prefill"] = {"value": fs, "unit": "s per full prefill of the stack (extrapolated)",
                                      "cores": cores, "kind": "oracle", "sample": fsample}
        # the same ratio as gdn_speedup_vs_full_prefill, on the host cores
        result["cpu_gdn_speedup_vs_full_prefill"] = fs / (R_stack / v + N_stack / sv)
    return result


def full_prefill_comparator(data, kernel, rp, pp, state, o, st_out, iters=3):
    """GPU full prefill of the same layers over prefix ++ suffix from a zero state."""
    import gated_deltanet_state_tail_b200 as gdn
    wl = data.wl
    plans = []
    for slots in data.launches:
        cu = np.array([s * data.seq for s in slots] + [(slots[-1] + 1) * data.seq], np.int32)
        plans.append(gdn.PrefillPlan(wl.H, wl.dk, wl.dv, wl.dtype, cu, kernel))
    o_full = torch.empty((data.layers * data.seq, wl.H, wl.dv), dtype=data.k.dtype, device="cuda")
    st_full = torch.empty_like(state)
    per = data.per_launch

    def full():
        for j, p in enumerate(plans):
            p.run(data.q, data.k, data.v, data.alpha, data.beta, o_full,
                  state_out=st_full[j * per:(j + 1) * per])
    full()
    torch.cuda.synchronize()
    times = []
    for _ in range(iters):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        full()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    for p in plans:
        p.check()
    # cache-hit path once more to compare its final states / outputs with the full prefill
    run_step(data, rp, pp, state, o, st_out)
    torch.cuda.synchronize()
    idx = torch.cat([torch.arange(s * data.seq + data.L, (s + 1) * data.seq, device="cuda")
                     for s in range(data.layers)])
    o_ref = o_full[idx].float()
    d_state = (st_out - st_full).flatten(2).norm(dim=2) / st_full.flatten(2).norm(dim=2)
    d_o = (o.float() - o_ref).norm() / o_ref.norm()
    full_ms = statistics.median(times)
    for p in plans:
        p.close()
    return {"full_prefill_ms": full_ms,
            "gdn_speedup_vs_full_prefill": None,
            "replay_vs_full_state_rel_frob": {"mean": float(d_state.mean()), "max": float(d_state.max())},
            "replay_vs_full_suffix_out_rel_frob": float(d_o)}


def launch_shapes(data, kernel, iters=5):
    """The same 24-layer rebuild as one launch of all layers and as one launch per layer
    (the bench line runs three launches of eight)."""
    import gated_deltanet_state_tail_b200 as gdn
    wl = data.wl
    H, dk, dv = wl.H, wl.dk, wl.dv
    state = torch.empty((data.layers, H, dk, dv), dtype=torch.float32, device="cuda")
    flush = torch.empty(L2_FLUSH_BYTES // 4, dtype=torch.float32, device="cuda")
    all_slots = list(range(data.layers))
    off, ml, R = data.replay_desc(all_slots)
    one = gdn.ReplayPlan(H, dk, dv, wl.dtype, off, ml, R, kernel)
    per_layer = []
    for s_ in all_slots:
        o1, m1, r1 = data.replay_desc([s_])
        per_layer.append(gdn.ReplayPlan(H, dk, dv, wl.dtype, o1, m1, r1, kernel))

    def one_launch():
        one.run(data.k, data.v, data.alpha, data.beta, state)

    def per_layer_launches():
        for s_, p in enumerate(per_layer):
            p.run(data.k, data.v, data.alpha, data.beta, state[s_:s_ + 1])

    t1 = _time_ms(one_launch, iters, flush)
    t24 = _time_ms(per_layer_launches, iters, flush)
    for p in [one] + per_layer:
        p.check()
        p.close()
    return {"rebuild_1x24_ms": t1, "rebuild_24x1_ms": t24}


def cpu_suffix_sample(wl):
    """The fp64 oracle's suffix prefill (with outputs) of one layer: all heads, N tokens from
    a random state; returns suffix tokens/s through the whole stack and the sample text."""
    import oracle
    N = wl.suffix_len[0]
    t = inputs.draw_tensors(N, wl.H, wl.dk, wl.dv, wl.dtype, wl.alpha_lo, wl.alpha_hi, 1, device="cpu")

    def bits(x):
        return x.contiguous().view(torch.int16).numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.numpy()
    si = np.random.default_rng(0).standard_normal((1, wl.H, wl.dk, wl.dv)) * 0.1
    t0 = time.perf_counter()
    oracle.prefill(bits(t["q"]), bits(t["k"]), bits(t["v"]), t["alpha"].numpy(), t["beta"].numpy(),
                   np.array([0, N], np.int32), state_in=si)
    dt = time.perf_counter() - t0
    return N / (dt * wl.layers), f"fp64 oracle suffix prefill of 1 of {wl.layers} layers ({wl.H} heads x {N} tokens, " \
                                 f"{dt:.2f} s), scaled x{wl.layers}"


def e2e_host_buffers(data, kernel, args, world):
    """Same metric through the C ABI with host buffers: every step copies the
    tail windows and the suffix inputs from pinned host memory, runs the
    replay and the suffix prefill, and reads states and outputs back.  The
    copies of one launch group overlap the kernels of another, and a step's
    read-back overlaps the next step's input copies (PCIe carries both
    directions at once)."""
    import gated_deltanet_state_tail_b200 as gdn
    wl = data.wl
    H, dk, dv = wl.H, wl.dk, wl.dv
    L, R, N, layers = data.L, data.R, data.N, data.layers
    tail_idx = torch.cat([torch.arange(s * data.seq + L - R, s * data.seq + L, device="cuda")
                          for s in range(layers)])
    host = {}
    for name, src in (("k", data.k), ("v", data.v), ("alpha", data.alpha), ("beta", data.beta)):
        host["t" + name] = src[tail_idx].cpu().pin_memory()
    for name, src in (("q", data.sq), ("k", data.sk), ("v", data.sv), ("alpha", data.sa), ("beta", data.sb)):
        host["s" + name] = src.cpu().pin_memory()
    dev = {k: torch.empty_like(v, device="cuda") for k, v in host.items()}
    state = torch.empty((layers, H, dk, dv), dtype=torch.float32, device="cuda")
    st_out = torch.empty_like(state)
    o = torch.empty((layers * N, H, dv), dtype=data.k.dtype, device="cuda")
    h_state = torch.empty(state.shape, dtype=torch.float32).pin_memory()
    h_o = torch.empty(o.shape, dtype=o.dtype).pin_memory()
    per = data.per_launch
    rp, pp = [], []
    for j in range(len(data.launches)):
        slots = range(j * per, (j + 1) * per)
        off = np.array([s * R for s in slots] + [(j + 1) * per * R], np.int32)
        rp.append(gdn.ReplayPlan(H, dk, dv, wl.dtype, off, np.full(per, R, np.int32),
                                 np.full(per, R, np.int32), kernel))
        cu = np.array([s * N for s in slots] + [(j + 1) * per * N], np.int32)
        pp.append(gdn.PrefillPlan(H, dk, dv, wl.dtype, cu, kernel))

    # The three launch groups are independent, so group j + 1's inputs cross PCIe while
    # group j replays and prefills (copy-in stream, compute stream), and group j's states
    # and outputs are read back on a third stream.  Across steps, group j's inputs are
    # overwritten once the last step's kernels of group j have read them (ev_done), and
    # its states and outputs once the last step has read them back (ev_out).
    cur = torch.cuda.current_stream()
    s_in, s_out = torch.cuda.Stream(), torch.cuda.Stream()
    n_groups = len(rp)
    ev_in = [torch.cuda.Event() for _ in range(n_groups)]
    ev_done = [torch.cuda.Event() for _ in range(n_groups)]
    ev_out = [torch.cuda.Event() for _ in range(n_groups)]

    def rows_of(name, j):
        per_rows = per * (R if name.startswith("t") else N)
        return slice(j * per_rows, (j + 1) * per_rows)

    def step():
        for j in range(n_groups):
            s_in.wait_event(ev_done[j])        # the last step's kernels of group j are done
            with torch.cuda.stream(s_in):
                for k in dev:
                    sl = rows_of(k, j)
                    dev[k][sl].copy_(host[k][sl], non_blocking=True)
            ev_in[j].record(s_in)
        for j in range(n_groups):
            cur.wait_event(ev_in[j])
            cur.wait_event(ev_out[j])          # the last step has read group j's results back
            gs, rs = slice(j * per, (j + 1) * per), slice(j * per * N, (j + 1) * per * N)
            rp[j].run(dev["tk"], dev["tv"], dev["talpha"], dev["tbeta"], state[gs])
            pp[j].run(dev["sq"], dev["sk"], dev["sv"], dev["salpha"], dev["sbeta"], o,
                      state_in=state[gs], state_out=st_out[gs])
            ev_done[j].record(cur)
            s_out.wait_event(ev_done[j])
            with torch.cuda.stream(s_out):
                h_state[gs].copy_(st_out[gs], non_blocking=True)
                h_o[rs].copy_(o[rs], non_blocking=True)
            ev_out[j].record(s_out)

    steps = max(3, min(args.steps, 10))
    for _ in range(2):
        step()
    cur.wait_stream(s_out)
    torch.cuda.synchronize()
    # the results every step reads back must not depend on how the steps overlap
    ref_state, ref_o = h_state.clone(), h_o.clone()
    barrier(world)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    s_in.wait_stream(cur)                      # no timed copy starts before the start event
    for _ in range(steps):
        step()
    cur.wait_stream(s_out)                     # the last step's results are on the host
    b.record()
    torch.cuda.synchronize()
    t = max_over_ranks(a.elapsed_time(b) / 1e3, world)
    torch.cuda.synchronize()
    same = bool(torch.equal(h_state, ref_state) and torch.equal(h_o, ref_o))
    for p in rp + pp:
        p.check()
        p.close()
    h2d = sum(v.numel() * v.element_size() for v in host.values())
    d2h = h_state.numel() * 4 + h_o.numel() * h_o.element_size()
    return {"value": R * steps * world / t, "unit": "replayed tokens/s",
            "h2d_bytes_per_step": h2d, "d2h_bytes_per_step": d2h, "steps": steps,
            "ms_per_step": t * 1e3 / steps, "results_identical_across_steps": same}


# --------------------------------------------------------------------------
# auxiliary workloads (not the headline line): budget sweep and varlen batch
# --------------------------------------------------------------------------
def _time_ms(fn, iters=5, flush=None):
    fn()
    torch.cuda.synchronize()
    ts = []
    for _ in range(iters):
        if flush is not None:
            flush.fill_(1.0)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        fn()
        b.record()
        torch.cuda.synchronize()
        ts.append(a.elapsed_time(b))
    return statistics.median(ts)


def replay_bytes(H, dk, dv, R_list):
    """Algorithmic HBM bytes of a bf16 replay launch: per (sequence, head) unit the k and v
    rows of its window (2 x d x 2 B per token) and the fp32 gates (8 B per token), plus the
    fp32 state written (dk x dv x 4 B)."""
    return sum(H * (r * (dk * 2 + dv * 2 + 8) + dk * dv * 4) for r in R_list)


def _hbm_roofline(nbytes, ms, peaks):
    gbs = nbytes / (ms / 1e3) / 1e9
    return {"bound": "hbm", "achieved": gbs, "peak": peaks["hbm_gbs"], "unit": "GB/s",
            "frac": gbs / peaks["hbm_gbs"], "bytes_per_launch": nbytes, "peak_source": peaks["source"]}


def _oracle_timed(fn, min_seconds=1.0, max_reps=50):
    """Run fn() until min_seconds have passed; returns (seconds per run, runs, result)."""
    reps, t0 = 0, time.perf_counter()
    while True:
        out = fn()
        reps += 1
        dt = time.perf_counter() - t0
        if dt >= min_seconds or reps >= max_reps:
            return dt / reps, reps, out


def workload_layer(flush, peaks, iters=20):
    """One GDN layer, 16 heads, d = 128, bf16: matched prefix L = 8192, replay R = 410 (5%),
    suffix N = 512.  Rebuild and suffix prefill (one launch each), the full prefill of
    L + N as the GPU comparator, and the fp64 oracle's rebuild and suffix prefill on the
    host cores (the whole workload, repeated for at least 1 s each)."""
    import gated_deltanet_state_tail_b200 as gdn
    import oracle
    wl = inputs.single_layer_workload()
    H, L, R, N = wl.H, wl.match_len[0], wl.R[0], wl.suffix_len[0]
    t = inputs.draw_tensors(L + N, H, 128, 128, "bf16", wl.alpha_lo, wl.alpha_hi, wl.seeds[0], device="cuda")
    rp = gdn.ReplayPlan(H, 128, 128, "bf16", [0, L + N], [L], [R])
    pp = gdn.PrefillPlan(H, 128, 128, "bf16", [0, N])
    fp = gdn.PrefillPlan(H, 128, 128, "bf16", [0, L + N])
    st = torch.empty((1, H, 128, 128), device="cuda")
    st2 = torch.empty_like(st)
    o = torch.empty((N, H, 128), dtype=torch.bfloat16, device="cuda")
    of = torch.empty((L + N, H, 128), dtype=torch.bfloat16, device="cuda")
    s = {n: t[n][L:] for n in t}
    rep_ms = _time_ms(lambda: rp.run(t["k"], t["v"], t["alpha"], t["beta"], st), iters, flush)
    suf_ms = _time_ms(lambda: pp.run(s["q"], s["k"], s["v"], s["alpha"], s["beta"], o, state_in=st,
                                     state_out=st2), iters, flush)
    full_ms = _time_ms(lambda: fp.run(t["q"], t["k"], t["v"], t["alpha"], t["beta"], of, state_out=st2),
                       5, flush)
    for p_ in (rp, pp, fp):
        p_.check()
        p_.close()
    # the oracle on the same workload: the rebuild (R rows x H heads), then the suffix
    win = {n: _oracle_bits(t[n][L - R:L].cpu()) for n in ("k", "v", "alpha", "beta")}
    sh = {n: _oracle_bits(s[n].cpu()) for n in ("q", "k", "v", "alpha", "beta")}
    cpu_rep_s, nr, S = _oracle_timed(lambda: oracle.replay_state(win["k"], win["v"], win["alpha"], win["beta"],
                                                                 [0, R], [R], [R]))
    cpu_suf_s, ns, _ = _oracle_timed(lambda: oracle.prefill(sh["q"], sh["k"], sh["v"], sh["alpha"], sh["beta"],
                                                            [0, N], state_in=S))
    units = H
    return {"workload": wl.name, "heads": H, "matched_prefix": L, "replay": R, "suffix": N,
            "rebuild_ms": rep_ms, "suffix_prefill_ms": suf_ms, "full_prefill_ms": full_ms,
            "replayed_tokens_per_s": R / (rep_ms / 1e3),
            "gdn_speedup_vs_full_prefill": full_ms / (rep_ms + suf_ms),
            "ctas_per_launch": units,
            "roofline": _hbm_roofline(replay_bytes(H, 128, 128, [R]), rep_ms, peaks),
            "cpu_baseline": {"value": R / cpu_rep_s, "unit": "replayed tokens/s", "rebuild_ms": cpu_rep_s * 1e3,
                             "suffix_prefill_ms": cpu_suf_s * 1e3, "cores": oracle.num_threads(),
                             "kind": "oracle",
                             "sample": f"the whole workload: fp64 oracle rebuild ({H} heads x {R} tokens, "
                                       f"{nr} runs) and suffix prefill ({H} heads x {N} tokens, {ns} runs)"},
            "timing": f"median of {iters} launches, 256 MB L2 flush before each"}


def workload_varlen(flush, peaks, iters=10):
    """64 ragged requests, 16 heads: every tail replayed, then every suffix prefilled (one
    launch each).  The fp64 oracle runs requests 0-3 on the host cores."""
    import gated_deltanet_state_tail_b200 as gdn
    wl = inputs.varlen_workload(64, seed=0)
    off, cu = wl.seq_offsets(), wl.suffix_cu()
    H = wl.H
    cache = inputs.draw_tensors(int(off[-1]), H, 128, 128, "bf16", wl.alpha_lo, wl.alpha_hi, 100,
                                device="cuda", with_q=False)
    suf = inputs.draw_tensors(int(cu[-1]), H, 128, 128, "bf16", wl.alpha_lo, wl.alpha_hi, 101, device="cuda")
    rp = gdn.ReplayPlan(H, 128, 128, "bf16", off, wl.match_len, wl.R)
    pp = gdn.PrefillPlan(H, 128, 128, "bf16", cu)
    st = torch.empty((wl.batch, H, 128, 128), device="cuda")
    st2 = torch.empty_like(st)
    o = torch.empty((int(cu[-1]), H, 128), dtype=torch.bfloat16, device="cuda")
    rep_ms = _time_ms(lambda: rp.run(cache["k"], cache["v"], cache["alpha"], cache["beta"], st), iters, flush)
    suf_ms = _time_ms(lambda: pp.run(suf["q"], suf["k"], suf["v"], suf["alpha"], suf["beta"], o,
                                     state_in=st, state_out=st2), iters, flush)
    rp.check()
    pp.check()
    rp.close()
    pp.close()
    Reff = [min(r, l) for r, l in zip(wl.R, wl.match_len)]
    cpu = cpu_varlen_sample(wl, off, cu, cache, suf)
    del cache, suf
    return {"workload": wl.name, "requests": wl.batch, "heads": H,
            "replayed_tokens": int(sum(Reff)), "suffix_tokens": int(sum(wl.suffix_len)),
            "rebuild_ms": rep_ms, "suffix_prefill_ms": suf_ms,
            "replayed_tokens_per_s": sum(Reff) / (rep_ms / 1e3),
            "suffix_tokens_per_s": sum(wl.suffix_len) / (suf_ms / 1e3),
            "longest_window": int(max(Reff)),
            "roofline": _hbm_roofline(replay_bytes(H, 128, 128, Reff), rep_ms, peaks),
            "cpu_baseline": cpu, "timing": f"median of {iters} launches, 256 MB L2 flush before each",
            "match_len": wl.match_len, "R": wl.R, "suffix_len": wl.suffix_len}


def workload_sweep(flush, peaks, sample_heads=(0, 17), iters=5):
    """Replay budget R/L in {1, 2, 5, 10, 25, 100}% at L = 8K, 16K, 32K (one layer, 32 heads,
    slow decay alpha ~ U[0.97, 0.9999]).  Per point: the replay's latency and roofline
    fraction, the full prefill of L (per L), and on sampled heads

    * `truncation_rel_frob`: ||S_R - S_L|| / ||S_L|| from the fp64 oracle alone, the
      state error that replaying only the tail causes (no kernel rounding in it);
    * `kernel_vs_oracle`: the GPU replay's own error against the oracle's replay of the
      same window (max|err| / max|ref| and relative Frobenius), its rounding floor.

    The oracle's host time per point is extrapolated by token-heads from bounded samples."""
    import gated_deltanet_state_tail_b200 as gdn
    import oracle
    th = max(1, oracle.num_threads())
    rep_tps, rep_dt = oracle_throughput("replay", "bf16", th, 128, 128, 2048, 0.97, 0.9999)
    pre_tps, pre_dt = oracle_throughput("prefill", "bf16", th, 128, 128, 2048, 0.97, 0.9999)
    cpu_sample = (f"fp64 oracle on {th} heads x 2048 tokens, each kind repeated for at least 1 s (replay "
                  f"{rep_dt:.1f} s, prefill with outputs {pre_dt:.1f} s); extrapolated by token-heads")
    heads = list(sample_heads)
    points = []
    for L in (8192, 16384, 32768):
        wls = [w for w in inputs.sweep_workloads() if w.match_len[0] == L]
        H = wls[0].H
        t = inputs.draw_tensors(L, H, 128, 128, "bf16", 0.97, 0.9999, 0, device="cuda")
        full_state = torch.empty((1, H, 128, 128), device="cuda")
        pf = gdn.PrefillPlan(H, 128, 128, "bf16", [0, L])
        o = torch.empty((L, H, 128), dtype=torch.bfloat16, device="cuda")
        full_ms = _time_ms(lambda: pf.run(t["q"], t["k"], t["v"], t["alpha"], t["beta"], o,
                                          state_out=full_state), iters, flush)
        pf.check()
        pf.close()
        sub = {n: _oracle_bits(t[n][:, heads].cpu()) for n in ("k", "v", "alpha", "beta")}
        S_full = oracle.replay_state(sub["k"], sub["v"], sub["alpha"], sub["beta"], [0, L], [L], [L])[0]
        for w in wls:
            R = w.R[0]
            plan = gdn.ReplayPlan(H, 128, 128, "bf16", [0, L], [L], [R])
            st = torch.empty_like(full_state)
            rep_ms = _time_ms(lambda: plan.run(t["k"], t["v"], t["alpha"], t["beta"], st), iters, flush)
            plan.check()
            plan.close()
            S_rep = oracle.replay_state(sub["k"], sub["v"], sub["alpha"], sub["beta"], [0, L], [L], [R])[0]
            got = st[0, heads].double().cpu().numpy()
            trunc = [float(np.linalg.norm(S_rep[i] - S_full[i]) / np.linalg.norm(S_full[i]))
                     for i in range(len(heads))]
            k_max = [float(np.max(np.abs(got[i] - S_rep[i])) / np.max(np.abs(S_rep[i]))) for i in range(len(heads))]
            k_frob = [float(np.linalg.norm(got[i] - S_rep[i]) / np.linalg.norm(S_rep[i])) for i in range(len(heads))]
            points.append({"L": L, "pct": w.extra["pct"], "R": R, "replay_ms": rep_ms, "full_prefill_ms": full_ms,
                           "replay_speedup_vs_full_prefill": full_ms / rep_ms,
                           "replayed_tokens_per_s": R / (rep_ms / 1e3),
                           "roofline_frac": _hbm_roofline(replay_bytes(H, 128, 128, [R]), rep_ms, peaks)["frac"],
                           "truncation_rel_frob": {"mean": float(np.mean(trunc)), "max": float(np.max(trunc))},
                           "kernel_vs_oracle": {"max_err_over_max_ref": float(np.max(k_max)),
                                                "rel_frob": float(np.max(k_frob))},
                           "cpu_baseline_ms": {"replay": R * H / rep_tps * 1e3, "full_prefill": L * H / pre_tps * 1e3}})
        del t
    return {"workload": "sweep-H32-d128-bf16-L8K16K32K-alpha0.97-0.9999", "heads": 32,
            "sampled_heads": heads, "points": points,
            "cpu_baseline": {"cores": th, "kind": "oracle", "sample": cpu_sample},
            "timing": f"median of {iters} launches, 256 MB L2 flush before each"}


def bench_sweep(args):
    """The replay-budget sweep as one auxiliary line per point."""
    flush = torch.empty(L2_FLUSH_BYTES // 4, dtype=torch.float32, device="cuda")
    sw = workload_sweep(flush, measured_peaks())
    return [dict(p, metric="replay-budget sweep", workload=f"sweep-L{p['L']}-p{p['pct']}", heads=sw["heads"],
                 sampled_heads=sw["sampled_heads"], alpha="U[0.97, 0.9999]", dtype="bf16", data="synthetic",
                 cpu_sample=sw["cpu_baseline"]["sample"])
            for p in sw["points"]]


def bench_varlen(args):
    """64 ragged requests (16 heads): replay of every tail, then every suffix."""
    flush = torch.empty(L2_FLUSH_BYTES // 4, dtype=torch.float32, device="cuda")
    v = workload_varlen(flush, measured_peaks())
    return [dict(v, metric="varlen replay + suffix", dtype="bf16", data="synthetic")]


def varlen_tail_windows(wl, off, cache, nreq):
    """The replay windows of the first `nreq` requests, copied to the host as sequences of
    their own: (k, v, alpha, beta, offsets, lengths)."""
    ml = [min(l, int(c)) for l, c in zip(wl.match_len[:nreq], np.diff(off)[:nreq])]
    rr = [max(0, min(r, l)) for r, l in zip(wl.R[:nreq], ml)]
    rows = torch.cat([torch.arange(int(off[b]) + ml[b] - rr[b], int(off[b]) + ml[b], dtype=torch.long)
                      for b in range(nreq)]).to(cache["k"].device)
    k, v = cache["k"][rows].cpu(), cache["v"][rows].cpu()
    a, b_ = cache["alpha"][rows].cpu().numpy(), cache["beta"][rows].cpu().numpy()
    woff = np.concatenate([[0], np.cumsum(rr)]).astype(np.int32)
    return k, v, a, b_, woff, rr


def cpu_varlen_sample(wl, off, cu, cache, suf, nreq=4):
    """The fp64 oracle on the first `nreq` requests of the varlen batch (all heads): the
    replay of their tails, then their suffix prefill from the replayed states.  The
    tails are copied out as sequences of their own (a replay reads only its window)."""
    import oracle
    k, v, a, b_, woff, rr = varlen_tail_windows(wl, off, cache, nreq)
    t0 = time.perf_counter()
    states = oracle.replay_state(_oracle_bits(k), _oracle_bits(v), a, b_, woff, rr, rr)
    t_rep = time.perf_counter() - t0
    n_suf = int(cu[nreq])
    sq, sk, sv = (suf[x][:n_suf].cpu() for x in ("q", "k", "v"))
    t0 = time.perf_counter()
    oracle.prefill(_oracle_bits(sq), _oracle_bits(sk), _oracle_bits(sv), suf["alpha"][:n_suf].cpu().numpy(),
                   suf["beta"][:n_suf].cpu().numpy(), np.asarray(cu[:nreq + 1], np.int32), state_in=states)
    t_suf = time.perf_counter() - t0
    return {"replayed_tokens_per_s": sum(rr) / t_rep, "suffix_tokens_per_s": n_suf / t_suf,
            "cores": oracle.num_threads(), "kind": "oracle",
            "sample": f"fp64 oracle on requests 0-{nreq - 1} of {wl.batch} ({wl.H} heads): replay of "
                      f"{sum(rr)} tail tokens {t_rep:.1f} s, suffix prefill of {n_suf} tokens {t_suf:.1f} s"}


def bench_decode(args):
    """One decode step (the token after the prefill) of the 24-layer stack for 64 requests:
    32 heads, d = 128, bf16 q/k/v/o, fp32 states updated in place.  The layers are folded into
    the batch (24 x 64 = 1536 state slots, 6.4 GB of state, larger than L2), one launch.
    --layers sets fewer layers for a profiling capture."""
    import gated_deltanet_state_tail_b200 as gdn
    layers, B, H, d = args.layers, 64, 32, 128
    nb = layers * B
    t = inputs.draw_tensors(nb, H, d, d, "bf16", 0.9, 0.999, 7, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    state = torch.randn((nb, H, d, d), generator=g, device="cuda") * 0.05
    o = torch.empty((nb, H, d), dtype=torch.bfloat16, device="cuda")

    def step():
        gdn.gdn_decode_step(t["q"], t["k"], t["v"], t["alpha"], t["beta"], state, state, o)

    for _ in range(args.warmup):
        step()
    ms = _time_ms(step, max(args.steps, 10))
    nbytes = nb * H * (2 * d * d * 4 + 4 * d * 2 + 8)   # state read + write, q k v o, alpha beta
    peaks = measured_peaks()
    gbs = nbytes / (ms / 1e3) / 1e9
    return [{"metric": f"GDN decode step ({layers} layers x {B} requests)", "value": ms, "unit": "ms",
             "higher_is_better": False, "workload": f"decode{layers}-B{B}-H{H}-d{d}-bf16", "layers": layers,
             "requests": B, "heads": H, "tokens_per_s": B / (ms / 1e3),
             "roofline": {"bound": "hbm", "achieved": gbs, "peak": peaks["hbm_gbs"], "unit": "GB/s",
                          "frac": gbs / peaks["hbm_gbs"], "traffic": None, "peak_source": peaks["source"],
                          "bytes_per_launch": nbytes},
             "l2": f"{nb * H * d * d * 4 / 1e9:.2f} GB of state per launch (L2 is 126 MB)", "dtype": "bf16",
             "data": "synthetic"}]


def bench_outputs(args):
    """Replay with the window's outputs (layer chaining inside a replay group) against the
    state-only replay, on one bench launch: 8 layers x 32 heads, R = 3277 rows each."""
    import gated_deltanet_state_tail_b200 as gdn
    layers, H, d, R = 8, 32, 128, 3277
    t = inputs.draw_tensors(layers * R, H, d, d, "bf16", 0.9, 0.999, 9, device="cuda")
    off = np.arange(layers + 1, dtype=np.int32) * R
    plan = gdn.ReplayPlan(H, d, d, "bf16", off, [R] * layers, [R] * layers)
    st = torch.empty((layers, H, d, d), device="cuda")
    o = torch.empty((layers * R, H, d), dtype=torch.bfloat16, device="cuda")
    flush = torch.empty(L2_FLUSH_BYTES // 4, dtype=torch.float32, device="cuda")
    state_ms = _time_ms(lambda: plan.run(t["k"], t["v"], t["alpha"], t["beta"], st), 10, flush)
    out_ms = _time_ms(lambda: plan.run_outputs(t["q"], t["k"], t["v"], t["alpha"], t["beta"], o,
                                               state_out=st), 10, flush)
    plan.check()
    plan.close()
    tokens = layers * R
    return [{"metric": "replay with window outputs", "workload": "replay8-H32-d128-bf16-R3277",
             "layers": layers, "heads": H, "R": R, "state_only_ms": state_ms, "with_outputs_ms": out_ms,
             "with_outputs_tokens_per_s": tokens / (out_ms / 1e3), "dtype": "bf16", "data": "synthetic"}]


def bench_overlap(args):
    """Host-to-device copy of the full-attention layers' KV cache on a second stream while
    the 24-layer tail replay runs on the first.  The pages give no FA-layer shape; the
    8 FA layers of the 3:1 stack are taken as wide as the GDN layers (32 heads x 128,
    K and V, bf16) at the 32K prefix: 8 x 32768 x 2 x 32 x 128 x 2 B = 4 GiB, pinned."""
    import gated_deltanet_state_tail_b200 as gdn
    wl = inputs.stack_workload(24)
    data = StackData(wl, "cuda", compact=True)
    rp, pp, state, o, st_out, _ = build_stack_runner(data, gdn.GDN_KERNEL_AUTO)
    kv_bytes = 8 * wl.match_len[0] * 2 * wl.H * wl.dk * 2
    host = torch.empty(kv_bytes, dtype=torch.uint8, pin_memory=True)
    dev = torch.empty(kv_bytes, dtype=torch.uint8, device="cuda")
    s_rep = torch.cuda.current_stream()
    s_copy = torch.cuda.Stream()
    per = data.per_launch

    def replay():
        for j, plan in enumerate(rp):
            plan.run(data.k, data.v, data.alpha, data.beta, state[j * per:(j + 1) * per], stream=s_rep)

    def timed(do_replay, do_copy):
        torch.cuda.synchronize()
        e0 = torch.cuda.Event(enable_timing=True)
        er = torch.cuda.Event(enable_timing=True)
        ec = torch.cuda.Event(enable_timing=True)
        e0.record(s_rep)
        s_copy.wait_event(e0)
        if do_copy:
            with torch.cuda.stream(s_copy):
                dev.copy_(host, non_blocking=True)
        ec.record(s_copy)
        if do_replay:
            replay()
        er.record(s_rep)
        torch.cuda.synchronize()
        return e0.elapsed_time(er), e0.elapsed_time(ec)

    for _ in range(args.warmup):
        timed(True, False)
    timed(False, True)
    # the 4 GiB copy varies by a few ms between repetitions on a shared host, more than
    # the replay itself: interleave copy-alone and copy-with-replay runs and take the
    # fastest of each
    reps = 7
    t_rep = min(timed(True, False)[0] for _ in range(reps))
    copies, both = [], []
    for _ in range(reps):
        copies.append(timed(False, True)[1])
        both.append(timed(True, True))
    t_copy = min(copies)
    t_both = min(max(a, b) for a, b in both)
    t_rep_in = statistics.median(a for a, _ in both)
    for p in rp + pp:
        p.check()
        p.close()
    hidden = max(0.0, min(1.0, (t_rep + t_copy - t_both) / min(t_rep, t_copy)))   # of the shorter
    return [{"metric": "transfer/replay overlap", "workload": "stack24 replay + FA-KV H2D (4 GiB)",
             "fa_kv_bytes": kv_bytes, "replay_ms": t_rep, "copy_ms": t_copy, "both_ms": t_both,
             "timing": "fastest of 7 interleaved runs each",
             "replay_ms_during_copy": t_rep_in, "h2d_gbs": kv_bytes / (t_copy / 1e3) / 1e9,
             "hidden_fraction_of_shorter": hidden, "serial_ms": t_rep + t_copy,
             "fa_kv_shape": "8 layers x 32768 tokens x (K, V) x 32 heads x 128 x bf16 (reading: FA layers "
                            "as wide as the GDN layers, no head sharing)",
             "dtype": "bf16", "data": "synthetic"}]


def bench_hybrid(args):
    """The full-attention layers of the stack at the same cache hit (3:1, so 8 beside 24 GDN
    layers; as wide as those: 32 heads x 128, no head sharing, bf16): the 1024-token suffix
    behind the 32K prefix through norm + rotation + append and paged attention, then one
    decoded token.  Each layer has its own paged cache of 64-token pages in shuffled order
    (0.55 GB, so no layer finds its keys in L2)."""
    import gated_deltanet_state_tail_b200 as gdn
    wl = inputs.stack_workload(args.layers)
    layers, H, d, page = wl.layers // GDN_PER_GROUP, wl.H, wl.dk, 64
    L, N = wl.match_len[0], wl.suffix_len[0]
    pages = -(-(L + N + 1) // page)
    g = torch.Generator(device="cuda").manual_seed(11)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    kc = torch.empty((layers, pages, page, H, d), **bf).normal_(generator=g)
    vc = torch.empty((layers, pages, page, H, d), **bf).normal_(generator=g)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    inv = 10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    qw, kw = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    attn = gdn.PagedAttention(H, H, d, "bf16", max_batch=1, max_rows=N)
    i32 = dict(dtype=torch.int32, device="cuda")

    def part(first, rows):
        """(prepare, attend) of `rows` tokens at position `first` through every layer."""
        qkv = torch.randn((layers, rows, 3 * H, d), generator=g, device="cuda").bfloat16()
        pos = torch.arange(first, first + rows, device="cuda")
        slots = table[0, pos // page].long() * page + pos % page
        q, o = torch.empty((layers, rows, H, d), **bf), torch.empty((layers, rows, H, d), **bf)
        cu, ctx = torch.tensor([0, rows], **i32), torch.tensor([first + rows], **i32)

        def prepare():
            for n in range(layers):
                x = qkv[n]
                gdn.qk_norm_rope(x[:, :H], x[:, H:2 * H], pos, inv, qw, kw, v=x[:, 2 * H:], k_cache=kc[n], v_cache=vc[n],
                                 slots=slots, q_out=q[n])

        def attend():
            for n in range(layers):
                attn.run(q[n], kc[n], vc[n], table, cu, ctx, o[n])

        prepare()
        attend()
        attn.check()
        return prepare, attend

    peaks = measured_peaks()
    flush = torch.empty(L2_FLUSH_BYTES // 4, dtype=torch.float32, device="cuda")
    out = {"metric": f"full-attention layers of the cache hit ({layers} layers)", "unit": "ms", "higher_is_better": False,
           "workload": f"hybrid{layers}-H{H}-d{d}-bf16-L{L}-N{N}", "layers": layers, "heads": H, "page": page,
           "l2": "flushed before every timed part", "dtype": "bf16", "data": "synthetic"}
    reps = max(3, min(args.steps, 20))
    for name, first, rows in (("suffix", L, N), ("decode", L + N, 1)):
        prepare, attend = part(first, rows)
        prep_ms, attn_ms = _time_ms(prepare, reps, flush), _time_ms(attend, reps, flush)
        row_bytes = rows * H * d * 2
        pairs = rows * first + rows * (rows + 1) // 2
        out[name] = {"norm_rope_ms": prep_ms, "attention_ms": attn_ms,
                     "norm_rope_roofline": _hbm_roofline(layers * (6 * row_bytes + 16 * rows), prep_ms, peaks)}
        if name == "suffix":
            tf = 4.0 * pairs * H * d * layers / (attn_ms / 1e3) / 1e12
            out[name]["attention_roofline"] = {"bound": "tensor", "achieved": tf, "peak": peaks["bf16_tflops"],
                                               "unit": "TFLOP/s", "frac": tf / peaks["bf16_tflops"],
                                               "peak_source": peaks["source"]}
        else:
            nbytes = layers * (2 * (first + rows) * H * d * 2 + 2 * row_bytes)
            out[name]["attention_roofline"] = _hbm_roofline(nbytes, attn_ms, peaks)
    out["value"] = out["suffix"]["norm_rope_ms"] + out["suffix"]["attention_ms"]
    return [out]


def bench_fused(args):
    """Fused replay + suffix calls against separate replay and prefill launches, on the
    24-layer cache hit (3 calls of 8 layers; 256 units and 3277-token windows, so each fused
    call runs as a replay launch then a prefill launch) and on the one-layer 8K prefix at 5%
    (16 units, 410-token windows: one launch)."""
    import gated_deltanet_state_tail_b200 as gdn
    lines = []
    for wl in (inputs.stack_workload(24), inputs.single_layer_workload()):
        data = StackData(wl, "cuda", compact=True)
        rp, pp, state, o, st_out, _ = build_stack_runner(data, gdn.GDN_KERNEL_AUTO)
        fp = []
        for slots in data.launches:
            off, ml, R = data.replay_desc(slots)
            fp.append(gdn.FusedPlan(wl.H, wl.dk, wl.dv, wl.dtype, off, ml, R, data.suffix_cu(slots)))
        per = data.per_launch
        flush = torch.empty(L2_FLUSH_BYTES // 4, dtype=torch.float32, device="cuda")
        mid = torch.empty_like(state)

        def separate():
            run_step(data, rp, pp, state, o, st_out)

        def fused():
            for j, plan in enumerate(fp):
                sl = slice(j * per, (j + 1) * per)
                plan.run(data.k, data.v, data.alpha, data.beta, data.sq, data.sk, data.sv, data.sa, data.sb, o,
                         st_out[sl], state_mid=mid[sl])

        for _ in range(args.warmup):
            separate()
            fused()
        sep_ms = _time_ms(separate, 10, flush)
        ref = st_out.clone()
        fused_ms = _time_ms(fused, 10, flush)
        rel = float(((st_out - ref).norm() / ref.norm()).item())
        launches_fused = sum(p.launches for p in fp)
        for p in rp + pp + fp:
            p.check()
            p.close()
        lines.append({"metric": "fused replay + suffix prefill", "workload": wl.name, "layers": wl.layers,
                      "separate_ms": sep_ms, "fused_ms": fused_ms, "launches_separate": 2 * len(data.launches),
                      "launches_fused": launches_fused, "final_state_rel_diff_fused_vs_separate": rel,
                      "dtype": "bf16", "data": "synthetic"})
        del data, state, o, st_out, mid, flush
    return lines


# --------------------------------------------------------------------------
# reference arm: the fp64 CPU oracle as it stands
# --------------------------------------------------------------------------
def bench_reference(args, rank, world):
    if rank != 0:
        return None
    wl = inputs.stack_workload(24)
    vals = []
    for _ in range(args.warmup):
        oracle_replay_sample(wl)
    sample = None
    cores = None
    t0 = time.perf_counter()
    for _ in range(args.steps):
        v, cores, sample = oracle_replay_sample(wl)
        vals.append(v)
    wall = time.perf_counter() - t0
    value = statistics.median(vals)
    return {"impl": "reference",
            "metric": BENCH_METRIC,
            "value": value, "unit": "replayed tokens/s", "n_gpus": world, "steps": args.steps,
            "warmup": args.warmup, "ms_per_step": wall * 1e3 / max(args.steps, 1),
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64",
            "data": "synthetic (seeded q/k/v/alpha/beta; no datasets or weights)",
            "config": {"workload": wl.name, "layers": wl.layers, "heads": wl.H, "d_k": wl.dk,
                       "d_v": wl.dv, "matched_prefix": wl.match_len[0], "replay": wl.R[0],
                       "suffix": wl.suffix_len[0], "parallelism": "host cores"},
            "cpu_baseline": {"value": value, "unit": "replayed tokens/s", "cores": cores,
                             "kind": "oracle", "sample": sample},
            "e2e": {"value": value, "unit": "replayed tokens/s", "h2d_bytes_per_step": 0,
                    "d2h_bytes_per_step": 0}}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--impl", choices=["ours", "reference"], default="ours")
    ap.add_argument("--workload", default="stack",
                    choices=["stack", "sweep", "varlen", "decode", "outputs", "overlap", "fused", "hybrid"],
                    help="stack = the bench line; the others print auxiliary lines")
    ap.add_argument("--layers", type=int, default=24,
                    help="GDN layers in the stack (a multiple of 3; 24 is the bench line, "
                         "fewer only for profiling captures)")
    ap.add_argument("--kernel", choices=["auto", "recurrent", "chunked"], default="auto")
    ap.add_argument("--no-e2e", action="store_true")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-comparator", action="store_true")
    ap.add_argument("--no-extras", action="store_true",
                    help="skip the single-layer, varlen and sweep workloads of the bench line")
    args = ap.parse_args()
    if args.warmup < 3:
        raise SystemExit("--warmup must be >= 3")

    if args.impl == "reference":
        rank = int(os.environ.get("RANK", "0"))
        world = int(os.environ.get("WORLD_SIZE", "1"))
        res = bench_reference(args, rank, world)
        if res is not None:
            print(json.dumps(res), flush=True)
        return

    rank, world, local = dist_init(args.gpus)
    aux = {"sweep": bench_sweep, "varlen": bench_varlen, "decode": bench_decode, "outputs": bench_outputs,
           "overlap": bench_overlap, "fused": bench_fused, "hybrid": bench_hybrid}
    if args.workload in aux:
        if rank == 0:
            for line in aux[args.workload](args):
                print(json.dumps(line), flush=True)
        if world > 1:
            torch.distributed.destroy_process_group()
        return
    try:
        res = bench_ours(args, rank, world, local)
        if rank == 0:
            print(json.dumps(res), flush=True)
    finally:
        if world > 1:
            torch.distributed.destroy_process_group()


if __name__ == "__main__":
    main()
