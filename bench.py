#!/usr/bin/env python
"""Benchmark of the three-tier decode GEMV on a Llama-2-7B-shaped decoder block (batch one).

Workload (one step = one pass of the hot path over a batch of synthetic tokens):
  * one Llama-2-7B-shaped block: q, k, v, o 4096x4096; gate, up 11008x4096; down 4096x11008;
    bf16 N(0, 0.02) weights (seeded); q/k/v and gate/up packed as one matrix each, so a token
    runs four sites (attn-in -> qkv, o-in -> o, mlp-in -> gate/up, down-in -> down);
  * 64 tokens; block inputs fp32 Laplace(0, 1); the down input is SiLU(gate x) * (up x) from the
    block's own gate/up weights and the mlp input (fp64, prepared once, untimed);
  * tiers by |x| rank: 40% skipped, 30% 2-bit, 30% bf16 (TopK);
  * every token reads one of 32 weight replicas (round robin), as a 32-layer stack would, so all
    launches stream from HBM (inputs larger than L2; no flush needed).
A step = for each token, for each site: one spax_masked_gemv (the mask and the tiered GEMV in one
launch; tier codes, lists and counts are written as the mask writes them), captured once as a CUDA
graph (kernels chained with programmatic dependent launch) and replayed. The two-call path
(spax_build_mask + spax_tiered_gemv) and each kernel alone are timed the same way for reference.

Metric: us per token per decoder layer (lower is better), plus effective HBM GB/s of the tiered
GEMV over the bytes it must read, against the dense bf16 GEMV of the same kernel family.

Multi-GPU: replicas only (each rank decodes its own token stream on its own block; no
collective on the data path). `value` = max-over-ranks step time / (tokens x ranks).

--impl reference runs the CPU oracle (plain C, fp64) on a bounded sample of the same workload.
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

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch
import torch.distributed as dist

HIDDEN, INTER = 4096, 11008
N_TOKENS = 64
SKIP, APPROX, FULL = 0.4, 0.3, 0.3
N_REPLICAS = 32
METRIC = "\u00b5s/token per decoder layer and effective HBM GB/s (fraction of 8 TB/s), vs dense GEMV"
WORKLOAD = "llama2-7b-block-decode-b1"
# (name, d_out, d_in, input stream tensor id); q/k/v and gate/up are concatenated along d_out
SITES = [("qkv", 3 * HIDDEN, HIDDEN, 101), ("o", HIDDEN, HIDDEN, 102),
         ("gate_up", 2 * INTER, HIDDEN, 103), ("down", HIDDEN, INTER, None)]
WEIGHT_IDS = {"q": 1, "k": 2, "v": 3, "o": 4, "gate": 5, "up": 6, "down": 7}
FALLBACK_HBM_GBS = 6650.0


def workload_config(tokens: int, replicas: int, world: int) -> dict:
    """The workload description both arms print (the reference arm times a sample of it)."""
    return {"workload": WORKLOAD, "tokens_per_step": tokens,
            "tiers": {"skip": SKIP, "approx": APPROX, "full": FULL, "rule": "topk",
                      "boundary_guess": f"|x| quantiles calibrated on {N_CAL} separate tokens"},
            "weight_replicas": replicas,
            "l2": "inputs larger than L2: each token reads one of the weight replicas",
            "parallelism": f"replicas x{world}"}


def k_counts(d_in: int):
    kf = int(math.floor(FULL * d_in + 0.5))
    ka = int(math.floor(APPROX * d_in + 0.5))
    return kf, ka


# ----------------------------------------------------------------------------- distributed

def dist_setup():
    ws = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    if ws > 1 and not dist.is_initialized():
        backend = "nccl" if torch.cuda.is_available() else "gloo"
        if backend == "nccl":
            torch.cuda.set_device(local)
        import datetime
        dist.init_process_group(backend, timeout=datetime.timedelta(seconds=120))
    return rank, ws, local


def barrier():
    if dist.is_initialized():
        dist.barrier()


def max_over_ranks(v: float) -> float:
    """Max of a per-rank scalar over all ranks (the job's time is its slowest rank's)."""
    if not dist.is_initialized():
        return v
    dev = "cuda" if dist.get_backend() == "nccl" else "cpu"
    t = torch.tensor([v], dtype=torch.float64, device=dev)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def us_per_token_layer(ms_per_step: float, tokens_per_rank: int, world: int) -> float:
    """Whole-job us per token per layer: every rank decodes its own tokens through one layer."""
    return ms_per_step * 1000.0 / (tokens_per_rank * world)


# ----------------------------------------------------------------------------- clocks

class ClockSampler:
    """Samples SM clock and throttle reasons through NVML while the timed regions run."""

    REASONS = {0x1: "gpu_idle", 0x2: "applications_clocks_setting", 0x4: "sw_power_cap",
               0x8: "hw_slowdown", 0x20: "sw_thermal_slowdown", 0x40: "hw_thermal_slowdown",
               0x80: "hw_power_brake_slowdown", 0x100: "display_clock_setting"}

    def __init__(self, index: int, period_s: float = 0.005):
        self.samples, self.reasons, self.max_mhz = [], set(), None
        self._stop = threading.Event()
        self._thr = None
        try:
            import pynvml

            pynvml.nvmlInit()
            self._nv = pynvml
            self._h = pynvml.nvmlDeviceGetHandleByIndex(index)
            self.max_mhz = pynvml.nvmlDeviceGetMaxClockInfo(self._h, pynvml.NVML_CLOCK_SM)
        except Exception:
            self._nv = None
        self.period = period_s

    def _run(self):
        nv = self._nv
        while not self._stop.is_set():
            try:
                self.samples.append(nv.nvmlDeviceGetClockInfo(self._h, nv.NVML_CLOCK_SM))
                r = nv.nvmlDeviceGetCurrentClocksEventReasons(self._h)
                for bit, name in self.REASONS.items():
                    if r & bit and bit != 0x1:
                        self.reasons.add(name)
            except Exception:
                pass
            time.sleep(self.period)

    def __enter__(self):
        if self._nv is not None:
            self._thr = threading.Thread(target=self._run, daemon=True)
            self._thr.start()
        return self

    def __exit__(self, *a):
        self._stop.set()
        if self._thr:
            self._thr.join()

    def summary(self):
        return {"sm_mhz": statistics.median(self.samples) if self.samples else None,
                "sm_max_mhz": self.max_mhz, "reasons": sorted(self.reasons),
                "samples": len(self.samples)}


# ----------------------------------------------------------------------------- workload

def make_weights(device):
    from tiered_weight_gemv_b200 import synth
    W = {n: None for n in WEIGHT_IDS}
    shapes = {"q": (HIDDEN, HIDDEN), "k": (HIDDEN, HIDDEN), "v": (HIDDEN, HIDDEN),
              "o": (HIDDEN, HIDDEN), "gate": (INTER, HIDDEN), "up": (INTER, HIDDEN),
              "down": (HIDDEN, INTER)}
    for n, tid in WEIGHT_IDS.items():
        W[n] = synth.weight(*shapes[n], 0, tid, device=device)
    return {"qkv": torch.cat([W["q"], W["k"], W["v"]], 0).contiguous(), "o": W["o"],
            "gate_up": torch.cat([W["gate"], W["up"]], 0).contiguous(), "down": W["down"]}


def make_inputs(mats, n_tokens, device, seed=0):
    from tiered_weight_gemv_b200 import synth
    xs = {}
    for name, d_out, d_in, tid in SITES:
        if tid is not None:
            xs[name] = synth.laplace((n_tokens, d_in), seed, tid, device=device)
    gu = mats["gate_up"].to(torch.float64) @ xs["gate_up"].to(torch.float64).T  # [2*INTER, T]
    xs["down"] = synth.silu_gated(gu[:INTER].T, gu[INTER:].T).contiguous()
    return xs


N_CAL = 16  # calibration tokens per site: their own seed, never the timed tokens


def calibrated_guesses(mats, device):
    """Per site, the |x| quantiles at the skip and skip-or-approximate fractions of the TopK
    counts (spax_calibrate_thresholds over N_CAL separate tokens): the TopK rule takes them in
    t_skip / t_full as a guess of its boundary keys, which changes how fast the kernels find the
    boundaries but never which columns they select."""
    from tiered_weight_gemv_b200 import spax
    cal = make_inputs(mats, N_CAL, device, seed=1)
    out = {}
    for name, d_out, d_in, _ in SITES:
        kf, ka = k_counts(d_in)
        ws = torch.empty(spax.spax_workspace_bytes(spax.OP_CALIBRATE, 0, d_in), dtype=torch.uint8,
                         device=device)
        t = torch.empty(2, device=device)
        st = torch.zeros(1, dtype=torch.int32, device=device)
        spax.spax_calibrate_thresholds(cal[name], round((d_in - kf - ka) * 10000 / d_in),
                                       round((d_in - kf) * 10000 / d_in), t, st, ws)
        torch.cuda.synchronize()
        if int(st.item()) != 0:
            raise RuntimeError(f"calibration status {int(st.item())} at site {name}")
        out[name] = tuple(float(v) for v in t.cpu())  # (t_skip, t_full)
    del cal
    return out


def fused_bytes(d_out, d_in, kf, ka):
    """Bytes one masked GEMV (mask + GEMV in one launch) must move: selected weights (+ scales),
    x once, the tier codes, the two index lists and counts it writes, and the output vector."""
    from tiered_weight_gemv_b200 import spax
    return spax.spax_weight_bytes(d_out, spax.FULL_BF16, kf, ka) + 5 * d_in + (kf + ka) * 4 + d_out * 4 + 16


def algorithmic_bytes(d_out, d_in, kf, ka):
    """Bytes one tiered GEMV must move: selected weights (+ scales), the gathered x entries, the
    two index lists and the output vector."""
    from tiered_weight_gemv_b200 import spax
    return spax.spax_weight_bytes(d_out, spax.FULL_BF16, kf, ka) + (kf + ka) * 8 + d_out * 4 + 16


# ----------------------------------------------------------------------------- GPU arm

def time_graph(g, steps, warmup, stream):
    """Mean ms per replay of graph g over `steps` replays on `stream` (events on that stream)."""
    with torch.cuda.stream(stream):
        for _ in range(warmup):
            g.replay()
        torch.cuda.synchronize()
        barrier()
        start = torch.cuda.Event(enable_timing=True)
        end = torch.cuda.Event(enable_timing=True)
        start.record(stream)
        for _ in range(steps):
            g.replay()
        end.record(stream)
        torch.cuda.synchronize()
        barrier()
    return start.elapsed_time(end) / steps


def run_gpu(args, rank, world, local):
    from tiered_weight_gemv_b200 import spax

    dev = torch.device("cuda", local)
    torch.cuda.set_device(dev)
    n_tok, n_rep = args.tokens, args.replicas
    SEL = [s for s in SITES if not args.sites or s[0] in args.sites.split(",")]
    mats = make_weights(dev)
    xs = make_inputs(mats, n_tok, dev)
    guess = calibrated_guesses(mats, dev)
    host = None
    if rank == 0 and world == 1 and not args.no_cpu_baseline:
        host = ({n: m.cpu() for n, m in mats.items()}, {n: v.cpu() for n, v in xs.items()})

    # packed replicas (pack once, copy) and per-site buffers
    packed = {}
    for name, d_out, d_in, _ in SEL:
        pm = spax.alloc_packed(d_out, d_in, spax.FULL_BF16, device=dev)
        spax.spax_pack_weights(mats[name], spax.FULL_BF16, pm)
        reps = [pm] + [spax.PackedMatrix(d_out, d_in, spax.FULL_BF16, pm.full.clone(),
                                         pm.approx.clone()) for _ in range(n_rep - 1)]
        packed[name] = reps
    torch.cuda.synchronize()
    del mats
    buf = {}
    for name, d_out, d_in, _ in SEL:
        kf, ka = k_counts(d_in)
        buf[name] = dict(
            tier=torch.empty(n_tok, d_in, dtype=torch.uint8, device=dev),
            fidx=torch.empty(n_tok, d_in, dtype=torch.int32, device=dev),
            aidx=torch.empty(n_tok, d_in, dtype=torch.int32, device=dev),
            counts=torch.empty(n_tok, 4, dtype=torch.int32, device=dev),
            y=torch.empty(n_tok, d_out, dtype=torch.float32, device=dev),
            yd=torch.empty(n_tok, d_out, dtype=torch.float32, device=dev),
            yc=torch.empty(n_tok, d_out, dtype=torch.float32, device=dev),
            status=torch.zeros(1, dtype=torch.int32, device=dev),
            ws=spax.alloc_workspace(spax.OP_TIERED_GEMV, d_out, d_in, device=dev),
            dws=spax.alloc_workspace(spax.OP_DENSE_GEMV, d_out, d_in, device=dev),
            prm=spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka, t_skip=guess[name][0],
                                 t_full=guess[name][1]),
            prm_unguessed=spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka),
            prm_missed=spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka,
                                        t_skip=2 * guess[name][0], t_full=2 * guess[name][1]),
            desc=[pm.desc() for pm in packed[name]],
            kf=kf, ka=ka)

    def step_tiered(mask=True, gemv=True, sites=None):
        for t in range(n_tok):
            for name, d_out, d_in, _ in SEL:
                if sites is not None and name not in sites:
                    continue
                b = buf[name]
                if mask:
                    spax.spax_build_mask(xs[name][t], b["prm"], b["tier"][t], b["fidx"][t],
                                         b["aidx"][t], b["counts"][t], b["status"])
                if gemv:
                    pm = packed[name][t % n_rep]
                    spax.spax_tiered_gemv(pm, xs[name][t], b["fidx"][t], b["aidx"][t],
                                          b["counts"][t], b["y"][t], b["status"], b["ws"],
                                          desc=b["desc"][t % n_rep])

    def step_fused(sites=None, prm="prm", xsrc=None, ydst=None):
        """The headline step: one spax_masked_gemv per token and site (mask outputs written).
        xsrc / ydst: other input / output buffers (the end-to-end run's second set)."""
        xsrc = xs if xsrc is None else xsrc
        for t in range(n_tok):
            for name, d_out, d_in, _ in SEL:
                if sites is not None and name not in sites:
                    continue
                b = buf[name]
                y = b["y"] if ydst is None else ydst[name]
                spax.spax_masked_gemv(packed[name][t % n_rep], xsrc[name][t], b[prm], y[t],
                                      b["status"], b["ws"], tier=b["tier"][t],
                                      full_idx=b["fidx"][t], approx_idx=b["aidx"][t],
                                      counts=b["counts"][t], desc=b["desc"][t % n_rep])

    def step_chained():
        """The decoder layer's MLP chained on the device: down's input is formed inside its
        launch from the tiered gate/up output, x = silu(g) * u (informational; the headline feeds
        every site its prepared input so each site's parity stands alone)."""
        for t in range(n_tok):
            for name, d_out, d_in, _ in SEL:
                b = buf[name]
                if name == "down" and "gate_up" in buf:
                    spax.spax_masked_gemv_swiglu(packed[name][t % n_rep], buf["gate_up"]["y"][t],
                                                 b["prm"], b["yc"][t], b["status"], b["ws"],
                                                 desc=b["desc"][t % n_rep])
                else:
                    spax.spax_masked_gemv(packed[name][t % n_rep], xs[name][t], b["prm"], b["y"][t],
                                          b["status"], b["ws"], desc=b["desc"][t % n_rep])

    def step_dense(sites=None):
        for t in range(n_tok):
            for name, d_out, d_in, _ in SEL:
                if sites is not None and name not in sites:
                    continue
                b = buf[name]
                spax.spax_dense_gemv(packed[name][t % n_rep].full, xs[name][t], b["yd"][t],
                                     d_out, d_in, b["status"], b["dws"])

    stream = torch.cuda.Stream(device=dev)
    graphs = {}
    with torch.cuda.stream(stream):
        step_fused()
        step_tiered()  # eager run: fills the lists used by the GEMV-only graphs
        step_dense()
    torch.cuda.synchronize()
    for name, *_ in SEL:
        st = int(buf[name]["status"].item())
        if st != 0:
            raise RuntimeError(f"device status {st} ({spax.status_string(st)}) at site {name}")

    def capture(fn, *a, **k):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            fn(*a, **k)
        return g

    graphs["fused"] = capture(step_fused)
    # the end-to-end run's second buffer set: step i uses set i % 2, so the copies of one step
    # overlap the compute of its neighbours
    names = [s[0] for s in SEL]  # the sites this run executes
    xs_b = {n: xs[n].clone() for n in names}
    y_b = {n: torch.empty_like(buf[n]["y"]) for n in names}
    graphs["fused_b"] = capture(step_fused, xsrc=xs_b, ydst=y_b)
    graphs["fused_unguessed"] = capture(step_fused, prm="prm_unguessed")
    graphs["fused_missed"] = capture(step_fused, prm="prm_missed")
    graphs["tiered"] = capture(step_tiered)
    graphs["dense"] = capture(step_dense)
    graphs["chained"] = capture(step_chained)
    for name, *_ in SEL:
        graphs["fused_" + name] = capture(step_fused, sites=[name])
        graphs["gemv_" + name] = capture(step_tiered, mask=False, gemv=True, sites=[name])
        graphs["mask_" + name] = capture(step_tiered, mask=True, gemv=False, sites=[name])
        graphs["dense_" + name] = capture(step_dense, sites=[name])

    res = {}
    sampler = ClockSampler(local)
    with sampler:
        res["fused"] = max_over_ranks(time_graph(graphs["fused"], args.steps, args.warmup, stream))
        res["fused_unguessed"] = max_over_ranks(
            time_graph(graphs["fused_unguessed"], args.steps, args.warmup, stream))
        res["fused_missed"] = max_over_ranks(
            time_graph(graphs["fused_missed"], args.steps, args.warmup, stream))
        res["tiered"] = max_over_ranks(time_graph(graphs["tiered"], args.steps, args.warmup, stream))
        res["dense"] = max_over_ranks(time_graph(graphs["dense"], args.steps, args.warmup, stream))
        res["chained"] = max_over_ranks(time_graph(graphs["chained"], args.steps, args.warmup, stream))
        for name, *_ in SEL:
            res["fused_" + name] = max_over_ranks(
                time_graph(graphs["fused_" + name], args.steps, args.warmup, stream))
            res["gemv_" + name] = max_over_ranks(
                time_graph(graphs["gemv_" + name], args.steps, args.warmup, stream))
            res["mask_" + name] = max_over_ranks(
                time_graph(graphs["mask_" + name], args.steps, args.warmup, stream))
            res["dense_" + name] = max_over_ranks(
                time_graph(graphs["dense_" + name], args.steps, args.warmup, stream))
        # end to end: every step copies its inputs in from pinned host memory and its outputs
        # back, through the same C-ABI calls. Two buffer sets, a copy-in and a copy-out stream:
        # step i's copies overlap the compute of steps i - 1 and i + 1 (events keep each set's
        # copy-in after the compute two steps back, and its compute after that step's copy-out).
        xin = {n: xs[n].cpu().pin_memory() for n in names}
        yout = {n: torch.empty(buf[n]["y"].shape, dtype=torch.float32).pin_memory() for n in names}
        h2d = sum(v.numel() * 4 for v in xin.values())
        d2h = sum(v.numel() * 4 for v in yout.values())
        sets = [(xs, {n: buf[n]["y"] for n in names}, graphs["fused"]),
                (xs_b, y_b, graphs["fused_b"])]
        s_in, s_out = torch.cuda.Stream(device=dev), torch.cuda.Stream(device=dev)
        ev_in = [torch.cuda.Event(), torch.cuda.Event()]
        ev_comp = [torch.cuda.Event(), torch.cuda.Event()]
        ev_out = [torch.cuda.Event(), torch.cuda.Event()]

        def e2e_run(n_steps, start=None):
            if start is not None:
                s_in.wait_event(start)
                s_out.wait_event(start)
            for i in range(n_steps):
                k = i % 2
                xd, yd, g = sets[k]
                with torch.cuda.stream(s_in):
                    if i >= 2:
                        s_in.wait_event(ev_comp[k])
                    for n in names:
                        xd[n].copy_(xin[n], non_blocking=True)
                    ev_in[k].record(s_in)
                with torch.cuda.stream(stream):
                    stream.wait_event(ev_in[k])
                    if i >= 2:
                        stream.wait_event(ev_out[k])
                    g.replay()
                    ev_comp[k].record(stream)
                with torch.cuda.stream(s_out):
                    s_out.wait_event(ev_comp[k])
                    for n in names:
                        yout[n].copy_(yd[n], non_blocking=True)
                    ev_out[k].record(s_out)
            for k in range(min(2, n_steps)):
                stream.wait_event(ev_out[k])

        e2e_run(max(2, args.warmup))
        torch.cuda.synchronize()
        barrier()
        s0, s1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        s0.record(stream)
        e2e_run(args.steps, start=s0)
        s1.record(stream)
        torch.cuda.synchronize()
        barrier()
        res["e2e"] = max_over_ranks(s0.elapsed_time(s1) / args.steps)
    for name, *_ in SEL:
        st = int(buf[name]["status"].item())
        if st != 0:
            raise RuntimeError(f"device status {st} after timing at site {name}")
        if not torch.isfinite(buf[name]["y"]).all() or not torch.isfinite(y_b[name]).all():
            raise RuntimeError(f"non-finite output at site {name}")
        if not torch.equal(buf[name]["y"], y_b[name]):  # same inputs, same launches
            raise RuntimeError(f"the two end-to-end buffer sets disagree at site {name}")

    launches_per_step = n_tok * len(SEL)
    sites = {}
    tot_bytes = tot_ms = 0.0
    for name, d_out, d_in, _ in SEL:
        b = buf[name]
        by = algorithmic_bytes(d_out, d_in, b["kf"], b["ka"])
        fb = fused_bytes(d_out, d_in, b["kf"], b["ka"])
        ms = res["gemv_" + name]
        fms = res["fused_" + name]
        tot_bytes += fb * n_tok
        tot_ms += fms
        S, R = spax.spax_gemv_plan(spax.OP_TIERED_GEMV, d_out, d_in)
        sites[name] = {"d_out": d_out, "d_in": d_in, "n_full": b["kf"], "n_approx": b["ka"],
                       "masked_gemv_us": round(fms * 1000 / n_tok, 3),
                       "masked_gemv_bytes_per_launch": fb,
                       "masked_gemv_GBps": round(fb * n_tok / (fms * 1e-3) / 1e9, 1),
                       "gemv_us": round(ms * 1000 / n_tok, 3),
                       "mask_us": round(res["mask_" + name] * 1000 / n_tok, 3),
                       "bytes_per_launch": by,
                       "gemv_GBps": round(by * n_tok / (ms * 1e-3) / 1e9, 1),
                       "dense_us": round(res["dense_" + name] * 1000 / n_tok, 3),
                       "dense_GBps": round(2 * d_out * d_in * n_tok / (res["dense_" + name] * 1e-3) / 1e9, 1),
                       "splits": S, "row_tile": R}
    return res, sites, tot_bytes, tot_ms, launches_per_step, h2d, d2h, sampler.summary(), host


# ----------------------------------------------------------------------------- extra measurements

LLAMA3_SITES = [("qkv", 6144, 4096, 201), ("o", 4096, 4096, 202), ("gate_up", 28672, 4096, 203),
                ("down", 4096, 14336, 204)]
LLAMA3_POINTS = [(f, a) for f in (0.1, 0.2, 0.3) for a in (0.2, 0.3)]
LLAMA3_LAYERS, LLAMA3_TOKENS = 32, 256
GUIDED_TARGETS = (0.3, 0.5, 0.7)
GUIDED_DELTA_BP = 100
N_GUIDED_CAL = 512  # calibration tokens per (layer, site) for the guided thresholds
N_SENS_CAL = 16     # calibration tokens per (layer, site) for the measured sensitivity
S_PROBE_BP = 5000   # probe sparsity of the sensitivity pass
L70_SITES = [("gate_up", 2 * 28672, 8192, 401), ("down", 8192, 28672, 402)]
L70_TOKENS = 128
L70_SPLITS = [(0.5, 0.25, 0.25), (0.7, 0.15, 0.15)]  # skip / approx / full
L2_BYTES = 126 * 2 ** 20


def _replicas_for(bytes_per_replica: float) -> int:
    """Weight replicas so that a round robin over them reads at least 3x L2 between reuses."""
    return max(4, math.ceil(3 * L2_BYTES / bytes_per_replica))


def _k(frac: float, d: int) -> int:
    return int(math.floor(frac * d + 0.5))


def _timed_graph(fn, stream, steps, warmup):
    """Run fn once eagerly, capture it as one CUDA graph and time its replays (ms per replay)."""
    with torch.cuda.stream(stream):
        fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        fn()
    ms = time_graph(g, steps, warmup, stream)
    del g
    return ms


def run_dequant(args, dev):
    """Dequantisation against loading on 4096x4096 and 22016x4096: all-bf16, all-2-bit, mixed
    25/25 and all-2-bit on one L2-resident weight copy, each through the masked GEMV and through
    the list-driven GEMV on lists built beforehand (no selection in the timed launches). The
    list-driven all-2-bit L2-resident case is the decode's own cost, without HBM or selection."""
    from tiered_weight_gemv_b200 import spax, synth

    n_tok = 16
    steps, warmup = max(5, min(args.steps, 20)), args.warmup
    stream = torch.cuda.Stream(device=dev)
    out = {}
    for label, d_out, d_in, tid in [("proj_4096x4096", 4096, 4096, 301),
                                    ("gate_up_22016x4096", 22016, 4096, 302)]:
        W = synth.weight(d_out, d_in, 6, tid, device=dev)
        pm = spax.alloc_packed(d_out, d_in, spax.FULL_BF16, device=dev)
        spax.spax_pack_weights(W, spax.FULL_BF16, pm)
        reps = [pm] + [spax.PackedMatrix(d_out, d_in, spax.FULL_BF16, pm.full.clone(), pm.approx.clone())
                       for _ in range(_replicas_for(2.3 * d_out * d_in) - 1)]
        del W
        X = synth.laplace((n_tok, d_in), 6, tid + 10, device=dev)
        y = torch.empty(n_tok, d_out, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        ws = spax.alloc_workspace(spax.OP_TIERED_GEMV, d_out, d_in, device=dev)
        descs = [r.desc() for r in reps]
        tier = torch.empty(n_tok, d_in, dtype=torch.uint8, device=dev)
        fi = torch.empty(n_tok, d_in, dtype=torch.int32, device=dev)
        ai = torch.empty(n_tok, d_in, dtype=torch.int32, device=dev)
        cnt = torch.empty(n_tok, 4, dtype=torch.int32, device=dev)
        q = _k(0.25, d_in)
        rows = {}
        for case, kf, ka, rotate in [("all_full", d_in, 0, True), ("all_approx", 0, d_in, True),
                                     ("mixed_25_25", q, q, True),
                                     ("all_approx_l2_resident", 0, d_in, False)]:
            prm = spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka)
            for t in range(n_tok):  # the lists of the list-driven arm, built outside the timing
                spax.spax_build_mask(X[t], prm, tier[t], fi[t], ai[t], cnt[t], st)

            def masked(prm=prm, rotate=rotate):
                for t in range(n_tok):
                    r = t % len(reps) if rotate else 0
                    spax.spax_masked_gemv(reps[r], X[t], prm, y[t], st, ws, desc=descs[r])

            def listed(rotate=rotate):
                for t in range(n_tok):
                    r = t % len(reps) if rotate else 0
                    spax.spax_tiered_gemv(reps[r], X[t], fi[t], ai[t], cnt[t], y[t], st, ws,
                                          desc=descs[r])

            ms = _timed_graph(masked, stream, steps, warmup)
            ms_l = _timed_graph(listed, stream, steps, warmup)
            by = fused_bytes(d_out, d_in, kf, ka)
            by_l = algorithmic_bytes(d_out, d_in, kf, ka)
            rows[case] = {"masked_us": round(ms * 1000 / n_tok, 3), "masked_bytes": by,
                          "masked_GBps": round(by * n_tok / (ms * 1e-3) / 1e9, 1),
                          "list_driven_us": round(ms_l * 1000 / n_tok, 3), "list_driven_bytes": by_l,
                          "list_driven_GBps": round(by_l * n_tok / (ms_l * 1e-3) / 1e9, 1),
                          "selection_us": round((ms - ms_l) * 1000 / n_tok, 3)}
        if int(st.item()) != 0:
            raise RuntimeError(f"device status {int(st.item())} in the dequant runs ({label})")
        rows["replicas"] = len(reps)
        out[label] = rows
        del reps, descs, ws, X, y, tier, fi, ai, cnt
        torch.cuda.empty_cache()
    out["note"] = ("list_driven_* time spax_tiered_gemv on lists built beforehand (no selection in "
                   "the timed launches); selection_us = masked - list-driven; the all-2-bit "
                   "L2-resident list-driven case is the 2-bit decode's own cost")
    return out


def run_llama3_stack(args, dev):
    """The Llama-3-8B-shaped projection stack at its stated size: 32 layers with their own
    seeded weights, 256 tokens of Laplace activations per site and layer, every launch on weights
    no other launch of the step shares (6.5 GB of packed pools: L2-cold).
      * The (full, approx) sweep with TopK masks, with and without calibrated boundary-key
        guesses, and its fit time = c0 + bytes/BW (the ByteCross abstract's method).
      * The dense GEMV and torch.mv (cuBLAS) over the same stack.
      * The measured block sensitivity (TopK-Guided §2.2) at probe sparsity 0.5 on calibration
        tokens, and the TopK-Guided masks at targets 0.3 / 0.5 / 0.7 (±0.01): per-layer
        thresholds calibrated on 512 tokens, per-block budgets (λ = 0.5, clamp [0.05, 0.95])
        from the synthetic profile and from the measured sensitivity; bytes counted from the
        realised lists of every launch."""
    from tiered_weight_gemv_b200 import spax, synth

    L, T = LLAMA3_LAYERS, LLAMA3_TOKENS
    steps, warmup = 3, args.warmup
    stream = torch.cuda.Stream(device=dev)
    names = [s[0] for s in LLAMA3_SITES]
    pm, X = {}, {}
    for l in range(L):
        for name, d_out, d_in, tid in LLAMA3_SITES:
            W = synth.weight(d_out, d_in, 7, 1000 * l + tid, device=dev)
            p = spax.alloc_packed(d_out, d_in, spax.FULL_BF16, device=dev)
            spax.spax_pack_weights(W, spax.FULL_BF16, p)
            pm[l, name] = p
            X[l, name] = synth.laplace((T, d_in), 7, 100000 + 1000 * l + tid, device=dev)
            del W
    torch.cuda.synchronize()
    desc = {k: v.desc() for k, v in pm.items()}
    shape = {name: (d_out, d_in) for name, d_out, d_in, _ in LLAMA3_SITES}
    ws = {n: spax.alloc_workspace(spax.OP_TIERED_GEMV, *shape[n], device=dev) for n in names}
    dws = {n: spax.alloc_workspace(spax.OP_DENSE_GEMV, *shape[n], device=dev) for n in names}
    y = {n: torch.empty(T, shape[n][0], device=dev) for n in names}
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    cal_ws = {n: torch.empty(spax.spax_workspace_bytes(spax.OP_CALIBRATE, 0, shape[n][1]),
                             dtype=torch.uint8, device=dev) for n in names}
    t2 = torch.empty(2, device=dev)

    def calibrate(cal, d_in, s_skip, s_below_full, name):
        spax.spax_calibrate_thresholds(cal, round(s_skip * 10000), round(s_below_full * 10000), t2,
                                       st, cal_ws[name])
        return tuple(float(v) for v in t2.cpu())

    def run_masked(prm):
        for t in range(T):
            for l in range(L):
                for n in names:
                    spax.spax_masked_gemv(pm[l, n], X[l, n][t], prm[l, n], y[n][t], st, ws[n],
                                          desc=desc[l, n])

    out = {"layers": L, "tokens": T, "sites": {n: list(shape[n]) for n in names},
           "packed_GB": round(sum(v.full.numel() + v.approx.numel() for v in pm.values()) / 1e9, 2)}
    # ---- config 3: the (full, approx) sweep ----
    guess_cal = {(l, n): synth.laplace((N_CAL, shape[n][1]), 8, 200000 + 1000 * l + i, device=dev)
                 for l in range(L) for i, n in enumerate(names)}
    points = []
    for f, a in LLAMA3_POINTS:
        prms, prms0 = {}, {}
        for l in range(L):
            for n in names:
                d_in = shape[n][1]
                kf, ka = _k(f, d_in), _k(a, d_in)
                ts, tf = calibrate(guess_cal[l, n], d_in, (d_in - kf - ka) / d_in, (d_in - kf) / d_in, n)
                prms[l, n] = spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka, t_skip=ts, t_full=tf)
                prms0[l, n] = spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka)
        ms = _timed_graph(lambda: run_masked(prms), stream, steps, warmup)
        ms0 = _timed_graph(lambda: run_masked(prms0), stream, steps, warmup)
        by = sum(fused_bytes(*shape[n], _k(f, shape[n][1]), _k(a, shape[n][1])) for n in names)
        us = ms * 1000 / (T * L)
        points.append({"full": f, "approx": a, "us_per_token_layer": round(us, 3),
                       "unguessed_us_per_token_layer": round(ms0 * 1000 / (T * L), 3),
                       "bytes_per_token_layer": by, "GBps": round(by / (us * 1e-6) / 1e9, 1),
                       "frac_of_8TBps": round(by / (us * 1e-6) / 8e12, 4)})
    del guess_cal
    if int(st.item()) != 0:
        raise RuntimeError(f"device status {int(st.item())} in the Llama-3 sweep")
    out["points"] = points
    out["fit_time_vs_bytes"] = fit_c0_bw([(p["bytes_per_token_layer"], p["us_per_token_layer"]) for p in points])
    out["unguessed_fit_time_vs_bytes"] = fit_c0_bw([(p["bytes_per_token_layer"], p["unguessed_us_per_token_layer"]) for p in points])
    out["guess_note"] = ("the TopK parameters carry |x| quantiles calibrated on 16 separate tokens per "
                         "layer, site and point; unguessed_* is the same launches without them")

    def run_dense():
        for t in range(T):
            for l in range(L):
                for n in names:
                    spax.spax_dense_gemv(pm[l, n].full, X[l, n][t], y[n][t], *shape[n], st, dws[n])

    Xh = {k: v.to(torch.bfloat16) for k, v in X.items()}

    def run_mv():
        for t in range(T):
            for l in range(L):
                for n in names:
                    d_out, d_in = shape[n]
                    torch.mv(pm[l, n].full.view(torch.bfloat16).view(d_in, d_out).t(), Xh[l, n][t])

    dense_bytes = sum(2 * d_out * d_in for d_out, d_in in shape.values())
    ms_d = _timed_graph(run_dense, stream, steps, warmup)
    ms_mv = _timed_graph(run_mv, stream, steps, warmup)
    del Xh
    out["dense_us_per_token_layer"] = round(ms_d * 1000 / (T * L), 3)
    out["dense_GBps"] = round(dense_bytes * T * L / (ms_d * 1e-3) / 1e9, 1)
    out["torch_mv_bf16_us_per_token_layer"] = round(ms_mv * 1000 / (T * L), 3)
    out["torch_mv_note"] = "cuBLAS through torch.mv on the same bf16 pools with bf16 x (sanity figure)"

    # ---- the measured block sensitivity (TopK-Guided §2.2) ----
    y2 = {n: torch.empty(2 * shape[n][0], device=dev) for n in names}
    acc = torch.zeros(L, len(names), 2, dtype=torch.float64, device=dev)
    for l in range(L):
        for i, n in enumerate(names):
            cal = synth.laplace((N_SENS_CAL, shape[n][1]), 9, 300000 + 1000 * l + i, device=dev)
            spax.spax_probe_sensitivity(pm[l, n], cal, S_PROBE_BP, y2[n], acc[l, i], st, ws[n],
                                        desc=desc[l, n])
    a = acc.cpu().numpy()
    sens_meas = np.sqrt(a[:, :, 0].sum(1) / a[:, :, 1].sum(1))
    sens_syn = 1.0 + 3.0 * np.exp(-np.arange(L) / 4.0)
    out["sensitivity"] = {"probe_sparsity": S_PROBE_BP / 10000, "calibration_tokens": N_SENS_CAL,
                          "measured": [round(float(v), 6) for v in sens_meas],
                          "synthetic_profile": "1 + 3 exp(-b/4)"}

    # ---- config 4: TopK-Guided masks on the stack ----
    cnt = torch.zeros(T, L, len(names), 4, dtype=torch.int32, device=dev)

    def run_guided(prm):
        for t in range(T):
            for l in range(L):
                for i, n in enumerate(names):
                    spax.spax_masked_gemv(pm[l, n], X[l, n][t], prm[l, n], y[n][t], st, ws[n],
                                          counts=cnt[t, l, i], desc=desc[l, n])

    guided = []
    for src, sens in (("synthetic", sens_syn), ("measured", sens_meas)):
        for s in GUIDED_TARGETS:
            s_b = spax.spax_block_budgets(sens, s, 0.5, 0.05, 0.95)
            prm = {}
            for l in range(L):
                s1 = float(s_b[l])
                s2 = s1 + (1.0 - s1) / 2.0  # the kept budget split evenly between the tiers
                for i, n in enumerate(names):
                    d_in = shape[n][1]
                    cal = synth.laplace((N_GUIDED_CAL, d_in), 10, 400000 + 1000 * l + i, device=dev)
                    ts, tf = calibrate(cal, d_in, s1, s2, n)
                    prm[l, n] = spax.mask_params(spax.MASK_GUIDED, t_skip=ts, t_full=tf,
                                                 s_skip_bp=round(s1 * 10000),
                                                 s_below_full_bp=round(s2 * 10000),
                                                 delta_bp=GUIDED_DELTA_BP)
                    del cal
            ms = _timed_graph(lambda: run_guided(prm), stream, steps, warmup)
            c = cnt.cpu().numpy().astype(np.int64)  # realised counts of the last replay
            nbytes = 0
            skip_dev = 0.0
            for l in range(L):
                for i, n in enumerate(names):
                    d_out, d_in = shape[n]
                    nf, na = c[:, l, i, 0], c[:, l, i, 1]
                    nbytes += sum(fused_bytes(d_out, d_in, int(f_), int(a_)) for f_, a_ in zip(nf, na))
                    real = (d_in - nf - na) / d_in
                    skip_dev = max(skip_dev, float(np.max(np.abs(real - round(float(s_b[l]) * 10000) / 10000))))
            us = ms * 1000 / (T * L)
            bpt = nbytes / (T * L)
            guided.append({"budgets_from": src, "target": s, "us_per_token_layer": round(us, 3),
                           "realised_bytes_per_token_layer": round(bpt),
                           "GBps": round(bpt / (us * 1e-6) / 1e9, 1),
                           "frac_of_8TBps": round(bpt / (us * 1e-6) / 8e12, 4),
                           "max_realised_skip_deviation": round(skip_dev, 5),
                           "block_budget_range": [round(float(s_b.min()), 4), round(float(s_b.max()), 4)]})
    if int(st.item()) != 0:
        raise RuntimeError(f"device status {int(st.item())} in the guided runs")
    out["topk_guided"] = guided
    out["topk_guided_note"] = ("guided rule, delta 0.01; thresholds per layer and site from 512 "
                               "calibration tokens; block budgets lambda 0.5, clamp [0.05, 0.95]; "
                               "bytes from the counts each launch wrote; the skip deviation is the "
                               "largest |realised - block target| over all launches (at most 0.01)")
    del pm, X, desc, y, ws, dws
    torch.cuda.empty_cache()
    return out


def run_llama2_70b_mlp(args, dev):
    """The Llama-2-70B-shaped MLP with the int4 full tier (group 128, symmetric) and the 2-bit
    approximate tier: gate/up (concatenated, 57344x8192) and down (8192x28672), 128 tokens of
    Laplace activations at each site, tiers 50/25/25 and 70/15/15 by |x| rank, against the same
    kernel with every column in the int4 tier (dense in the same weight format)."""
    from tiered_weight_gemv_b200 import spax, synth

    T = L70_TOKENS
    steps, warmup = max(3, min(args.steps, 10)), args.warmup
    stream = torch.cuda.Stream(device=dev)
    per_rep = sum(spax.spax_pack_bytes(d_out, d_in, spax.FULL_INT4_G128)[0] +
                  spax.spax_pack_bytes(d_out, d_in, spax.FULL_INT4_G128)[1]
                  for _, d_out, d_in, _ in L70_SITES)
    n_rep = _replicas_for(per_rep)
    reps, X, y, ws = {}, {}, {}, {}
    for name, d_out, d_in, tid in L70_SITES:
        W = synth.weight(d_out, d_in, 11, tid, device=dev)
        p = spax.alloc_packed(d_out, d_in, spax.FULL_INT4_G128, device=dev)
        spax.spax_pack_weights(W, spax.FULL_INT4_G128, p)
        del W
        torch.cuda.synchronize()
        reps[name] = [p] + [spax.PackedMatrix(d_out, d_in, spax.FULL_INT4_G128, p.full.clone(),
                                              p.approx.clone()) for _ in range(n_rep - 1)]
        X[name] = synth.laplace((T, d_in), 11, tid + 10, device=dev)
        y[name] = torch.empty(T, d_out, device=dev)
        ws[name] = spax.alloc_workspace(spax.OP_TIERED_GEMV, d_out, d_in, device=dev)
    desc = {n: [r.desc() for r in reps[n]] for n in reps}
    st = torch.zeros(1, dtype=torch.int32, device=dev)

    def run(split):
        for t in range(T):
            for name, d_out, d_in, _ in L70_SITES:
                _, a, f = split
                prm = spax.mask_params(spax.MASK_TOPK, k_full=_k(f, d_in), k_approx=_k(a, d_in))
                spax.spax_masked_gemv(reps[name][t % n_rep], X[name][t], prm, y[name][t], st,
                                      ws[name], desc=desc[name][t % n_rep])

    def bytes_of(split):
        _, a, f = split
        return sum(spax.spax_weight_bytes(d_out, spax.FULL_INT4_G128, _k(f, d_in), _k(a, d_in)) +
                   5 * d_in + 4 * (_k(f, d_in) + _k(a, d_in)) + 4 * d_out + 16
                   for _, d_out, d_in, _ in L70_SITES)

    out = {"sites": {n: [d_out, d_in] for n, d_out, d_in, _ in L70_SITES}, "tokens": T,
           "replicas": n_rep, "full_tier": "int4 g128 symmetric", "splits": []}
    dense = (0.0, 0.0, 1.0)
    ms_dense = _timed_graph(lambda: run(dense), stream, steps, warmup)
    for split in L70_SPLITS:
        ms = _timed_graph(lambda: run(split), stream, steps, warmup)
        us = ms * 1000 / T
        by = bytes_of(split)
        out["splits"].append({"skip": split[0], "approx": split[1], "full": split[2],
                              "us_per_token_mlp": round(us, 3), "bytes_per_token_mlp": by,
                              "GBps": round(by / (us * 1e-6) / 1e9, 1),
                              "frac_of_8TBps": round(by / (us * 1e-6) / 8e12, 4),
                              "speedup_vs_dense_int4": round(ms_dense / ms, 3)})
    by_d = bytes_of(dense)
    out["dense_int4_us_per_token_mlp"] = round(ms_dense * 1000 / T, 3)
    out["dense_int4_GBps"] = round(by_d / (ms_dense * 1e-3 / T) / 1e9, 1)
    if int(st.item()) != 0:
        raise RuntimeError(f"device status {int(st.item())} in the 70B MLP runs")
    del reps, desc, X, y, ws
    torch.cuda.empty_cache()
    return out


def run_scaled_guess(args, dev):
    """The headline's masked GEMV chain on tokens whose scale varies: each token of every site is
    multiplied by its own LogUniform[0.5, 2] factor. Three ways to pass the boundary-key guess:
    the headline's absolute quantiles (calibrated on unit-scale tokens, so most windows miss),
    TOPK_SCALED with the same quantiles divided by the calibration tokens' mean |x| (the window
    follows each token's mean), and no guess. All three select the same columns."""
    from tiered_weight_gemv_b200 import spax, synth

    n_tok = 16
    steps, warmup = max(5, min(args.steps, 20)), args.warmup
    stream = torch.cuda.Stream(device=dev)
    mats = make_weights(dev)
    xs = make_inputs(mats, n_tok, dev, seed=2)
    cal = make_inputs(mats, N_CAL, dev, seed=1)
    guess = calibrated_guesses(mats, dev)
    sites = []
    for name, d_out, d_in, tid in SITES:
        scale = synth.log_uniform((n_tok,), 2, 700 + (tid or 0), 0.5, 2.0, device=dev)
        x = (xs[name].double() * scale.double()[:, None]).float().contiguous()
        mean_cal = float(cal[name].abs().double().mean())
        kf, ka = k_counts(d_in)
        pm = spax.alloc_packed(d_out, d_in, spax.FULL_BF16, device=dev)
        spax.spax_pack_weights(mats[name], spax.FULL_BF16, pm)
        reps = [pm] + [spax.PackedMatrix(d_out, d_in, spax.FULL_BF16, pm.full.clone(), pm.approx.clone())
                       for _ in range(3)]
        prms = {"absolute": spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka,
                                             t_skip=guess[name][0], t_full=guess[name][1]),
                "scaled": spax.mask_params(spax.MASK_TOPK_SCALED, k_full=kf, k_approx=ka,
                                           t_skip=guess[name][0] / mean_cal,
                                           t_full=guess[name][1] / mean_cal),
                "none": spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka)}
        sites.append(dict(x=x, reps=reps, descs=[r.desc() for r in reps], prms=prms,
                          y=torch.empty(n_tok, d_out, device=dev),
                          ws=spax.alloc_workspace(spax.OP_TIERED_GEMV, d_out, d_in, device=dev)))
    del mats, cal
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    out = {"tokens": n_tok, "token_scale": "LogUniform[0.5, 2] per token and site"}
    for how in ("absolute", "scaled", "none"):
        def step(how=how):
            for t in range(n_tok):
                for sd in sites:
                    r = t % len(sd["reps"])
                    spax.spax_masked_gemv(sd["reps"][r], sd["x"][t], sd["prms"][how], sd["y"][t], st,
                                          sd["ws"], desc=sd["descs"][r])
        ms = _timed_graph(step, stream, steps, warmup)
        out[f"{how}_guess_us_per_token_layer"] = round(ms * 1000 / n_tok, 3)
    if int(st.item()) != 0:
        raise RuntimeError(f"device status {int(st.item())} in the scaled-guess runs")
    del sites
    torch.cuda.empty_cache()
    return out


HEADS, HEAD_DIM, KV_PAGE = 32, 128, 16  # the block's attention: one key head for each query head
LAYER_CONTEXTS = (512, 4096)


def run_decode_layer(args, dev):
    """The whole decoder layer of the headline's block as a decoder runs it, one token at a time:
    qkv, cache append with rotation, attention over the paged cache, o, residual norm, gate/up, down
    (fed in its own launch), and the last residual sum with the next layer's first norm, which are one
    call (so a layer begins with its normed input at hand). Each token reads its own weight replica and
    cache, so all of it streams from HBM. Beside it, the four projections alone on the same inputs: the
    difference is what the steps between them add."""
    from tiered_weight_gemv_b200 import spax, synth

    n_tok, n_rep = 16, 4
    steps, warmup = max(5, min(args.steps, 20)), args.warmup
    stream = torch.cuda.Stream(device=dev)
    mats = make_weights(dev)
    sites = {}
    for name, d_out, d_in, _ in SITES:
        kf, ka = k_counts(d_in)
        pm = spax.alloc_packed(d_out, d_in, spax.FULL_BF16, device=dev)
        spax.spax_pack_weights(mats[name], spax.FULL_BF16, pm)
        reps = [pm] + [spax.PackedMatrix(d_out, d_in, spax.FULL_BF16, pm.full.clone(), pm.approx.clone())
                       for _ in range(n_rep - 1)]
        sites[name] = dict(reps=reps, descs=[r.desc() for r in reps],
                           prm=spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka),
                           y=torch.empty(n_tok, d_out, device=dev),
                           ws=spax.alloc_workspace(spax.OP_TIERED_GEMV, d_out, d_in, device=dev))
    del mats
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    ones = torch.ones(HIDDEN, dtype=torch.bfloat16, device=dev)
    norm = spax.Norm(ones)
    rope = spax.Rope(10000.0 ** (-torch.arange(HEAD_DIM // 2, dtype=torch.float64, device=dev)
                                 / (HEAD_DIM // 2)))
    h = synth.laplace((n_tok, 1, HIDDEN), 0, 801, device=dev)
    x1, r, x2, r2, x3 = (torch.empty_like(h) for _ in range(5))
    spax.spax_residual_norm(h, None, None, x1, pre=norm)
    att = torch.empty(n_tok, 1, HEADS, HEAD_DIM, device=dev)
    out = {"tokens": n_tok, "weight_replicas": n_rep, "heads": HEADS, "head_dim": HEAD_DIM,
           "cache": "bf16, pages of %d" % KV_PAGE}

    def gemv(name, t, x):
        s = sites[name]
        spax.spax_masked_gemv(s["reps"][t % n_rep], x, s["prm"], s["y"][t], st, s["ws"],
                              desc=s["descs"][t % n_rep])

    def down(t):
        s = sites["down"]
        spax.spax_masked_gemv_swiglu(s["reps"][t % n_rep], sites["gate_up"]["y"][t], s["prm"],
                                     s["y"][t], st, s["ws"], desc=s["descs"][t % n_rep])

    for ctx in LAYER_CONTEXTS:
        pages = -(-ctx // KV_PAGE)
        n_cache = max(n_rep, math.ceil(3 * L2_BYTES / (ctx * HIDDEN * 4)))  # 4 B: key and value
        caches = []
        for c in range(n_cache):
            kv = spax.alloc_kv_cache(pages, KV_PAGE, HEADS, HEAD_DIM, device=dev)
            for pool in (kv.k, kv.v):
                pool.normal_()
            caches.append(kv)
        aws = spax.alloc_attention_workspace(caches[0], HEADS)
        table = torch.randperm(pages, device=dev).int().view(1, pages)
        pos = torch.full((1,), ctx - 1, dtype=torch.int32, device=dev)
        lens = torch.full((1,), ctx, dtype=torch.int32, device=dev)
        torch.cuda.synchronize()  # the caches, the table and x1, before `stream` reads them

        def between(t):  # qkv's row -> the attention's output
            kv = caches[t % n_cache]
            q, k, v = sites["qkv"]["y"][t].view(1, 3, HEADS, HEAD_DIM).unbind(1)
            spax.spax_kv_append(kv, q, k, v, pos, table, st, rope=rope)
            spax.spax_paged_attention(kv, q, table, lens, att[t], st, aws, scale=HEAD_DIM ** -0.5)

        def layer():
            for t in range(n_tok):
                gemv("qkv", t, x1[t].view(-1))
                between(t)
                gemv("o", t, att[t].view(-1))
                spax.spax_residual_norm(h[t], sites["o"]["y"][t].view(1, -1), r[t], x2[t], pre=norm)
                gemv("gate_up", t, x2[t].view(-1))
                down(t)
                spax.spax_residual_norm(r[t], sites["down"]["y"][t].view(1, -1), r2[t], x3[t], pre=norm)

        def projections():
            for t in range(n_tok):
                gemv("qkv", t, x1[t].view(-1))
                gemv("o", t, att[t].view(-1))
                gemv("gate_up", t, x2[t].view(-1))
                down(t)

        whole = _timed_graph(layer, stream, steps, warmup) * 1000 / n_tok
        alone = _timed_graph(projections, stream, steps, warmup) * 1000 / n_tok
        out[f"context_{ctx}"] = {
            "layer_us_per_token": round(whole, 3), "projections_us_per_token": round(alone, 3),
            "between_us_per_token": round(whole - alone, 3),
            "cache_bytes": ctx * HIDDEN * 4, "caches": n_cache,
            "cache_us_at_8TBps": round(ctx * HIDDEN * 4 / 8e6, 3)}
        if int(st.item()) != 0:
            raise RuntimeError(f"device status {int(st.item())} in the decoder layer")
        del caches
        torch.cuda.empty_cache()
    del sites
    torch.cuda.empty_cache()
    return out


def run_extras(args, dev):
    """Measurements beside the headline, on one GPU, each a CUDA graph timed like the headline."""
    out = {"dequant_vs_load": run_dequant(args, dev)}
    out["guess_under_token_scale"] = run_scaled_guess(args, dev)
    out["llama3_8b_stack"] = run_llama3_stack(args, dev)
    out["llama2_70b_mlp_int4"] = run_llama2_70b_mlp(args, dev)
    out["decode_layer"] = run_decode_layer(args, dev)
    out["host_link_offload"] = run_host_link(args, dev)
    torch.cuda.empty_cache()
    return out


def run_decode_case(args, dev):
    """Profiling aid (no timing, no JSON line): the list-driven GEMV on 22016x4096 with every
    column in the 2-bit tier, lists built beforehand, one L2-resident weight copy, 4 launches
    after one mask launch. Under ncu it isolates the 2-bit decode from HBM and from the
    selection."""
    from tiered_weight_gemv_b200 import spax, synth

    d_out, d_in = 22016, 4096
    W = synth.weight(d_out, d_in, 6, 302, device=dev)
    pm = spax.alloc_packed(d_out, d_in, spax.FULL_BF16, device=dev)
    spax.spax_pack_weights(W, spax.FULL_BF16, pm)
    torch.cuda.synchronize()
    del W
    x = synth.laplace((d_in,), 6, 312, device=dev)
    tier = torch.empty(d_in, dtype=torch.uint8, device=dev)
    fi = torch.empty(d_in, dtype=torch.int32, device=dev)
    ai = torch.empty(d_in, dtype=torch.int32, device=dev)
    cnt = torch.empty(4, dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    y = torch.empty(d_out, device=dev)
    ws = spax.alloc_workspace(spax.OP_TIERED_GEMV, d_out, d_in, device=dev)
    spax.spax_build_mask(x, spax.mask_params(spax.MASK_TOPK, k_full=0, k_approx=d_in), tier, fi, ai,
                         cnt, st)
    for _ in range(4):
        spax.spax_tiered_gemv(pm, x, fi, ai, cnt, y, st, ws)
    torch.cuda.synchronize()
    if int(st.item()) != 0:
        raise RuntimeError(f"device status {int(st.item())}")
    return 0


def run_host_link(args, dev):
    """The pages' own setting: the Llama-2-7B block's packed pools in page-locked host memory, read
    by the same kernels over the host link (zero-copy), masked GEMV against dense. The roofline is
    a measured host-to-device copy of pinned memory; the bytes that must cross the link are the
    selected weights (x, lists and y stay in device memory)."""
    from tiered_weight_gemv_b200 import spax

    n_tok, n_rep = 8, 2
    steps, warmup = max(3, min(args.steps, 5)), args.warmup
    stream = torch.cuda.Stream(device=dev)
    mats = make_weights(dev)
    xs = make_inputs(mats, n_tok, dev)
    sites = {}
    for name, d_out, d_in, _ in SITES:
        pm = spax.alloc_packed(d_out, d_in, spax.FULL_BF16, device=dev)
        spax.spax_pack_weights(mats[name], spax.FULL_BF16, pm)
        torch.cuda.synchronize()
        reps = [spax.packed_to_host(pm) for _ in range(n_rep)]
        del pm
        kf, ka = k_counts(d_in)
        sites[name] = dict(reps=reps, descs=[r.desc() for r in reps], d_out=d_out, d_in=d_in, kf=kf,
                           ka=ka, prm=spax.mask_params(spax.MASK_TOPK, k_full=kf, k_approx=ka),
                           y=torch.empty(n_tok, d_out, device=dev),
                           st=torch.zeros(1, dtype=torch.int32, device=dev),
                           ws=spax.alloc_workspace(spax.OP_TIERED_GEMV, d_out, d_in, device=dev),
                           dws=spax.alloc_workspace(spax.OP_DENSE_GEMV, d_out, d_in, device=dev))
    del mats
    torch.cuda.synchronize()

    def masked():
        for t in range(n_tok):
            for name, *_ in SITES:
                b = sites[name]
                r = t % n_rep
                spax.spax_masked_gemv(b["reps"][r], xs[name][t], b["prm"], b["y"][t], b["st"], b["ws"],
                                      desc=b["descs"][r])

    def dense():
        for t in range(n_tok):
            for name, *_ in SITES:
                b = sites[name]
                spax.spax_dense_gemv(b["reps"][t % n_rep].full, xs[name][t], b["y"][t], b["d_out"],
                                     b["d_in"], b["st"], b["dws"])

    res = {}
    for label, fn in (("masked", masked), ("dense", dense)):
        with torch.cuda.stream(stream):
            fn()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            fn()
        res[label] = time_graph(g, steps, warmup, stream) * 1000 / n_tok  # us per token-layer
        del g
    for name, *_ in SITES:
        if int(sites[name]["st"].item()) != 0:
            raise RuntimeError(f"device status {int(sites[name]['st'].item())} (host pools, {name})")
    # the link's measured rate: one 1 GiB copy of pinned host memory to the device
    src = torch.empty(1 << 30, dtype=torch.uint8, pin_memory=True)
    dst = torch.empty(1 << 30, dtype=torch.uint8, device=dev)
    with torch.cuda.stream(stream):
        for _ in range(2):
            dst.copy_(src, non_blocking=True)
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(stream)
        for _ in range(3):
            dst.copy_(src, non_blocking=True)
        e1.record(stream)
        torch.cuda.synchronize()
    copy_gbps = 3 * (1 << 30) / (e0.elapsed_time(e1) * 1e-3) / 1e9
    link_bytes = sum(spax.spax_weight_bytes(b["d_out"], spax.FULL_BF16, b["kf"], b["ka"])
                     for b in sites.values())
    dense_bytes = sum(2 * b["d_out"] * b["d_in"] for b in sites.values())
    achieved = link_bytes / (res["masked"] * 1e-6) / 1e9
    return {"tokens": n_tok, "replicas_in_host_memory": n_rep,
            "masked_us_per_token_layer": round(res["masked"], 1),
            "dense_us_per_token_layer": round(res["dense"], 1),
            "speedup_vs_dense": round(res["dense"] / res["masked"], 3),
            "selected_bytes_per_token_layer": link_bytes,
            "dense_bytes_per_token_layer": dense_bytes,
            "masked_link_GBps": round(achieved, 1),
            "dense_link_GBps": round(dense_bytes / (res["dense"] * 1e-6) / 1e9, 1),
            "h2d_copy_GBps": round(copy_gbps, 1),
            "masked_frac_of_copy": round(achieved / copy_gbps, 4)}


def fit_c0_bw(points):
    """Least-squares time = c0 + bytes / BW over (bytes, us) points: the fixed per-launch cost and
    the streaming rate (the byte-account method of the ByteCross abstract)."""
    b = np.array([p[0] for p in points], np.float64)
    t = np.array([p[1] for p in points], np.float64)
    A = np.stack([np.ones_like(b), b], 1)
    (c0, inv_bw), *_ = np.linalg.lstsq(A, t, rcond=None)
    pred = A @ np.array([c0, inv_bw])
    ss = float(((t - t.mean()) ** 2).sum())
    r2 = 1.0 - float(((t - pred) ** 2).sum()) / ss if ss > 0 else 1.0
    return {"c0_us": round(float(c0), 3), "GBps": round(1e-3 / inv_bw, 1) if inv_bw > 0 else None,
            "r2": round(r2, 4)}


TRAFFIC_FILE = os.path.join(ROOT, "profiles", "tiered_gemv_traffic.json")
GEMV_SOURCES = ["gemv.cu", "select.cuh", "common.cuh", "internal.h"]


def gemv_source_hash() -> str:
    import hashlib
    h = hashlib.sha256()
    for f in GEMV_SOURCES:
        with open(os.path.join(ROOT, "tiered_weight_gemv_b200", "csrc", f), "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def measured_traffic():
    """Per-site DRAM bytes (read + write) per tiered-GEMV launch from the committed ncu capture,
    or None when the GEMV sources changed since it was taken."""
    try:
        with open(TRAFFIC_FILE) as f:
            t = json.load(f)
    except Exception:
        return None
    return t["sites"] if t.get("source_sha256") == gemv_source_hash() else None


def measured_peak():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        with open(p) as f:
            return float(json.load(f)["hbm_gbs"]), "measured"
    except Exception:
        return FALLBACK_HBM_GBS, "fallback"


# ----------------------------------------------------------------------------- CPU oracle

def host_workload():
    """Host copies of the block and its inputs (generated on the GPU when there is one)."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    mats = make_weights(dev)
    xs = make_inputs(mats, N_TOKENS, dev)
    return {n: m.cpu() for n, m in mats.items()}, {n: v.cpu() for n, v in xs.items()}


class OracleRunner:
    """The oracle as it stands, on host copies of the same block (replica 0)."""

    def __init__(self, mats, xs):
        import oracle
        self.o = oracle
        self.xs = {n: v.numpy() for n, v in xs.items()}
        self.pools = {}
        for name, d_out, d_in, _ in SITES:
            wb = mats[name].view(torch.int16).numpy().view(np.uint16)
            self.pools[name] = oracle.pack(wb, oracle.FULL_BF16)

    def token(self, t):
        o = self.o
        for name, d_out, d_in, _ in SITES:
            kf, ka = k_counts(d_in)
            st, tier, fi, ai, c = o.tiers(self.xs[name][t], o.MODE_TOPK, k_full=kf, k_approx=ka)
            o.tiered_gemv(*self.pools[name], o.FULL_BF16, d_out, d_in, self.xs[name][t], tier)


def cpu_baseline(n_tokens, mats, xs, omp=True):
    r = OracleRunner(mats, xs)
    t0 = time.perf_counter()
    for t in range(n_tokens):
        r.token(t)
    dt = time.perf_counter() - t0
    res = {"value": round(dt * 1e6 / n_tokens, 1), "unit": "us/token/layer", "cores": 1,
           "kind": "oracle",
           "sample": f"{n_tokens} of the {N_TOKENS} tokens, all four sites, single-threaded C "
                     f"oracle (fp64), {dt:.1f} s"}
    if omp:  # the same oracle source built with OpenMP: row chunks over every host core
        threads = r.o.use_openmp(True)
        try:
            t0 = time.perf_counter()
            for t in range(n_tokens):
                r.token(t)
            dto = time.perf_counter() - t0
        finally:
            r.o.use_openmp(False)
        res["openmp"] = {"value": round(dto * 1e6 / n_tokens, 1), "unit": "us/token/layer",
                         "cores": threads, "sample": f"the same {n_tokens} tokens, {dto:.1f} s"}
    return res


def run_reference(args, rank, world):
    if rank != 0:
        return 0
    r = OracleRunner(*host_workload())
    per_step = max(1, args.ref_tokens)
    for w in range(args.warmup):
        r.token(w % N_TOKENS)
    t0 = time.perf_counter()
    for s in range(args.steps):
        for k in range(per_step):
            r.token((s * per_step + k) % N_TOKENS)
    dt = time.perf_counter() - t0
    val = dt * 1e6 / (args.steps * per_step)
    line = {"metric": METRIC, "value": round(val, 1), "unit": "us/token/layer", "n_gpus": world,
            "steps": args.steps, "warmup": args.warmup,
            "ms_per_step": round(dt * 1e3 / args.steps, 3), "higher_is_better": False,
            "scaling": "weak", "vs_baseline": None, "dtype": "f64", "data": "synthetic",
            "impl": "reference",
            "config": workload_config(args.tokens, args.replicas, world),
            "cpu_baseline": {"value": round(val, 1), "unit": "us/token/layer", "cores": 1,
                             "kind": "oracle",
                             "sample": f"{per_step} of the {N_TOKENS} tokens per step (tokens "
                                       f"cycled), all four sites, single-threaded C oracle "
                                       f"(fp64), weight replica 0"},
            "e2e": {"value": round(val, 1), "unit": "us/token/layer", "h2d_bytes_per_step": 0,
                    "d2h_bytes_per_step": 0}}
    print(json.dumps(line), flush=True)
    return 0


# ----------------------------------------------------------------------------- main

def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--impl", choices=["spax", "reference"], default="spax")
    ap.add_argument("--tokens", type=int, default=N_TOKENS)
    ap.add_argument("--replicas", type=int, default=N_REPLICAS)
    ap.add_argument("--cpu-tokens", type=int, default=24)
    ap.add_argument("--ref-tokens", type=int, default=1)
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--decode-case", action="store_true",
                    help="profiling aid: run only the list-driven all-2-bit GEMV on 22016x4096 (one "
                         "mask launch, then 4 GEMV launches on one L2-resident copy); no JSON line")
    ap.add_argument("--host-link-only", action="store_true",
                    help="profiling aid: run only the host-link offload measurement (pools in "
                         "page-locked host memory) and print its JSON; not the benchmark line")
    ap.add_argument("--no-extras", action="store_true",
                    help="skip the measurements beside the headline (dequant vs load, the "
                         "Llama-3-8B sweep and fit, dense and torch.mv)")
    ap.add_argument("--sites", default="", help="comma-separated subset of qkv,o,gate_up,down "
                    "(profiling runs); the default runs the whole block")
    args = ap.parse_args()
    if args.warmup < 3:
        args.warmup = 3
    rank, world, local = dist_setup()
    try:
        if args.impl == "reference":
            return run_reference(args, rank, world)
        if args.decode_case:
            torch.cuda.set_device(local)
            return run_decode_case(args, torch.device("cuda", local)) if rank == 0 else 0
        if args.host_link_only:
            torch.cuda.set_device(local)
            if rank == 0:
                print(json.dumps({"host_link_offload": run_host_link(args, torch.device("cuda", local))}),
                      flush=True)
            return 0
        res, sites, tot_bytes, tot_ms, lps, h2d, d2h, clocks, host = run_gpu(args, rank, world, local)
        ms = res["fused"]
        value = us_per_token_layer(ms, args.tokens, world)
        two_call = us_per_token_layer(res["tiered"], args.tokens, world)
        dense = us_per_token_layer(res["dense"], args.tokens, world)
        e2e = us_per_token_layer(res["e2e"], args.tokens, world)
        peak, peak_kind = measured_peak()
        traffic_sites = measured_traffic()
        traffic = None
        if traffic_sites and all(n in traffic_sites for n in sites):
            traffic = round(sum(traffic_sites[n] for n in sites) / len(sites))
            for n in sites:
                sites[n]["dram_bytes_per_launch"] = traffic_sites[n]
        achieved = tot_bytes / (tot_ms * 1e-3) / 1e9
        step_bytes = sum(s["masked_gemv_bytes_per_launch"] for s in sites.values()) * args.tokens
        dense_bytes = sum(2 * v["d_out"] * v["d_in"] for v in sites.values()) * args.tokens
        line = {
            "metric": METRIC, "value": round(value, 3), "unit": "us/token/layer",
            "n_gpus": world, "steps": args.steps, "warmup": args.warmup,
            "ms_per_step": round(ms, 4), "higher_is_better": False, "scaling": "weak",
            "vs_baseline": None, "dtype": "f32-accumulate (bf16 + 2-bit weights)",
            "data": "synthetic (seeded bf16 N(0,0.02) weights, Laplace(0,1) activations)",
            "config": workload_config(args.tokens, args.replicas, world),
            "effective_GBps": round(step_bytes / (ms * 1e-3) / 1e9, 1),
            "frac_of_8TBps": round(step_bytes / (ms * 1e-3) / 8e12, 4),
            "dense_us_per_token_layer": round(dense, 3),
            "dense_effective_GBps": round(dense_bytes / (res["dense"] * 1e-3) / 1e9, 1),
            "speedup_vs_dense": round(dense / value, 3),
            "two_call_us_per_token_layer": round(two_call, 3),
            "unguessed_us_per_token_layer": round(us_per_token_layer(res["fused_unguessed"], args.tokens, world), 3),
            "unguessed_note": "the headline step without the calibrated guess of the TopK boundary "
                              "keys (same selected columns, found by the full selection)",
            "guess_missed_us_per_token_layer": round(us_per_token_layer(res["fused_missed"], args.tokens, world), 3),
            "guess_missed_note": "the same step with every guess twice the calibrated key, so every "
                                 "launch misses its windows and then runs the full selection (the "
                                 "worst case of a wrong guess)",
            "chained_us_per_token_layer": round(us_per_token_layer(res["chained"], args.tokens, world), 3),
            "chained_note": "down fed from the tiered gate/up output in its own launch "
                            "(spax_masked_gemv_swiglu); informational",
            "sites": sites,
            "fit_time_vs_bytes": {"tiered": fit_c0_bw([(v["masked_gemv_bytes_per_launch"], v["masked_gemv_us"]) for v in sites.values()]),
                                  "dense": fit_c0_bw([(2 * v["d_out"] * v["d_in"], v["dense_us"]) for v in sites.values()])},
            "roofline": {"bound": "hbm", "kernel": "tiered_gemv_kernel (fused mask)",
                         "achieved": round(achieved, 1), "peak": peak, "unit": "GB/s",
                         "frac": round(achieved / peak, 4), "peak_source": peak_kind,
                         "traffic": traffic,
                         "algorithmic_bytes_per_launch": round(tot_bytes / args.tokens / len(sites))},
            "e2e": {"value": round(e2e, 3), "unit": "us/token/layer", "h2d_bytes_per_step": h2d,
                    "d2h_bytes_per_step": d2h,
                    "note": "every step copies its inputs in from pinned host memory and its "
                            "outputs back; two buffer sets and separate copy streams overlap a "
                            "step's copies with its neighbours' compute"},
            "gpu_launches": lps * args.steps,
            "clocks": {k: clocks[k] for k in ("sm_mhz", "sm_max_mhz", "reasons")},
        }
        if world == 1 and not args.no_extras and not args.sites:
            line["extras"] = run_extras(args, torch.device("cuda", local))
        if host is not None:
            line["cpu_baseline"] = cpu_baseline(args.cpu_tokens, *host)
        if rank == 0:
            print(json.dumps(line), flush=True)
        return 0
    finally:
        if dist.is_initialized():
            dist.destroy_process_group()


if __name__ == "__main__":
    sys.exit(main())
