#!/usr/bin/env python3
"""Benchmark of the FP8 W8A8 rollout linear path on GB300.

One step = one pass of the hot path over one Qwen3-8B-shaped decoder layer:
  1. weight sync: the layer's seven bf16 linears quantised to E4M3 with fp32
     128x128 block scales (one batched launch);
  2. rollout forward of the same layer on a batch of M tokens: 1x128 activation
     quantisation of each linear's input, then the four block-scaled GEMMs
     (fused qkv, o_proj, fused gate-up, down);
  3. the MoE expert pair of a Qwen3-30B-A3B-shaped layer (grouped gate-up and
     down GEMMs over replayed top-8 routing of T tokens, activations quantised
     per 1x128 group).
`value` is the step's weight-sync throughput in GB/s (algorithmic bytes of
step 1 over the device time of step 1, summed over ranks), the first part of
the headline metric; the GEMM TFLOPS and every phase's roofline fraction ride
in the same JSON line.  Extra sections, timed in the same run outside the step:
the full-model weight sync (36 layers), the MoE weight sync (48 layers x 128
experts), the GEMM sweep over M in {16, 128, 1024, 8192}, and the UE8M0 variants.

`--impl reference` times the CPU oracle on a bounded sample of the same
workload (the reference arm of this build; there is no other implementation).
"""
from __future__ import annotations

import argparse
import json
import os
import statistics
import subprocess
import threading
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

METRIC = "weight-sync quant GB/s; W8A8 block-scaled GEMM TFLOPS; % of roofline, 1 GB300"
UNIT = "GB/s"
WORKLOAD = "qwen3-8b-layer"
STEP_M = 8192          # tokens in the step's forward batch
NOMINAL_FP8_DENSE_TFLOPS = 4500.0  # GB300 dense FP8 tensor rate as published (context only)

# DRAM bytes (read + write) per launch of the dominant kernel, taken from one
# ncu capture of the same launch (the 8192 x 24576 x 4096 gate-up GEMM).
# Reported only while the GEMM's sources are those the capture was taken with.
TRAFFIC = {
    "gemm_gate_up": {
        "bytes": 151.327488e6 + 372.452096e6,
        "sources": {
            "gemm.cu": "6fd895098b82807637e85bb8c33aefeedb0dfbfe92cfe5310cceb6a471775fcd",
            "ptx.cuh": "7611be7f4488dec541b5332e198986f65689abe958fd940e526f41325f47e1be",
            "common.cuh": "6401f31a7a6a92810a87d55c9eae24512fe80ad094dc69922897bb43c8e0894d",
        },
    },
}


def captured_traffic(kernel: str):
    """The captured DRAM bytes of `kernel`, or None if its sources changed since."""
    import hashlib
    entry = TRAFFIC.get(kernel)
    if entry is None:
        return None
    csrc = os.path.join(os.path.dirname(os.path.abspath(__file__)), "fp8_w8a8_rollout_gb300", "csrc")
    for name, digest in entry["sources"].items():
        try:
            with open(os.path.join(csrc, name), "rb") as f:
                if hashlib.sha256(f.read()).hexdigest() != digest:
                    return None
        except OSError:
            return None
    return entry["bytes"]
MOE_T = 4096           # tokens of the MoE layer (x top-8 = 32768 grouped rows)
L2_BYTES = 129 * 2 ** 20


def parse():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--impl", default="ours", choices=["ours", "reference"])
    ap.add_argument("--sections", default="all",
                    help="comma list of extra sections: model,moe_sync,sweep,ue8m0,fused,kv,moe_layer,tis,decode "
                         "(or all/none)")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-clocks", action="store_true")
    ap.add_argument("--case", default=None,
                    help="time one kernel alone (for profiling): gemm:M:N:K[:fmt], aqg:M:N:K[:fmt], grouped:gate_up|down[:fmt], "
                         "wq:layer[:fmt], aq:M:K[:fmt], fused:M[:fmt], fused_moe[:fmt], kv:TOKENS, "
                         "kvcal:TOKENS, moe_plan, moe_dispatch, moe_combine, tis[:RESPONSES], op:NAME (a case of "
                         "perf/operators.py, through the binding's helpers)")
    ap.add_argument("--bn", type=int, default=0, help="with --case: force the GEMM tile width (128 or 256)")
    ap.add_argument("--wait-mode", type=int, default=0, help="with --case: GEMM wait style (test hook 4)")
    ap.add_argument("--l2-prefetch", type=int, default=-1, help="with --case: GEMM L2 prefetch distance (test hook 5)")
    ap.add_argument("--graph", action="store_true", help="with --case: also time replays of a CUDA graph")
    ap.add_argument("--streamk", type=int, default=-1,
                    help="with --case gemm: call the workspace entry point; 0 chooses, 1 never, 2 always stream-K")
    ap.add_argument("--streamk-grid", type=int, default=0, help="with --streamk: stream-K CTA count (0: one per SM)")
    ap.add_argument("--out-stage", type=int, default=0,
                    help="with --case: tile stores, 0 chosen, 1 through shared memory + TMA, 2 from registers")
    ap.add_argument("--pair", type=int, default=0,
                    help="with --case: dense tiles on tensor-core pairs, 0 chosen, 1 always, 2 never")
    ap.add_argument("--mx", type=int, default=0,
                    help="with --case: UE8M0 whole tiles, 0 chosen by K, 1 per-chunk promotion, 2 block-scaled MMA")
    ap.add_argument("--no-overlap", action="store_true",
                    help="with --case: launch the activation quantiser and decode GEMM without overlap")
    return ap.parse_args()


# --------------------------------------------------------------------------- algorithmic work

def wq_bytes(n, k, scale_bytes=4):
    """Weight-sync bytes: bf16 in, E4M3 out, one scale per 128x128 block."""
    return 3 * n * k + scale_bytes * ((n + 127) // 128) * ((k + 127) // 128)


def aq_bytes(m, k, scale_bytes=4):
    return 3 * m * k + scale_bytes * m * ((k + 127) // 128)


def gemm_flops(m, n, k):
    return 2 * m * n * k


def gemm_bytes(m, n, k, scale_bytes=4):
    return n * k + m * k + 2 * m * n + scale_bytes * (m * (k // 128) + (n // 128) * (k // 128))


def grouped_gemm_bytes(experts, rows, n, k, scale_bytes=4):
    """Every expert's weights once, the routed rows' codes in, bf16 out, scales."""
    return (experts * n * k + rows * k + 2 * rows * n +
            scale_bytes * (rows * (k // 128) + experts * (n // 128) * (k // 128)))


def fp8_peak(peaks):
    """Dense FP8 tensor roofline: 2 x the measured BURST bf16 GEMM rate (the
    nominal fp8:bf16 ratio).  The burst figure is the one for kernels timed
    in isolation or inside a step of a few milliseconds, as every GEMM here
    is; the sustained figure (a seconds-long loop under the power cap) is
    reported beside it only as a second, labelled fraction."""
    return 2.0 * peaks["bf16_tflops"]


FP8_PEAK_BASIS = "2 x bf16_tflops (burst), the nominal fp8:bf16 ratio"


def load_peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        d = json.load(open(p))
        peaks = {"hbm_gbs": d["hbm_gbs"], "bf16_tflops": d["bf16_tflops"],
                 "bf16_tflops_sustained": d.get("bf16_tflops_sustained", d["bf16_tflops"]),
                 "source": "measured"}
    else:
        peaks = {"hbm_gbs": 6800.0, "bf16_tflops": 1900.0, "bf16_tflops_sustained": 1700.0,
                 "source": "fallback"}
    peaks["fp8_tflops"] = fp8_peak(peaks)
    peaks["fp8_basis"] = FP8_PEAK_BASIS
    return peaks


# --------------------------------------------------------------------------- clocks

class ClockSampler:
    """nvidia-smi clock and throttle samples around the timed region: the
    sampler runs before the region starts (the first sample has arrived), a
    reader thread stamps each sample with the host clock, and the summary
    keeps the samples taken between mark_start() and mark_end()."""
    FIELDS = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")
    INTERVAL_MS = 20

    def __init__(self, index: str, enabled: bool = True, command=None):
        self.index = index
        self.proc = None
        self.enabled = enabled
        self.command = command  # a stand-in for nvidia-smi (tests)
        self.samples = []       # (host time, csv line)
        self.t0 = self.t1 = None
        self.thread = None

    def _read(self):
        for ln in self.proc.stdout:
            if ln.strip():
                self.samples.append((time.monotonic(), ln.strip()))

    def __enter__(self):
        if self.enabled:
            cmd = self.command or ["nvidia-smi", f"--id={self.index}", f"--query-gpu={self.FIELDS}",
                                   "--format=csv,noheader,nounits", "-lms", str(self.INTERVAL_MS)]
            try:
                self.proc = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
            except OSError:
                self.proc = None
            if self.proc is not None:
                self.thread = threading.Thread(target=self._read, daemon=True)
                self.thread.start()
                deadline = time.monotonic() + 5.0
                while not self.samples and time.monotonic() < deadline and self.proc.poll() is None:
                    time.sleep(0.005)
        return self

    def mark_start(self):
        self.t0 = time.monotonic()

    def mark_end(self):
        self.t1 = time.monotonic()
        # a region shorter than the sampling interval still gets the sample
        # that was being taken while it ran
        if self.proc is not None:
            time.sleep(self.INTERVAL_MS / 1000.0 * 1.5)

    def __exit__(self, *exc):
        if self.proc is not None:
            self.proc.terminate()
            try:
                self.proc.wait(timeout=5)
            except subprocess.TimeoutExpired:
                self.proc.kill()
                self.proc.wait()
        if self.thread is not None:
            self.thread.join(timeout=5)

    def window(self):
        """The samples stamped inside the region (a sample's line is printed
        up to one interval after it was taken, so the window ends one
        interval late)."""
        if self.t0 is None or self.t1 is None:
            return [ln for _, ln in self.samples]
        late = self.INTERVAL_MS / 1000.0
        return [ln for t, ln in self.samples if self.t0 <= t <= self.t1 + late]

    def summary(self):
        lines = self.window()
        sm, mx, reasons = [], 0.0, set()
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for ln in lines:
            parts = [p.strip() for p in ln.split(",")]
            if len(parts) < 9:
                continue
            try:
                sm.append(float(parts[1]))
                mx = max(mx, float(parts[2]))
            except ValueError:
                continue
            for name, val in zip(names, parts[5:9]):
                if val.lower().startswith("active"):
                    reasons.add(name)
        if not sm:
            return None
        return {"sm_mhz": statistics.median(sm), "sm_max_mhz": mx, "reasons": sorted(reasons),
                "samples": len(sm), "interval_ms": self.INTERVAL_MS}


def gpu_smi_id(torch, local: int) -> str:
    """nvidia-smi --id of this process's GPU (its UUID, so that a remapped
    CUDA_VISIBLE_DEVICES still names the right physical device)."""
    try:
        u = str(torch.cuda.get_device_properties(local).uuid)
        return u if u.startswith("GPU-") else "GPU-" + u
    except Exception:
        vis = os.environ.get("CUDA_VISIBLE_DEVICES", "")
        ids = [v for v in vis.split(",") if v.strip()]
        return ids[local] if local < len(ids) else str(local)


# --------------------------------------------------------------------------- our arm

class Timer:
    """Per-phase CUDA-event timing on the launching stream."""

    def __init__(self, torch, stream):
        self.torch = torch
        self.stream = stream
        self.pending = []
        self.totals = {}
        self.counts = {}

    def phase(self, name):
        timer = self

        class _P:
            def __enter__(self_inner):
                self_inner.a = timer.torch.cuda.Event(enable_timing=True)
                self_inner.b = timer.torch.cuda.Event(enable_timing=True)
                self_inner.a.record(timer.stream)

            def __exit__(self_inner, *exc):
                self_inner.b.record(timer.stream)
                timer.pending.append((name, self_inner.a, self_inner.b))
        return _P()

    def collect(self):
        self.torch.cuda.synchronize()
        for name, a, b in self.pending:
            self.totals[name] = self.totals.get(name, 0.0) + a.elapsed_time(b)
            self.counts[name] = self.counts.get(name, 0) + 1
        self.pending = []

    def avg_ms(self, name):
        return self.totals[name] / self.counts[name]


def gemm_available(fp8rl, torch):
    """True once the library's GEMM entry points run (not FP8RL_ERR_UNSUPPORTED)."""
    dev = torch.device("cuda")
    xq = torch.zeros((1, 128), dtype=torch.uint8, device=dev)
    sx = torch.ones((1, 1), dtype=torch.float32, device=dev)
    wq = torch.zeros((128, 128), dtype=torch.uint8, device=dev)
    sw = torch.ones((1, 1), dtype=torch.float32, device=dev)
    try:
        fp8rl.gemm(xq, sx, wq, sw)
        torch.cuda.synchronize()
        return True
    except fp8rl.Fp8rlError as e:
        if e.status == 4:
            return False
        raise


def build_step_inputs(torch, synth, fp8rl, dev, seed, have_gemm):
    """Everything the step reads, resident in HBM before timing starts."""
    layer = synth.qwen3_8b_layer(0, seed, device=dev)
    weights = [w for _, w in layer]
    wout = [(torch.empty(w.shape, dtype=torch.uint8, device=dev),
             torch.empty(((w.shape[0] + 127) // 128, (w.shape[1] + 127) // 128),
                         dtype=torch.float32, device=dev)) for w in weights]
    descs = fp8rl.weight_descs([(w, q, s) for w, (q, s) in zip(weights, wout)])
    inp = {"weights": weights, "wout": wout, "descs": descs, "gemms": [], "moe": None}
    if not have_gemm:
        return inp
    # fused forward weights, pre-quantised once (the step re-quantises the
    # per-matrix weights above; the GEMMs read these fused copies)
    for name, n, k in synth.QWEN3_8B_GEMMS:
        w = synth.weight_bf16(n, k, seed, "step-fused", name, device=dev)
        wq, sw = fp8rl.quant_weight(w)
        del w
        x = synth.activation_bf16(STEP_M, k, seed, "step-x", name, device=dev)
        xq = torch.empty((STEP_M, k), dtype=torch.uint8, device=dev)
        sx = torch.empty((k // 128, STEP_M), dtype=torch.float32, device=dev)
        y = torch.empty((STEP_M, n), dtype=torch.bfloat16, device=dev)
        inp["gemms"].append((name, n, k, x, xq, sx, wq, sw, y))
    # MoE expert pair, one layer
    _, offsets, _, _, rows = moe_plan_for(torch, synth, fp8rl, dev, seed)
    moe = {"offsets": offsets, "rows": rows, "pairs": []}
    for which, n, k in (("gate_up", 2 * synth.MOE_INTER, synth.MOE_HIDDEN),
                        ("down", synth.MOE_HIDDEN, synth.MOE_INTER)):
        wb = synth.moe_expert_weights(n, k, synth.MOE_EXPERTS, seed, 0, which, device=dev)
        wq, sw = fp8rl.quant_weight(wb.view(-1, k))
        del wb
        wq = wq.view(synth.MOE_EXPERTS, n, k)
        sw = sw.view(synth.MOE_EXPERTS, n // 128, k // 128)
        x = synth.normal_bf16((rows, k), 1.0, seed, "moe-x", which, device=dev)
        xq = torch.empty((rows, k), dtype=torch.uint8, device=dev)
        sx = torch.empty((k // 128, rows), dtype=torch.float32, device=dev)
        y = torch.empty((rows, n), dtype=torch.bfloat16, device=dev)
        moe["pairs"].append((which, n, k, x, xq, sx, wq, sw, y))
    inp["moe"] = moe
    return inp


def run_step(fp8rl, inp, timer, stream):
    """One pass of the hot path; returns the number of kernel launches."""
    launches = 0
    with timer.phase("weight_sync"):
        fp8rl.fp8rl_quant_weight_blockwise_batched(inp["descs"], len(inp["weights"]), 0, stream)
    launches += 1
    for name, n, k, x, xq, sx, wq, sw, y in inp["gemms"]:
        with timer.phase(f"act_quant_{name}"):
            fp8rl.fp8rl_quant_act_group(x, STEP_M, k, k, xq, k, sx, 0, stream)
        with timer.phase(f"gemm_{name}"):
            fp8rl.fp8rl_gemm_blockscaled(xq, sx, wq, sw, y, STEP_M, n, k, 0, stream)
        launches += 2
    if inp["moe"] is not None:
        moe = inp["moe"]
        for which, n, k, x, xq, sx, wq, sw, y in moe["pairs"]:
            with timer.phase(f"moe_act_quant_{which}"):
                fp8rl.fp8rl_quant_act_group(x, moe["rows"], k, k, xq, k, sx, 0, stream)
            with timer.phase(f"moe_gemm_{which}"):
                fp8rl.fp8rl_grouped_gemm_blockscaled(xq, sx, wq, sw, moe["offsets"], wq.shape[0],
                                                     moe["rows"], n, k, y, 0, stream)
            launches += 2
    return launches


def step_rooflines(inp, timer, peaks):
    """Per-phase achieved rate against its bound (HBM for quantisers and
    weight-streaming GEMMs, FP8 tensor peak for the others)."""
    hbm = peaks["hbm_gbs"]
    fp8 = fp8_peak(peaks)
    out = {}
    wbytes = sum(wq_bytes(*w.shape) for w in inp["weights"])
    ms = timer.avg_ms("weight_sync")
    out["weight_sync"] = {"bound": "hbm", "ms": ms, "achieved": wbytes / ms / 1e6, "peak": hbm,
                          "unit": "GB/s", "frac": wbytes / ms / 1e6 / hbm, "bytes": wbytes}
    for name, n, k, *_ in inp["gemms"]:
        ms = timer.avg_ms(f"act_quant_{name}")
        b = aq_bytes(STEP_M, k)
        out[f"act_quant_{name}"] = {"bound": "hbm", "ms": ms, "achieved": b / ms / 1e6, "peak": hbm,
                                    "unit": "GB/s", "frac": b / ms / 1e6 / hbm, "bytes": b}
        ms = timer.avg_ms(f"gemm_{name}")
        f = gemm_flops(STEP_M, n, k)
        out[f"gemm_{name}"] = gemm_roof(f, gemm_bytes(STEP_M, n, k), ms, hbm, fp8)
    if inp["moe"] is not None:
        rows = inp["moe"]["rows"]
        for which, n, k, x, xq, sx, wq, sw, y in inp["moe"]["pairs"]:
            ms = timer.avg_ms(f"moe_act_quant_{which}")
            b = aq_bytes(rows, k)
            out[f"moe_act_quant_{which}"] = {"bound": "hbm", "ms": ms, "achieved": b / ms / 1e6,
                                             "peak": hbm, "unit": "GB/s",
                                             "frac": b / ms / 1e6 / hbm, "bytes": b}
            ms = timer.avg_ms(f"moe_gemm_{which}")
            e = wq.shape[0]
            bytes_ = grouped_gemm_bytes(e, rows, n, k)
            out[f"moe_gemm_{which}"] = gemm_roof(gemm_flops(rows, n, k), bytes_, ms, hbm, fp8)
    return out


def gemm_roof(flops, bytes_, ms, hbm_gbs, fp8_tflops):
    """The lower of the two roofs decides the bound."""
    t_tensor = flops / (fp8_tflops * 1e12)
    t_hbm = bytes_ / (hbm_gbs * 1e9)
    if t_hbm > t_tensor:
        return {"bound": "hbm", "ms": ms, "achieved": bytes_ / ms / 1e6, "peak": hbm_gbs,
                "unit": "GB/s", "frac": bytes_ / ms / 1e6 / hbm_gbs, "bytes": bytes_,
                "tflops": flops / ms / 1e9}
    return {"bound": "tensor", "ms": ms, "achieved": flops / ms / 1e9, "peak": fp8_tflops,
            "unit": "TFLOP/s", "frac": flops / ms / 1e9 / fp8_tflops, "flops": flops,
            "tflops": flops / ms / 1e9}


def e2e_weight_sync(torch, fp8rl, inp, stream, steps):
    """Weight sync through the library's C ABI from pinned HOST buffers to
    pinned HOST buffers, every byte crossing the CPU-GPU link inside the timed
    region.  Two ways are timed and the faster is reported:
    fp8rl_quant_weight_host_batched (the library's copy-in / quantise /
    copy-out pipeline over ~32 MB chunks on three streams; "pipelined"), and
    fp8rl_quant_weight_blockwise_batched given host pointers (the quantiser
    reading and writing host memory directly, one launch; "direct")."""
    host_w = [w.cpu().pin_memory() for w in inp["weights"]]
    wbytes = sum(wq_bytes(*w.shape) for w in inp["weights"])
    results = {}
    for mode in ("direct", "pipelined"):
        host_q = [torch.empty(q.shape, dtype=q.dtype, pin_memory=True) for q, _ in inp["wout"]]
        host_s = [torch.empty(s.shape, dtype=s.dtype, pin_memory=True) for _, s in inp["wout"]]
        hs = fp8rl.HostWeightSync(host_w, host_q, host_s, direct=(mode == "direct"))
        for _ in range(2):
            hs.run()
        torch.cuda.synchronize()
        a = torch.cuda.Event(enable_timing=True)
        b = torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(steps):
            hs.run()
        b.record()
        torch.cuda.synchronize()
        ms = a.elapsed_time(b) / steps
        ok = all(torch.equal(hq, dq.cpu()) for hq, (dq, _) in zip(host_q, inp["wout"]))
        results[mode] = {"value": wbytes / ms / 1e6, "ms_per_step": ms, "matches_device_result": ok,
                         "h2d_bytes_per_step": hs.h2d_bytes, "d2h_bytes_per_step": hs.d2h_bytes}
    best = max(results, key=lambda m: results[m]["value"] if results[m]["matches_device_result"] else -1)
    r = results[best]
    return {"value": r["value"], "unit": UNIT, "ms_per_step": r["ms_per_step"],
            "h2d_bytes_per_step": r["h2d_bytes_per_step"], "d2h_bytes_per_step": r["d2h_bytes_per_step"],
            "mode": best, "modes": {m: round(v["value"], 1) for m, v in results.items()},
            "entry_point": {"pipelined": "fp8rl_quant_weight_host_batched",
                            "direct": "fp8rl_quant_weight_blockwise_batched"}[best],
            "matches_device_result": r["matches_device_result"]}


def l2_flusher(torch, dev, mb=512):
    """A call that reads a buffer 4x the L2 (129 MB), so that the next timed
    call starts with none of its inputs in L2.  A read leaves clean lines: a
    flush by writing would leave 129 MB of dirty lines whose write-back the
    timed kernel would pay for."""
    buf = torch.ones(mb << 18, dtype=torch.float32, device=dev)
    return lambda: buf.sum()


def moe_plan_for(torch, synth, fp8rl, dev, seed, tokens=None):
    """The replayed top-8 routing of the Qwen3-30B-A3B-shaped layer and its
    dispatch plan, made by the library's plan kernels: (routing, offsets,
    row_of_pair, token_of_row, routed rows)."""
    r = synth.moe_routing(tokens or MOE_T, synth.MOE_EXPERTS, synth.MOE_TOPK, seed, 0)
    off, rop, tor = fp8rl.moe_plan(torch.from_numpy(r.topk).to(dev), synth.MOE_EXPERTS)
    return r, off, rop, tor, int(off[-1].item())


def time_loop(torch, fn, iters, warmup, flush=None):
    """Per-call device time of fn (CUDA events around `iters` back-to-back calls;
    with a flush, the median of single calls each preceded by an L2 flush)."""
    for _ in range(warmup):
        fn()
    torch.cuda.synchronize()
    if flush is None:
        a = torch.cuda.Event(enable_timing=True)
        b = torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(iters):
            fn()
        b.record()
        b.synchronize()
        return a.elapsed_time(b) / iters
    times = []
    for _ in range(iters):
        flush()
        a = torch.cuda.Event(enable_timing=True)
        b = torch.cuda.Event(enable_timing=True)
        a.record()
        fn()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return statistics.median(times)


def time_graph(torch, fn, reps, warmup=3):
    """Per-call device time of fn replayed from a CUDA graph (captures `reps`
    calls once; times graph replays), so host call overhead does not show."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(warmup):
            fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(reps):
            fn()
    g.replay()
    torch.cuda.synchronize()
    a = torch.cuda.Event(enable_timing=True)
    b = torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(3):
        g.replay()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / (3 * reps)


def section_model_sync(torch, synth, fp8rl, dev, seed, peaks, fmt=0):
    """Full-model weight sync: 36 layers x 7 linears (~6.95e9 params) in one pass."""
    weights = []
    for layer in range(synth.QWEN3_8B_LAYERS):
        weights += [w for _, w in synth.qwen3_8b_layer(layer, seed, device=dev)]
    sb = 4 if fmt == 0 else 1
    outs = [(torch.empty(w.shape, dtype=torch.uint8, device=dev),
             torch.empty(((w.shape[0] + 127) // 128, (w.shape[1] + 127) // 128),
                         dtype=torch.float32 if fmt == 0 else torch.uint8, device=dev))
            for w in weights]
    descs = fp8rl.weight_descs([(w, q, s) for w, (q, s) in zip(weights, outs)])
    ms = time_loop(torch, lambda: fp8rl.fp8rl_quant_weight_blockwise_batched(descs, len(weights), fmt),
                   5, 2)
    b = sum(wq_bytes(*w.shape, sb) for w in weights)
    res = {"matrices": len(weights), "params": sum(w.numel() for w in weights), "ms": ms,
           "gbs": b / ms / 1e6, "frac_hbm": b / ms / 1e6 / peaks["hbm_gbs"],
           "launches": (len(weights) + 255) // 256}
    del weights, outs
    torch.cuda.empty_cache()
    return res


def section_moe_sync(torch, synth, fp8rl, dev, seed, peaks, fmt=0):
    """Weight sync of all MoE experts: 48 layers x 128 experts x (gate-up, down)."""
    weights = []
    for layer in range(synth.MOE_LAYERS):
        for which, n, k in (("gate_up", 2 * synth.MOE_INTER, synth.MOE_HIDDEN),
                            ("down", synth.MOE_HIDDEN, synth.MOE_INTER)):
            w = synth.normal_bf16((synth.MOE_EXPERTS * n, k), synth.WEIGHT_STD, seed, "moe-sync",
                                  layer, which, device=dev)
            weights.append(w)
    outs = [(torch.empty(w.shape, dtype=torch.uint8, device=dev),
             torch.empty(((w.shape[0] + 127) // 128, (w.shape[1] + 127) // 128),
                         dtype=torch.float32 if fmt == 0 else torch.uint8, device=dev))
            for w in weights]
    descs = fp8rl.weight_descs([(w, q, s) for w, (q, s) in zip(weights, outs)])
    ms = time_loop(torch, lambda: fp8rl.fp8rl_quant_weight_blockwise_batched(descs, len(weights), fmt),
                   3, 1)
    sb = 4 if fmt == 0 else 1
    b = sum(wq_bytes(*w.shape, sb) for w in weights)
    res = {"params": sum(w.numel() for w in weights), "ms": ms, "gbs": b / ms / 1e6,
           "frac_hbm": b / ms / 1e6 / peaks["hbm_gbs"]}
    del weights, outs
    torch.cuda.empty_cache()
    return res


def section_sweep(torch, synth, fp8rl, dev, seed, peaks, fmt=0):
    """GEMM sweep at Qwen3-8B shapes; small working sets rotate copies > 4x L2."""
    fp8 = fp8_peak(peaks)
    res = {}
    sdt = torch.float32 if fmt == 0 else torch.uint8
    for name, n, k in synth.QWEN3_8B_GEMMS:
        w = synth.weight_bf16(n, k, seed, "sweep", name, device=dev)
        wq, sw = fp8rl.quant_weight(w, fmt)
        del w
        for m in synth.GEMM_SWEEP_M:
            x = synth.activation_bf16(m, k, seed, "sweep-x", name, m, device=dev)
            xq, sx = fp8rl.quant_act(x, fmt)
            ws = n * k + m * k + 2 * m * n
            copies = max(1, min(16, (4 * L2_BYTES) // ws + 1))
            sets = [(xq, sx, wq, sw, torch.empty((m, n), dtype=torch.bfloat16, device=dev))]
            for _ in range(copies - 1):
                sets.append((xq.clone(), sx.clone(), wq.clone(), sw.clone(),
                             torch.empty((m, n), dtype=torch.bfloat16, device=dev)))
            it = [0]

            def call():
                a = sets[it[0] % len(sets)]
                it[0] += 1
                fp8rl.fp8rl_gemm_blockscaled(a[0], a[1], a[2], a[3], a[4], m, n, k, fmt)
            # replayed from a CUDA graph: device time of back-to-back launches
            ms = time_graph(torch, call, max(20, len(sets) * 2))
            r = gemm_roof(gemm_flops(m, n, k), gemm_bytes(m, n, k, 4 if fmt == 0 else 1), ms,
                          peaks["hbm_gbs"], fp8)
            res[f"{name}_m{m}"] = {"m": m, "n": n, "k": k, "ms": ms, "tflops": r["tflops"],
                                   "bound": r["bound"], "frac": r["frac"]}
            del sets
        del wq, sw
    torch.cuda.empty_cache()
    return res


def section_ue8m0(torch, synth, fp8rl, dev, seed, peaks, have_gemm):
    """UE8M0 (power-of-two) scale variants: layer weight sync and the gate-up GEMM."""
    layer = [w for _, w in synth.qwen3_8b_layer(0, seed, device=dev)]
    outs = [(torch.empty(w.shape, dtype=torch.uint8, device=dev),
             torch.empty(((w.shape[0] + 127) // 128, (w.shape[1] + 127) // 128), dtype=torch.uint8,
                         device=dev)) for w in layer]
    descs = fp8rl.weight_descs([(w, q, s) for w, (q, s) in zip(layer, outs)])
    ms = time_loop(torch, lambda: fp8rl.fp8rl_quant_weight_blockwise_batched(descs, len(layer), 1), 20, 5)
    b = sum(wq_bytes(*w.shape, 1) for w in layer)
    res = {"weight_sync_layer": {"ms": ms, "gbs": b / ms / 1e6, "frac_hbm": b / ms / 1e6 / peaks["hbm_gbs"]}}
    if have_gemm:
        res["gemm"] = section_sweep_one(torch, synth, fp8rl, dev, seed, peaks, "gate_up", 24576, 4096,
                                        STEP_M, 1)
        # the MoE expert pair (T = 4096, top-8) with UE8M0 scales, against the
        # same pair with fp32 scales
        _, offsets, _, _, rows = moe_plan_for(torch, synth, fp8rl, dev, seed)
        for which in ("gate_up", "down"):
            n, k = (2 * synth.MOE_INTER, synth.MOE_HIDDEN) if which == "gate_up" else (synth.MOE_HIDDEN, synth.MOE_INTER)
            wb = synth.moe_expert_weights(n, k, synth.MOE_EXPERTS, seed, 0, which, device=dev)
            x = synth.normal_bf16((rows, k), 1.0, seed, "ue8m0-moe-x", which, device=dev)
            y = torch.empty((rows, n), dtype=torch.bfloat16, device=dev)
            entry = {"rows": rows, "n": n, "k": k}
            for fmt, label in ((1, "ue8m0"), (0, "fp32")):
                wq, sw = fp8rl.quant_weight(wb.view(-1, k), fmt)
                xq, sx = fp8rl.quant_act(x, fmt)
                fn = lambda: fp8rl.fp8rl_grouped_gemm_blockscaled(xq, sx, wq, sw, offsets, synth.MOE_EXPERTS, rows,
                                                                  n, k, y, fmt)
                ms = time_loop(torch, fn, 20, 5)
                sb = 4 if fmt == 0 else 1
                b = synth.MOE_EXPERTS * (n * k + sb * (n // 128) * (k // 128)) + rows * k + 2 * rows * n + \
                    sb * rows * (k // 128)
                entry[label] = {"ms": ms, "gbs": b / ms / 1e6, "frac_hbm": b / ms / 1e6 / peaks["hbm_gbs"],
                                "tflops": gemm_flops(rows, n, k) / ms / 1e9}
                del wq, sw, xq, sx
            res[f"moe_{which}_t{MOE_T}"] = entry
            del wb, x, y
    return res


def fused_mlp_inputs(torch, synth, fp8rl, dev, seed, m, fmt, moe=False):
    """Gate/up weights quantised straight into the interleaved layout, and the
    quantised activations, for the dense Qwen3-8B MLP or the Qwen3-30B-A3B
    experts (T = 4096, top-8)."""
    if moe:
        inter, k, e = synth.MOE_INTER, synth.MOE_HIDDEN, synth.MOE_EXPERTS
        gate = synth.moe_expert_weights(inter, k, e, seed, 0, "gate", device=dev)
        up = synth.moe_expert_weights(inter, k, e, seed, 0, "up", device=dev)
        _, offsets, _, _, m = moe_plan_for(torch, synth, fp8rl, dev, seed)
        x = synth.normal_bf16((m, k), 1.0, seed, "fused-moe-x", device=dev)
    else:
        inter, k = 12288, 4096
        gate = synth.weight_bf16(inter, k, seed, "fused-gate", device=dev)
        up = synth.weight_bf16(inter, k, seed, "fused-up", device=dev)
        offsets = None
        x = synth.activation_bf16(m, k, seed, "fused-x", device=dev)
    wq, sw = fp8rl.quant_gate_up_interleaved(gate, up, fmt)
    del gate, up
    xq, sx = fp8rl.quant_act(x, fmt)
    return {"m": m, "inter": inter, "k": k, "wq": wq, "sw": sw, "xq": xq, "sx": sx, "offsets": offsets,
            "experts": synth.MOE_EXPERTS if moe else 1}


def section_fused_mlp(torch, synth, fp8rl, dev, seed, peaks, fmt=0):
    """The fused gate-up path (GEMM + SiLU(gate) * up + 1x128 quantisation in
    one kernel) against the two kernels it replaces: the gate-up GEMM to bf16
    and the activation quantiser on the [m, inter] intermediate (the separate
    SwiGLU pass of an unfused path is not even counted)."""
    res = {}
    for name, moe, m in (("qwen3_8b_mlp_m8192", False, STEP_M), ("qwen3_30b_a3b_experts_t4096", True, 0)):
        d = fused_mlp_inputs(torch, synth, fp8rl, dev, seed, m, fmt, moe)
        m, inter, k = d["m"], d["inter"], d["k"]
        hq = torch.empty((m, inter), dtype=torch.uint8, device=dev)
        hs = torch.empty((inter // 128, m), dtype=torch.float32 if fmt == 0 else torch.uint8, device=dev)
        y = torch.empty((m, 2 * inter), dtype=torch.bfloat16, device=dev)
        q2 = torch.empty((m, inter), dtype=torch.uint8, device=dev)
        if moe:
            fused = lambda: fp8rl.fp8rl_grouped_gemm_swiglu_quant(d["xq"], d["sx"], d["wq"], d["sw"], d["offsets"],
                                                                 d["experts"], m, inter, k, hq, hs, fmt)
            gemm = lambda: fp8rl.fp8rl_grouped_gemm_blockscaled(d["xq"], d["sx"], d["wq"], d["sw"], d["offsets"],
                                                               d["experts"], m, 2 * inter, k, y, fmt)
        else:
            fused = lambda: fp8rl.fp8rl_gemm_swiglu_quant(d["xq"], d["sx"], d["wq"], d["sw"], m, inter, k, hq, hs,
                                                         fmt)
            gemm = lambda: fp8rl.fp8rl_gemm_blockscaled(d["xq"], d["sx"], d["wq"], d["sw"], y, m, 2 * inter, k,
                                                       fmt)
        aq = lambda: fp8rl.fp8rl_quant_act_group(y, m, inter, 2 * inter, q2, inter, hs, fmt)
        t_fused = time_loop(torch, fused, 20, 5)
        t_gemm = time_loop(torch, gemm, 20, 5)
        t_aq = time_loop(torch, aq, 20, 5)
        flops = 2.0 * m * 2 * inter * k
        res[name] = {"m": m, "inter": inter, "k": k, "fused_ms": t_fused, "unfused_gemm_ms": t_gemm,
                     "unfused_act_quant_ms": t_aq, "saved_ms": t_gemm + t_aq - t_fused,
                     "fused_tflops": flops / t_fused / 1e9,
                     "fused_frac_fp8": flops / t_fused / 1e9 / fp8_peak(peaks)}
        del d, hq, hs, y, q2
        torch.cuda.empty_cache()
    return res


KV_DIM, Q_DIM = 1024, 4096  # Qwen3-8B: 8 KV heads and 32 query heads of 128


def kv_inputs(torch, synth, dev, seed, tokens, slots_total):
    k = synth.normal_bf16((tokens, KV_DIM), 1.0, seed, "bench-kv-k", device=dev)
    v = synth.normal_bf16((tokens, KV_DIM), 1.0, seed, "bench-kv-v", device=dev)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    slots = torch.randperm(slots_total, generator=gen, device=dev)[:tokens].to(torch.int32)
    kc = torch.empty((slots_total, KV_DIM), dtype=torch.uint8, device=dev)
    vc = torch.empty((slots_total, KV_DIM), dtype=torch.uint8, device=dev)
    return k, v, slots, kc, vc


def section_kv_cache(torch, synth, fp8rl, dev, seed, peaks):
    """FP8 KV cache of one Qwen3-8B layer: the per-step scale calibration over
    a prefill (K, V and Q of 8192 tokens), a prefill-size append (32768
    tokens into a 65536-slot cache) and a decode-size append (256 tokens)."""
    res = {}
    k, v, _, _, _ = kv_inputs(torch, synth, dev, seed, STEP_M, STEP_M)
    q = synth.normal_bf16((STEP_M, Q_DIM), 1.0, seed, "bench-kv-q", device=dev)
    scales = torch.zeros(3, dtype=torch.float32, device=dev)
    # 100 MB fits in L2, and back-to-back calls would time the host's issue
    # rate: single calls, each after an L2 flush that the host's enqueueing
    # overlaps
    t = time_loop(torch, lambda: fp8rl.kv_calibrate(k, v, q, out=scales), 20, 5, l2_flusher(torch, dev))
    b = STEP_M * (2 * KV_DIM + Q_DIM) * 2
    res["calibrate_prefill_8192"] = {"ms": t, "gbs": b / t / 1e6, "frac_hbm": b / t / 1e6 / peaks["hbm_gbs"],
                                     "l2": "flushed before each call"}
    for name, tokens in (("append_prefill_32768", 32768), ("append_decode_256", 256)):
        k, v, slots, kc, vc = kv_inputs(torch, synth, dev, seed, tokens, 65536)
        fn = lambda: fp8rl.kv_append(k, v, slots, kc, vc, scales)
        t = time_loop(torch, fn, 20, 5)
        b = tokens * KV_DIM * 2 * 3 + tokens * 4  # bf16 in, E4M3 out, K and V; slot indices
        entry = {"ms": t, "gbs": b / t / 1e6, "frac_hbm": b / t / 1e6 / peaks["hbm_gbs"]}
        if tokens < 1024:
            entry["ms_graph"] = time_graph(torch, fn, 50)
        res[name] = entry
    return res


def moe_layer_inputs(torch, synth, fp8rl, dev, seed):
    """Replayed routing of T = 4096 tokens (top-8 of 128 experts), the plan
    buffers, the hidden states [T, 2048] bf16, the grouped gate-up input
    buffers and a down output [T * 8, 2048] bf16 to combine."""
    t, e, k, h = MOE_T, synth.MOE_EXPERTS, synth.MOE_TOPK, synth.MOE_HIDDEN
    r = synth.moe_routing(t, e, k, seed, 0)
    rows = t * k
    d = {"t": t, "e": e, "k": k, "h": h, "rows": rows,
         "topk": torch.from_numpy(r.topk).to(dev), "gate": torch.from_numpy(r.gate).to(dev),
         "ws": torch.empty(fp8rl.fp8rl_moe_plan_workspace_size(t, k, e), dtype=torch.uint8, device=dev),
         "off": torch.empty(e + 1, dtype=torch.int32, device=dev),
         "rop": torch.empty(rows, dtype=torch.int32, device=dev),
         "tor": torch.empty(rows, dtype=torch.int32, device=dev),
         "x": synth.normal_bf16((t, h), 1.0, seed, "bench-moe-layer-x", device=dev),
         "xq": torch.empty((rows, h), dtype=torch.uint8, device=dev),
         "sx": torch.empty((h // 128, rows), dtype=torch.float32, device=dev),
         "y": synth.normal_bf16((rows, h), 1.0, seed, "bench-moe-layer-y", device=dev),
         "out": torch.empty((t, h), dtype=torch.bfloat16, device=dev)}
    d["plan"] = lambda: fp8rl.fp8rl_moe_plan(d["topk"], t, k, e, d["off"], d["rop"], d["tor"], d["ws"],
                                             d["ws"].numel())
    d["dispatch"] = lambda: fp8rl.fp8rl_moe_dispatch_quant(d["x"], t, h, h, d["rop"], k, rows, d["xq"], h, d["sx"],
                                                           0)
    d["combine"] = lambda: fp8rl.fp8rl_moe_combine(d["y"], rows, h, h, d["rop"], d["gate"], t, k, d["out"], h)
    d["plan"]()
    # algorithmic bytes: hidden states read once, codes + scales + row map
    # written; combine: k expert rows read, one row written, plus the map
    d["dispatch_bytes"] = 2 * t * h + rows * h + 4 * rows * (h // 128) + 4 * rows
    d["combine_bytes"] = 2 * rows * h + 2 * t * h + 8 * rows
    return d


def section_moe_layer(torch, synth, fp8rl, dev, seed, peaks):
    """The MoE layer around the grouped GEMMs (Qwen3-30B-A3B shape, T = 4096,
    top-8 of 128 experts, hidden 2048): the dispatch plan of the replayed
    indices, the dispatch with 1x128 quantisation into the grouped gate-up
    input, and the weighted combine of the down outputs.  The working sets are
    near or below the L2 size, so L2 is flushed before every timed call."""
    hbm = peaks["hbm_gbs"]
    flush = l2_flusher(torch, dev)
    d = moe_layer_inputs(torch, synth, fp8rl, dev, seed)
    res = {"tokens": d["t"], "experts": d["e"], "topk": d["k"], "hidden": d["h"], "l2": "flushed before each call"}
    res["plan"] = {"ms": time_loop(torch, d["plan"], 20, 5, flush), "ms_graph": time_graph(torch, d["plan"], 50),
                   "launches": 1 if d["rows"] <= 8192 and d["e"] <= 256 else 3}
    for name in ("dispatch", "combine"):
        t = time_loop(torch, d[name], 20, 5, flush)
        b = d[name + "_bytes"]
        res[name] = {"ms": t, "bytes": b, "gbs": b / t / 1e6, "frac_hbm": b / t / 1e6 / hbm}
    # context: the plain quantiser over an already-gathered [T * 8, 2048] input
    rows, h = d["rows"], d["h"]
    aq = lambda: fp8rl.fp8rl_quant_act_group(d["y"], rows, h, h, d["xq"], h, d["sx"], 0)
    t = time_loop(torch, aq, 20, 5, flush)
    res["act_quant_gathered_rows"] = {"ms": t, "gbs": aq_bytes(rows, h) / t / 1e6}
    return res


def section_tis(torch, synth, fp8rl, dev, seed, peaks):
    """Token-level TIS weights and the mismatch KL over a rollout batch of
    512 responses x 16384 tokens (8.4 M tokens, 13 bytes each; L2 flushed
    before every timed call, as the 109 MB working set fits in L2)."""
    flush = l2_flusher(torch, dev)
    lt, lr, m = synth.rollout_logprobs(seed=seed, device=dev)
    n = lt.numel()
    ws = torch.zeros(fp8rl.fp8rl_tis_workspace_size(n), dtype=torch.uint8, device=dev)
    w = torch.empty(n, dtype=torch.float32, device=dev)
    kl = torch.empty(3, dtype=torch.float64, device=dev)
    fn = lambda: fp8rl.fp8rl_tis_weights(lt, lr, m, n, 2.0, w, kl, ws, ws.numel())
    t = time_loop(torch, fn, 20, 5, flush)
    b = 13 * n
    return {"tokens": n, "ms": t, "bytes": b, "gbs": b / t / 1e6, "frac_hbm": b / t / 1e6 / peaks["hbm_gbs"],
            "launches": 1, "l2": "flushed before each call"}


def section_decode_layer(torch, synth, fp8rl, dev, seed, peaks, m=16, layers=8):
    """The linear path of a rollout decode step at m tokens: per layer the four
    Qwen3-8B projections (qkv, o_proj, gate-up, down), each behind the 1x128
    quantisation of its input (the attention and SwiGLU outputs that feed
    o_proj and down are synthetic stand-ins of their shapes), over `layers`
    layers' weights (1.5 GB of codes, far beyond L2), captured once in a CUDA
    graph and replayed.  Timed as one fused call per projection
    (fp8rl_gemm_act_quant), and as two calls (quantiser, GEMM) with
    overlapped launches (the default: each kernel starts while the one before
    it finishes) and without them.  The same algorithmic bytes for all three
    (the fused form also writes the codes and scales out)."""
    gemms = synth.QWEN3_8B_GEMMS
    W = []
    for l in range(layers):
        per = []
        for name, n, k in gemms:
            w = synth.weight_bf16(n, k, seed, "decode", l, name, device=dev)
            wq, sw = fp8rl.quant_weight(w)
            del w
            per.append((n, k, wq, sw))
        W.append(per)
    ks = sorted({k for _, _, k in gemms})
    ns = sorted({n for _, n, _ in gemms})
    xs = {k: synth.activation_bf16(m, k, seed, "decode-x", k, device=dev) for k in ks}
    qs = {k: torch.empty((m, k), dtype=torch.uint8, device=dev) for k in ks}
    ss = {k: torch.empty((k // 128, m), dtype=torch.float32, device=dev) for k in ks}
    ys = {n: torch.empty((m, n), dtype=torch.bfloat16, device=dev) for n in ns}

    def run():
        for per in W:
            for n, k, wq, sw in per:
                fp8rl.fp8rl_quant_act_group(xs[k], m, k, k, qs[k], k, ss[k], 0)
                fp8rl.fp8rl_gemm_blockscaled(qs[k], ss[k], wq, sw, ys[n], m, n, k, 0)

    def run_fused():
        for per in W:
            for n, k, wq, sw in per:
                fp8rl.fp8rl_gemm_act_quant(xs[k], k, wq, sw, ys[n], m, n, k, 0, qs[k], ss[k])

    per_layer = sum(gemm_bytes(m, n, k) + aq_bytes(m, k) for _, n, k in gemms)
    res = {"m": m, "layers": layers, "bytes_per_layer": per_layer,
           "l2": "weights of all layers (%.2f GB) far larger than L2" % (layers * per_layer / 1e9)}
    hooks = os.environ.get("FP8RL_TEST_HOOKS")
    # two calls per projection (quantiser, GEMM) with and without overlapped
    # launches, and the one-call fused form (overlapped)
    for label, fn, off, launches in (("fused", run_fused, 0, len(gemms)), ("overlapped", run, 0, 2 * len(gemms)),
                                     ("serialised", run, 1, 2 * len(gemms))):
        if off:
            os.environ["FP8RL_TEST_HOOKS"] = "1"
            fp8rl.fp8rl_debug_set(fp8rl.DEBUG_PDL, 1)
        try:
            ms = time_graph(torch, fn, 1) / layers
        finally:
            if off:
                fp8rl.fp8rl_debug_set(fp8rl.DEBUG_PDL, 0)
                if hooks is None:
                    os.environ.pop("FP8RL_TEST_HOOKS", None)
                else:
                    os.environ["FP8RL_TEST_HOOKS"] = hooks
        gbs = per_layer / ms / 1e6
        res[label] = {"us_per_layer": ms * 1e3, "launches_per_layer": launches, "gbs": gbs,
                      "frac_hbm": gbs / peaks["hbm_gbs"]}
    return res


def section_sweep_one(torch, synth, fp8rl, dev, seed, peaks, name, n, k, m, fmt):
    w = synth.weight_bf16(n, k, seed, "ue8m0", name, device=dev)
    wq, sw = fp8rl.quant_weight(w, fmt)
    x = synth.activation_bf16(m, k, seed, "ue8m0-x", name, device=dev)
    xq, sx = fp8rl.quant_act(x, fmt)
    y = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    ms = time_loop(torch, lambda: fp8rl.fp8rl_gemm_blockscaled(xq, sx, wq, sw, y, m, n, k, fmt), 20, 5)
    r = gemm_roof(gemm_flops(m, n, k), gemm_bytes(m, n, k, 1), ms, peaks["hbm_gbs"],
                  fp8_peak(peaks))
    return {"m": m, "n": n, "k": k, "ms": ms, "tflops": r["tflops"], "frac": r["frac"], "bound": r["bound"]}


def cpu_baseline_sample(synth, seconds_cap=30.0):
    """The oracle, as it stands, on a bounded sample of the step's weight sync:
    the layer's matrices one after another until the time cap."""
    import oracle
    threads = oracle.default_threads()
    layer = synth.qwen3_8b_layer(0, 0, device="cpu")
    done_bytes, t0, names = 0, time.perf_counter(), []
    for name, w in layer:
        bits = synth.bf16_bits(w)
        oracle.quant_weight_blockwise(bits, oracle.SCALE_FP32, threads)
        done_bytes += wq_bytes(*w.shape)
        names.append(name)
        if time.perf_counter() - t0 > seconds_cap:
            break
    dt = time.perf_counter() - t0
    return {"value": done_bytes / dt / 1e9, "unit": UNIT, "cores": threads, "kind": "oracle",
            "sample": f"oracle weight sync of {'+'.join(names)} of one Qwen3-8B-shaped layer "
                      f"({done_bytes / 1e6:.0f} MB algorithmic), fp32 scales, {dt:.1f} s"}


def main_ours(args):
    import torch
    import torch.distributed as dist

    import fp8_w8a8_rollout_gb300 as fp8rl
    from fp8_w8a8_rollout_gb300 import synth

    world = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    if world > 1:
        dist.init_process_group("nccl")
    torch.cuda.set_device(local)
    dev = torch.device("cuda", local)
    fp8rl.load_library()
    stream = torch.cuda.current_stream().cuda_stream
    peaks = load_peaks()
    seed = 1000 + rank  # each rank syncs and runs its own layer replica (weak scaling)
    have_gemm = gemm_available(fp8rl, torch)

    inp = build_step_inputs(torch, synth, fp8rl, dev, seed, have_gemm)
    timer = Timer(torch, torch.cuda.current_stream())
    for _ in range(args.warmup):
        run_step(fp8rl, inp, timer, stream)
    torch.cuda.synchronize()
    timer = Timer(torch, torch.cuda.current_stream())

    def barrier():
        if world > 1:
            dist.barrier()
        torch.cuda.synchronize()

    launches = 0
    with ClockSampler(gpu_smi_id(torch, local), not args.no_clocks) as clocks:
        barrier()
        start = torch.cuda.Event(enable_timing=True)
        end = torch.cuda.Event(enable_timing=True)
        clocks.mark_start()
        start.record()
        for _ in range(args.steps):
            launches += run_step(fp8rl, inp, timer, stream)
        end.record()
        barrier()
        clocks.mark_end()
    total_ms = start.elapsed_time(end)
    timer.collect()
    status = fp8rl.fp8rl_sync_status()
    if status != 0:
        raise RuntimeError(f"device reported {fp8rl.STATUS.get(status, status)}")
    sync_ms = timer.avg_ms("weight_sync")
    wbytes = sum(wq_bytes(*w.shape) for w in inp["weights"])
    total_ms, sync_ms, value = aggregate_over_ranks(dist, torch, total_ms, sync_ms, wbytes, world, dev)

    if rank != 0:
        if world > 1:
            dist.barrier()
            dist.destroy_process_group()
        return

    roofs = step_rooflines(inp, timer, peaks)
    dominant = max(roofs, key=lambda k: roofs[k]["ms"])
    d = roofs[dominant]
    roofline = {"kernel": dominant, "bound": d["bound"], "achieved": d["achieved"], "peak": d["peak"],
                "unit": d["unit"], "frac": d["frac"], "traffic": captured_traffic(dominant),
                "peak_source": f"{peaks['source']} ({'hbm_gbs' if d['bound'] == 'hbm' else FP8_PEAK_BASIS})"}
    if d["bound"] == "tensor":
        # the same achieved rate against 2 x the sustained bf16 figure, for
        # comparison only (that figure belongs to seconds-long loops)
        roofline["frac_vs_2x_bf16_sustained"] = d["achieved"] / (2.0 * peaks["bf16_tflops_sustained"])
        # and against the nominal dense FP8 rate of the part (4.5 PFLOP/s),
        # the most conservative basis
        roofline["frac_vs_nominal_fp8_dense"] = d["achieved"] / NOMINAL_FP8_DENSE_TFLOPS
    e2e = e2e_weight_sync(torch, fp8rl, inp, stream, max(3, min(args.steps, 10)))
    sections = {}
    wanted = set(args.sections.split(",")) if args.sections not in ("all", "none") else (
        {"model", "moe_sync", "sweep", "ue8m0", "fused", "kv", "moe_layer", "tis", "decode"} if args.sections == "all"
        else set())
    del inp
    torch.cuda.empty_cache()
    if "model" in wanted:
        sections["model_sync_qwen3_8b_36_layers"] = section_model_sync(torch, synth, fp8rl, dev, seed, peaks)
    if "moe_sync" in wanted:
        sections["moe_sync_qwen3_30b_a3b_48x128_experts"] = section_moe_sync(torch, synth, fp8rl, dev, seed, peaks)
    if "sweep" in wanted and have_gemm:
        sections["gemm_sweep_qwen3_8b"] = section_sweep(torch, synth, fp8rl, dev, seed, peaks)
    if "ue8m0" in wanted:
        sections["ue8m0"] = section_ue8m0(torch, synth, fp8rl, dev, seed, peaks, have_gemm)
    if "fused" in wanted and have_gemm:
        sections["fused_mlp"] = section_fused_mlp(torch, synth, fp8rl, dev, seed, peaks)
    if "kv" in wanted:
        sections["kv_cache_qwen3_8b_layer"] = section_kv_cache(torch, synth, fp8rl, dev, seed, peaks)
    if "moe_layer" in wanted:
        sections["moe_dispatch_combine_qwen3_30b_a3b"] = section_moe_layer(torch, synth, fp8rl, dev, seed, peaks)
    if "tis" in wanted:
        sections["tis_rollout_512x16384"] = section_tis(torch, synth, fp8rl, dev, seed, peaks)
    if "decode" in wanted and have_gemm:
        sections["decode_layer_qwen3_8b_m16"] = section_decode_layer(torch, synth, fp8rl, dev, seed, peaks)
    cpu = None
    if not args.no_cpu_baseline and world == 1:
        cpu = cpu_baseline_sample(synth)

    line = {
        "metric": METRIC, "value": value, "unit": UNIT, "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": total_ms / args.steps, "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "e4m3 x e4m3 -> fp32 acc -> bf16",
        "data": "synthetic (seeded; N(0,0.02) weights with 0.1% x20 outliers, lognormal-channel activations)",
        "config": {"workload": WORKLOAD, "weight_sync": "7 linears, 192,937,984 bf16 params, fp32 128x128 scales",
                   "forward_tokens": STEP_M if have_gemm else 0, "moe_tokens": MOE_T if have_gemm else 0,
                   "parallelism": f"replicas x{world}",
                   "l2": "step working set > 1 GB, larger than L2 (129 MB); no explicit flush"},
        "weight_sync_ms": sync_ms,
        "gemm_available": have_gemm,
        "roofline": roofline,
        "phases": roofs,
        "e2e": e2e,
        "gpu_launches": launches,
        "cpu_baseline": cpu,
        "clocks": clocks.summary(),
        "sections": sections,
        "peaks": peaks,
    }
    print(json.dumps(line))
    sys.stdout.flush()
    if world > 1:
        dist.barrier()
        dist.destroy_process_group()


def aggregate_over_ranks(dist, torch, total_ms, sync_ms, wbytes, world, device):
    """Replicas (weak scaling): the timed region's and the weight-sync phase's
    times are the maximum over ranks; the value is the bytes all ranks synced
    divided by that time.  Returns (total_ms, sync_ms, GB/s)."""
    t = torch.tensor([total_ms, sync_ms], dtype=torch.float64, device=device)
    if world > 1:
        dist.all_reduce(t, op=dist.ReduceOp.MAX)
    total_ms, sync_ms = float(t[0]), float(t[1])
    return total_ms, sync_ms, world * wbytes / sync_ms / 1e6


def main_reference(args):
    """The CPU oracle as the reference arm, on rank 0 only."""
    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    if rank != 0:
        return
    import oracle
    from fp8_w8a8_rollout_gb300 import synth
    threads = oracle.default_threads()
    layer = synth.qwen3_8b_layer(0, 0, device="cpu")
    mats = [(name, synth.bf16_bits(w)) for name, w in layer]
    # each step quantises one matrix of the layer, rotating through them
    for i in range(args.warmup):
        oracle.quant_weight_blockwise(mats[i % len(mats)][1], oracle.SCALE_FP32, threads)
    t0 = time.perf_counter()
    done = 0
    for i in range(args.steps):
        bits = mats[i % len(mats)][1]
        oracle.quant_weight_blockwise(bits, oracle.SCALE_FP32, threads)
        done += wq_bytes(*bits.shape)
    dt = time.perf_counter() - t0
    value = done / dt / 1e9
    print(json.dumps({
        "impl": "reference", "metric": METRIC, "value": value, "unit": UNIT, "n_gpus": world,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": dt * 1e3 / args.steps,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64/f32 CPU",
        "data": "synthetic", "config": {"workload": WORKLOAD, "parallelism": "rank 0 only"},
        "cpu_baseline": {"value": value, "unit": UNIT, "cores": threads, "kind": "oracle",
                         "sample": "one matrix of the Qwen3-8B-shaped layer per step, rotating"},
        "e2e": {"value": value, "unit": UNIT, "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }))


def main_case(args):
    """One kernel alone, --warmup + --steps launches; prints its median time."""
    import torch

    import fp8_w8a8_rollout_gb300 as fp8rl
    from fp8_w8a8_rollout_gb300 import synth
    dev = torch.device("cuda")
    flush = None  # set by the cases whose inputs L2 could hold between calls
    os.environ["FP8RL_TEST_HOOKS"] = "1"  # --case may force tile widths and schedules
    fp8rl.load_library()
    if args.bn:
        fp8rl.fp8rl_debug_set(fp8rl.DEBUG_GEMM_BN, args.bn)
    if args.wait_mode:
        fp8rl.fp8rl_debug_set(4, args.wait_mode)
    if args.l2_prefetch >= 0:
        fp8rl.fp8rl_debug_set(5, args.l2_prefetch)
    if args.out_stage:
        fp8rl.fp8rl_debug_set(fp8rl.DEBUG_OUT_STAGE, args.out_stage)
    if args.mx:
        fp8rl.fp8rl_debug_set(fp8rl.DEBUG_MX, args.mx)
    if args.pair:
        fp8rl.fp8rl_debug_set(fp8rl.DEBUG_PAIR, args.pair)
    if args.no_overlap:
        fp8rl.fp8rl_debug_set(fp8rl.DEBUG_PDL, 1)
    parts = args.case.split(":")
    kind = parts[0]
    peaks = load_peaks()
    fp8 = fp8_peak(peaks)
    if kind == "gemm":
        m, n, k = (int(v) for v in parts[1:4])
        fmt = int(parts[4]) if len(parts) > 4 else 0
        w = synth.weight_bf16(n, k, 0, "case", device=dev)
        wq, sw = fp8rl.quant_weight(w, fmt)
        x = synth.activation_bf16(m, k, 0, "case-x", device=dev)
        xq, sx = fp8rl.quant_act(x, fmt)
        y = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
        if args.streamk >= 0:
            fp8rl.fp8rl_debug_set(fp8rl.DEBUG_STREAMK, args.streamk)
            fp8rl.fp8rl_debug_set(fp8rl.DEBUG_STREAMK_GRID, args.streamk_grid)
            ws = fp8rl.gemm_workspace(dev)
            fn = lambda: fp8rl.fp8rl_gemm_blockscaled_ws(xq, sx, wq, sw, y, m, n, k, fmt, ws, ws.numel())
        else:
            fn = lambda: fp8rl.fp8rl_gemm_blockscaled(xq, sx, wq, sw, y, m, n, k, fmt)
        work = gemm_roof(gemm_flops(m, n, k), gemm_bytes(m, n, k), 1.0, peaks["hbm_gbs"], fp8)
    elif kind == "grouped":
        which = parts[1]
        fmt = int(parts[2]) if len(parts) > 2 else 0
        n, k = (2 * synth.MOE_INTER, synth.MOE_HIDDEN) if which == "gate_up" else (synth.MOE_HIDDEN, synth.MOE_INTER)
        _, offsets, _, _, rows = moe_plan_for(torch, synth, fp8rl, dev, 0)
        wb = synth.moe_expert_weights(n, k, synth.MOE_EXPERTS, 0, 0, which, device=dev)
        wq, sw = fp8rl.quant_weight(wb.view(-1, k), fmt)
        wq = wq.view(synth.MOE_EXPERTS, n, k)
        sw = sw.view(synth.MOE_EXPERTS, n // 128, k // 128)
        x = synth.normal_bf16((rows, k), 1.0, 0, "case-x", device=dev)
        xq, sx = fp8rl.quant_act(x, fmt)
        y = torch.empty((rows, n), dtype=torch.bfloat16, device=dev)
        fn = lambda: fp8rl.fp8rl_grouped_gemm_blockscaled(xq, sx, wq, sw, offsets, synth.MOE_EXPERTS, rows, n, k, y,
                                                          fmt)
        sb = 4 if fmt == 0 else 1
        work = {"flops": gemm_flops(rows, n, k),
                "bytes": synth.MOE_EXPERTS * (n * k + sb * (n // 128) * (k // 128)) + rows * k + 2 * rows * n
                + sb * rows * (k // 128)}
    elif kind in ("fused", "fused_moe"):
        fmt = int(parts[-1]) if (kind == "fused" and len(parts) > 2) or (kind == "fused_moe" and len(parts) > 1) else 0
        d = fused_mlp_inputs(torch, synth, fp8rl, dev, 0, int(parts[1]) if kind == "fused" else 0, fmt,
                             kind == "fused_moe")
        m, inter, k = d["m"], d["inter"], d["k"]
        hq = torch.empty((m, inter), dtype=torch.uint8, device=dev)
        hs = torch.empty((inter // 128, m), dtype=torch.float32 if fmt == 0 else torch.uint8, device=dev)
        if kind == "fused_moe":
            fn = lambda: fp8rl.fp8rl_grouped_gemm_swiglu_quant(d["xq"], d["sx"], d["wq"], d["sw"], d["offsets"],
                                                              d["experts"], m, inter, k, hq, hs, fmt)
        else:
            fn = lambda: fp8rl.fp8rl_gemm_swiglu_quant(d["xq"], d["sx"], d["wq"], d["sw"], m, inter, k, hq, hs, fmt)
        work = {"flops": 2.0 * m * 2 * inter * k}
    elif kind == "kvcal":
        tokens = int(parts[1])
        k, v, _, _, _ = kv_inputs(torch, synth, dev, 0, tokens, tokens)
        q = synth.normal_bf16((tokens, Q_DIM), 1.0, 0, "case-kv-q", device=dev)
        scales = torch.zeros(3, dtype=torch.float32, device=dev)
        fn = lambda: fp8rl.kv_calibrate(k, v, q, out=scales)
        work = {"bytes": tokens * (2 * KV_DIM + Q_DIM) * 2}
        if tokens * (2 * KV_DIM + Q_DIM) * 2 < 2 * L2_BYTES:
            flush = l2_flusher(torch, dev)  # inputs L2 could hold: flush before every call
    elif kind == "kv":
        tokens = int(parts[1])
        k, v, slots, kc, vc = kv_inputs(torch, synth, dev, 0, tokens, max(65536, tokens))
        scales = fp8rl.kv_calibrate(k, v)
        fn = lambda: fp8rl.kv_append(k, v, slots, kc, vc, scales)
        work = {"bytes": tokens * KV_DIM * 2 * 3 + tokens * 4}
    elif kind in ("moe_plan", "moe_dispatch", "moe_combine"):
        d = moe_layer_inputs(torch, synth, fp8rl, dev, 0)
        fn = d[kind[4:]]
        work = {"bytes": d[kind[4:] + "_bytes"]} if kind != "moe_plan" else {}
    elif kind == "tis":
        lt, lr, msk = synth.rollout_logprobs(int(parts[1]) if len(parts) > 1 else synth.ROLLOUT_RESPONSES,
                                             device=dev)
        n = lt.numel()
        ws = torch.zeros(fp8rl.fp8rl_tis_workspace_size(n), dtype=torch.uint8, device=dev)
        w = torch.empty(n, dtype=torch.float32, device=dev)
        kl = torch.empty(3, dtype=torch.float64, device=dev)
        fn = lambda: fp8rl.fp8rl_tis_weights(lt, lr, msk, n, 2.0, w, kl, ws, ws.numel())
        work = {"bytes": 13 * n}
    elif kind == "op":
        from perf import operators as ops
        case = next((c for c in ops.listed() if c["name"] == parts[1]), None)
        if case is None:
            raise SystemExit(f"no case named {parts[1]!r}: " + ", ".join(c["name"] for c in ops.listed()))
        ops.own = True
        state = ops.prepare(case, 0)
        fn = lambda: ops.run(state)
        work = ops.work(case)
        if work["bytes"] < 2 * L2_BYTES:
            flush = l2_flusher(torch, dev)
    elif kind == "wq":
        fmt = int(parts[2]) if len(parts) > 2 else 0
        layer = [w for _, w in synth.qwen3_8b_layer(0, 0, device=dev)]
        outs = fp8rl.quant_weights_batched(layer, fmt)
        descs = fp8rl.weight_descs([(w, q, sc) for w, (q, sc) in zip(layer, outs)])
        fn = lambda: fp8rl.fp8rl_quant_weight_blockwise_batched(descs, len(layer), fmt)
        work = {"bytes": sum(wq_bytes(*w.shape, 4 if fmt == 0 else 1) for w in layer)}
    elif kind == "aq":
        m, k = int(parts[1]), int(parts[2])
        fmt = int(parts[3]) if len(parts) > 3 else 0
        x = synth.activation_bf16(m, k, 0, "case-x", device=dev)
        q = torch.empty((m, k), dtype=torch.uint8, device=dev)
        sc = torch.empty(((k + 127) // 128, m), dtype=torch.float32 if fmt == 0 else torch.uint8, device=dev)
        fn = lambda: fp8rl.fp8rl_quant_act_group(x, m, k, k, q, k, sc, fmt)
        work = {"bytes": aq_bytes(m, k, 4 if fmt == 0 else 1)}
    elif kind == "aqg":
        # the activation quantisation and the GEMM in one call (fp8rl_gemm_act_quant)
        m, n, k = (int(v) for v in parts[1:4])
        fmt = int(parts[4]) if len(parts) > 4 else 0
        w = synth.weight_bf16(n, k, 0, "case-w", device=dev)
        wq, sw = fp8rl.quant_weight(w, fmt)
        del w
        x = synth.activation_bf16(m, k, 0, "case-x", device=dev)
        q = torch.empty((m, k), dtype=torch.uint8, device=dev)
        sc = torch.empty((k // 128, m), dtype=torch.float32 if fmt == 0 else torch.uint8, device=dev)
        y = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
        fn = lambda: fp8rl.fp8rl_gemm_act_quant(x, k, wq, sw, y, m, n, k, fmt, q, sc)
        work = {"bytes": gemm_bytes(m, n, k, 4 if fmt == 0 else 1) + aq_bytes(m, k, 4 if fmt == 0 else 1)}
    else:
        raise SystemExit(f"unknown case {args.case}")
    ms = time_loop(torch, fn, max(1, args.steps), args.warmup, flush)
    assert fp8rl.fp8rl_sync_status() == 0
    out = {"case": args.case, "ms": ms, "bn": args.bn or "auto", "wait_mode": args.wait_mode,
           "l2_prefetch": args.l2_prefetch, "streamk": args.streamk, "out_stage": args.out_stage, "mx": args.mx, "pair": args.pair,
           "overlap": not args.no_overlap}
    if args.graph:
        out["ms_graph"] = time_graph(torch, fn, max(10, args.steps))
    if "flops" in work:
        out["tflops"] = work["flops"] / ms / 1e9
    if "bytes" in work:
        out["gbs"] = work["bytes"] / ms / 1e6
    print(json.dumps(out))


if __name__ == "__main__":
    a = parse()
    if a.case:
        main_case(a)
    elif a.impl == "reference":
        main_reference(a)
    else:
        main_ours(a)
