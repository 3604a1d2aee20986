#!/usr/bin/env python
"""Benchmark of the FP8 quantize + scaling-aware direct transpose hot path on B200.

    python bench.py [--gpus N] [--steps K] [--warmup W] [--impl ours|reference]

One step = one pass of the hot path over the dense-activation workload (X bf16
[8192, 7168], N(0,1) times a lognormal(0, 1.5) row factor, 7 outlier channels x100):
fp8q_quantize_rowwise (X -> Q, SF) and fp8q_direct_transpose (Q, SF -> Q^T, SF^T).
The kernels stream over four rotating buffer sets (944 MB, more than seven times the
L2): step k quantizes set k mod 4 and transposes set (k - 2) mod 4, whose codes were
written two steps (590 MB of traffic) earlier, so both kernels read their inputs from
HBM and each pays for the write-back of the lines it displaces, as in a long run; every
batch still goes through both kernels.  The K timed steps are bracketed by one pair of
CUDA events on the launching stream, with nothing between the launches; each kernel's
own duration (for the roofline) comes from K back-to-back launches of that kernel over
the same sets, again in one event pair.  The metric is algorithmic HBM bytes / time
(every input byte read once, every output byte written once), in GB/s.  With N ranks (torchrun, one GPU each) every rank runs its own batches (weak
scaling, no collective on the data path); the value is all ranks' bytes over the
slowest rank's time.  Rank 0 prints one JSON line.

--impl reference times the CPU oracle (plain C, the parity reference) on the host cores
on a bounded sample of the same workload; only rank 0 runs it.
"""
from __future__ import annotations

import argparse
import hashlib
import json
import os
import re
import statistics
import sys
import threading
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

WORKLOAD = "dense activation X bf16 [8192, 7168]: N(0,1) x lognormal(0,1.5) per row, 7 outlier channels x100"
ROWS, COLS = 8192, 7168
N_ELEM = ROWS * COLS
BYTES_QUANT = 2 * N_ELEM + N_ELEM + N_ELEM // 128            # read X, write Q + SF
BYTES_DIRECT = N_ELEM + N_ELEM // 128 + N_ELEM + N_ELEM // 128  # read Q + SF, write Q^T + SF^T
BYTES_STEP = BYTES_QUANT + BYTES_DIRECT
BYTES_ROWCOL = 2 * N_ELEM + 2 * (N_ELEM + N_ELEM // 128)      # read X, write Q + SF + Q^T + SF^T
BYTES_MX_QUANT = 3 * N_ELEM + N_ELEM // 32                      # 1x32 tiles
BYTES_MX_DIRECT = 2 * (N_ELEM + N_ELEM // 32)                   # 32x32 blocks
METRIC = "direct-transpose & quantize GB/s on 1 B200 (% of HBM peak); bit-exact vs oracle"
FLUSH_BYTES = 256 << 20
SETS = 4   # rotating buffer sets of the timed loop
LAG = 2    # the transpose of step k reads the codes quantized in step k - LAG
FALLBACK_HBM_GBS = 6650.0


# ------------------------------------------------------------------ host helpers
def measured_peak_gbs():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        with open(p) as f:
            v = float(json.load(f)["hbm_gbs"])
        return v, "measured"
    except Exception:
        return FALLBACK_HBM_GBS, "fallback"


def kernel_sources(kind: str):
    csrc = os.path.join(ROOT, "scaling_aware_transpose_b200", "csrc")
    main = {"quantize": "quantize_rowwise.cu", "direct": "direct_transpose.cu", "swiglu": "swiglu_quant.cu",
            "permute": "permute_pad_quant.cu", "rowwise_colwise": "quantize_rowwise_colwise.cu",
            "unpermute": "unpermute_unpad.cu", "unpermute_fp8": "unpermute_unpad.cu", "mx32": "mx32.cu",
            "mx32_quantize": "mx32.cu", "direct_grouped": "direct_transpose.cu", "naive": "naive_transpose.cu",
            "direct_stress": "direct_transpose.cu",
            "permute_fp8": "permute_pad_quant.cu", "ep_pack": "ep_dispatch.cu", "ep_recv": "ep_dispatch.cu",
            "permute_e512": "permute_pad_quant.cu", "permute_e4096": "permute_pad_quant.cu",
            "unpermute_fp8_k": "unpermute_unpad.cu", "router": "router.cu", "router_wide": "router.cu",
            "router_rows": "router.cu", "mxfp4_permute_few": "mxfp4_quant.cu",
            "swiglu_stash": "swiglu_quant.cu", "swiglu_bwd": "swiglu_bwd.cu", "swiglu_bwd_quant": "swiglu_bwd.cu",
            "mxfp4_quantize": "mxfp4_quant.cu", "mxfp4_permute": "mxfp4_quant.cu", "mxfp4_matmul": "mxfp4_matmul.cu",
            "mxfp4_token": "mxfp4_matmul.cu", "mxfp4_experts": "mxfp4_matmul.cu"}[kind]
    extra = ["permute_common.cuh", "permute_pad_quant.cu"] if kind in ("ep_pack", "ep_recv") else []
    if kind in ("permute", "permute_fp8", "permute_e512", "permute_e4096"):
        extra = ["permute_common.cuh"]
    if kind.startswith("router"):
        extra = ["cluster.cuh"]
    if kind in ("mxfp4_quantize", "mxfp4_permute", "mxfp4_permute_few"):
        extra = ["mxfp4.cuh", "permute_common.cuh"]
    if kind in ("mxfp4_matmul", "mxfp4_token", "mxfp4_experts"):
        extra = ["mxfp4.cuh", "bulk.cuh", "cluster.cuh"]
    return [os.path.join(csrc, main), os.path.join(csrc, "common.cuh")] + [os.path.join(csrc, e) for e in extra]


def source_digest(paths) -> str:
    h = hashlib.sha256()
    for p in paths:
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


def profiled_traffic(kind: str):
    """DRAM bytes per launch from the committed ncu summary of this kernel on this
    workload, or None when there is none or the kernel source changed since."""
    name = {"quantize": "quantize_rowwise_dense_8192x7168.md", "direct": "direct_transpose_dense_8192x7168.md",
            "rowwise_colwise": "quantize_rowwise_colwise_dense_8192x7168.md"}[kind]
    p = os.path.join(ROOT, "profiles", name)
    if not os.path.exists(p):
        return None
    txt = open(p).read()
    m = re.search(r"dram_bytes_per_launch:\s*(\d+)", txt)
    s = re.search(r"source_sha256:\s*([0-9a-f]+)", txt)
    if not m or not s or s.group(1) != source_digest(kernel_sources(kind)):
        return None
    return int(m.group(1))


def roofline(bytes_per_launch: int, avg_seconds: float, peak_gbs: float, peak_kind: str, traffic):
    achieved = bytes_per_launch / avg_seconds / 1e9
    return {"bound": "hbm", "achieved": round(achieved, 1), "peak": peak_gbs, "unit": "GB/s",
            "frac": round(achieved / peak_gbs, 4), "peak_source": f"{peak_kind} (MEASURED_PEAKS.json hbm_gbs)"
            if peak_kind == "measured" else "fallback", "traffic": traffic}


def reduce_max(value: float, dist_mod=None, device=None) -> float:
    """Max of a per-rank float over all ranks (identity without a process group)."""
    if dist_mod is None or not dist_mod.is_initialized() or dist_mod.get_world_size() == 1:
        return value
    import torch
    t = torch.tensor([value], dtype=torch.float64, device=device)
    dist_mod.all_reduce(t, op=dist_mod.ReduceOp.MAX)
    return float(t.item())


class ClockSampler:
    """Samples SM clock and clock-event (throttle) reasons through NVML in a thread."""

    REASONS = {0x1: "gpu_idle", 0x2: "applications_clocks_setting", 0x4: "sw_power_cap", 0x8: "hw_slowdown",
               0x10: "sync_boost", 0x20: "sw_thermal_slowdown", 0x40: "hw_thermal_slowdown",
               0x80: "hw_power_brake_slowdown", 0x100: "display_clock_setting"}

    def __init__(self, device_index: int, period_s: float = 0.005):
        self.samples, self.reasons, self.max_mhz = [], 0, None
        self.period, self.idx, self._stop, self._t = period_s, device_index, threading.Event(), None
        try:
            import pynvml
            pynvml.nvmlInit()
            self._nv = pynvml
            self._h = pynvml.nvmlDeviceGetHandleByIndex(device_index)
            self.max_mhz = pynvml.nvmlDeviceGetMaxClockInfo(self._h, pynvml.NVML_CLOCK_SM)
        except Exception:
            self._nv = None

    def _run(self):
        nv = self._nv
        while not self._stop.is_set():
            try:
                self.samples.append(nv.nvmlDeviceGetClockInfo(self._h, nv.NVML_CLOCK_SM))
                self.reasons |= int(nv.nvmlDeviceGetCurrentClocksEventReasons(self._h))
            except Exception:
                pass
            self._stop.wait(self.period)

    def __enter__(self):
        if self._nv is not None:
            self._t = threading.Thread(target=self._run, daemon=True)
            self._t.start()
        return self

    def __exit__(self, *exc):
        self._stop.set()
        if self._t is not None:
            self._t.join()

    def summary(self):
        reasons = [n for bit, n in self.REASONS.items() if self.reasons & bit and n != "gpu_idle"]
        return {"sm_mhz": statistics.median(self.samples) if self.samples else None, "sm_max_mhz": self.max_mhz,
                "reasons": reasons, "samples": len(self.samples), "source": "nvml" if self._nv else "unavailable"}


def cpu_baseline(x_bits, budget_s: float = 10.0, max_reps: int = 50):
    """The oracle (quantize + direct transpose) as it stands, on the host cores, over the
    full workload, repeated until the time budget is spent."""
    import oracle
    times, reps = [], 0
    t_end = time.perf_counter() + budget_s
    while reps < max_reps and (reps < 1 or time.perf_counter() < t_end):
        t0 = time.perf_counter()
        q, sf = oracle.quantize_rowwise(x_bits)
        oracle.direct_transpose(q, sf)
        times.append(time.perf_counter() - t0)
        reps += 1
    rows = x_bits.shape[0]
    step_bytes = BYTES_STEP * rows // ROWS
    avg = sum(times) / len(times)
    cores = oracle.num_threads()
    # one thread, on the first 1/8 of the rows (a few seconds)
    sub = x_bits[: max(128, rows // 8)]
    oracle.set_num_threads(1)
    try:
        t0 = time.perf_counter()
        q, sf = oracle.quantize_rowwise(sub)
        oracle.direct_transpose(q, sf)
        t1 = time.perf_counter() - t0
    finally:
        oracle.set_num_threads(cores)
    return {"value": round(step_bytes / avg / 1e9, 3), "unit": "GB/s", "cores": cores,
            "kind": "oracle", "sample": f"{rows}x{COLS} rows of the workload (quantize + direct transpose), "
                                        f"{reps} repetitions, {sum(times):.1f} s",
            "value_1_thread": round(BYTES_STEP * sub.shape[0] // ROWS / t1 / 1e9, 3),
            "sample_1_thread": f"{sub.shape[0]}x{COLS} rows, one repetition, {t1:.1f} s"}



def time_on_stream(fn, reps, stream, before=None):
    """Median device time (s) of fn() over reps launches, each bracketed by CUDA events on
    `stream`; `before` (e.g. an L2 flush) runs outside the events."""
    import torch
    pairs = []
    for _ in range(reps):
        if before is not None:
            before()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(stream)
        fn()
        b.record(stream)
        pairs.append((a, b))
    torch.cuda.synchronize()
    return statistics.median(a.elapsed_time(b) * 1e-3 for a, b in pairs)


def time_steady(calls, n, stream):
    """Mean device time (s) of n back-to-back launches cycling over `calls` (one callable
    per buffer set), bracketed by one pair of CUDA events on `stream`; nothing runs
    between the launches."""
    import torch
    for c in calls:
        c()
    torch.cuda.synchronize()
    torch.cuda._sleep(2_000_000)  # the host queues the launches while the GPU waits
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(stream)
    for i in range(n):
        calls[i % len(calls)]()
    b.record(stream)
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e-3 / n


def sets_for(bytes_per_set: int, l2_bytes: int) -> int:
    """Buffer sets a steady-state loop cycles over: together at least three times the L2,
    and never fewer than two (so no launch reads what the previous one touched)."""
    return max(2, -(-3 * l2_bytes // max(bytes_per_set, 1)))


def measure_workloads(reps, device, stream, peak):
    """The other hot-path rows on their own workloads, each kernel timed in steady state
    (back-to-back launches over rotating buffer sets, see time_steady): fused
    SwiGLU+quantize(+transpose) on gate/up [32768, 2048]; fused permute+pad(128)+quantize
    of X [16384, 7168] with top-8 of 32 Zipf(1.1) experts, the FP8-input permute, the
    grouped direct transpose on the permute's device offsets, and the combine-side
    unpermute+unpad of BF16 expert outputs (weighted) and of the FP8 rows (unit weights);
    the expert-parallel dispatch of the same tokens over 4 ranks (pack on one source
    rank, receive permute on one destination rank from four source segments); quantize +
    direct transpose on the range-stress X [65536, 7168]."""
    import torch

    import scaling_aware_transpose_b200 as sat
    from scaling_aware_transpose_b200 import synthetic
    sp = stream.cuda_stream
    l2 = torch.cuda.get_device_properties(device).L2_cache_size
    n = max(6, reps)

    def entry(nbytes, t, sets):
        gbs = nbytes / t / 1e9
        return {"us": round(t * 1e6, 2), "bytes": int(nbytes), "GB/s": round(gbs, 1),
                "frac_of_peak": round(gbs / peak, 4), "sets": sets}

    def copies(t, k):
        return [t] + [t.clone() for _ in range(k - 1)]

    out = {}
    # SwiGLU
    d = synthetic.swiglu()
    g0 = synthetic.to_torch_bf16(d["gate"]).to(device)
    u0 = synthetic.to_torch_bf16(d["up"]).to(device)
    R, C = g0.shape
    ne = R * C
    b_sw = 4 * ne + 2 * (ne + ne // 128)
    S = sets_for(b_sw, l2)
    g, u = copies(g0, S), copies(u0, S)
    q = [torch.empty((R, C), dtype=torch.uint8, device=device) for _ in range(S)]
    sf = [torch.empty((R, C // 128), dtype=torch.uint8, device=device) for _ in range(S)]
    qt = [torch.empty((C, R), dtype=torch.uint8, device=device) for _ in range(S)]
    sft = [torch.empty((C, R // 128), dtype=torch.uint8, device=device) for _ in range(S)]
    t = time_steady([lambda i=i: sat.fp8q_swiglu_quant(g[i], u[i], R, C, q[i], sf[i], qt[i], sft[i], sp)
                     for i in range(S)], n, stream)
    t_row = time_steady([lambda i=i: sat.fp8q_swiglu_quant(g[i], u[i], R, C, q[i], sf[i], None, None, sp)
                         for i in range(S)], n, stream)
    out["swiglu_quant [32768x2048] (+transpose)"] = entry(b_sw, t, S)
    out["swiglu_quant [32768x2048] (row-wise only)"] = entry(4 * ne + ne + ne // 128, t_row, S)
    del g, u, q, sf, qt, sft, g0, u0
    torch.cuda.empty_cache()
    # MoE: permute + pad + quantize, FP8-input permute, grouped direct transpose, combine
    d = synthetic.moe()
    x0 = synthetic.to_torch_bf16(d["x"]).to(device)
    idx = torch.from_numpy(d["topk_idx"]).to(device)
    T, H = x0.shape
    K, E, align = idx.shape[1], d["num_experts"], 128
    max_rows = sat.permute_max_rows(T, K, E, align)
    ws = torch.empty(sat.fp8q_permute_workspace_bytes(T, K, E), dtype=torch.uint8, device=device)
    off = torch.empty(E + 1, dtype=torch.int32, device=device)
    rmap = torch.empty(T * K, dtype=torch.int32, device=device)
    S = 2
    xs = copies(x0, S)
    q = [torch.empty((max_rows, H), dtype=torch.uint8, device=device) for _ in range(S)]
    sf = [torch.empty((max_rows, H // 128), dtype=torch.uint8, device=device) for _ in range(S)]
    t_perm = time_steady([lambda i=i: sat.fp8q_permute_pad_quant(xs[i], T, H, idx, K, E, align, q[i], sf[i], max_rows,
                                                                 off, rmap, ws, ws.numel(), sp) for i in range(S)],
                         n, stream)
    R = int(off[-1].item())
    # FP8-input permute (the dispatch delivered row-wise codes and scales)
    xq0, xsf0 = sat.quantize_rowwise(x0)
    xq, xsf = copies(xq0, S), copies(xsf0, S)
    q8 = [torch.empty_like(q[0]) for _ in range(S)]
    sf8 = [torch.empty_like(sf[0]) for _ in range(S)]
    t_perm8 = time_steady([lambda i=i: sat.fp8q_permute_pad_fp8(xq[i], xsf[i], T, H, idx, K, E, align, q8[i], sf8[i],
                                                                max_rows, off, rmap, ws, ws.numel(), sp)
                           for i in range(S)], n, stream)
    del q8, sf8
    torch.cuda.empty_cache()
    qt = [torch.empty(max_rows * H, dtype=torch.uint8, device=device) for _ in range(S)]
    sft = [torch.empty(max_rows * H // 128, dtype=torch.uint8, device=device) for _ in range(S)]
    t_gt = time_steady([lambda i=i: sat.fp8q_direct_transpose(q[i], sf[i], max_rows, H, off, E, qt[i], sft[i], sp)
                        for i in range(S)], n, stream)
    perm_bytes = 2 * T * H + 4 * T * K + R * (H + H // 128) + 4 * (E + 1) + 4 * T * K
    out[f"permute_pad_quant [16384x7168] top8/32 -> {R} rows"] = entry(perm_bytes, t_perm, S)
    perm8_bytes = T * (H + H // 128) + 4 * T * K + R * (H + H // 128) + 4 * (E + 1) + 4 * T * K
    out[f"permute_pad_fp8 [16384x7168] top8/32 -> {R} rows"] = entry(perm8_bytes, t_perm8, S)
    out[f"direct_transpose grouped [{R}x7168] 32 experts"] = entry(2 * R * (H + H // 128), t_gt, S)
    del qt, sft
    torch.cuda.empty_cache()
    # combine side: unpermute + unpad of BF16 expert outputs with routing weights, and of
    # the FP8 rows with unit weights (the permute's backward shape)
    c = synthetic.moe_combine(rows=R, topk=K)
    y0 = synthetic.to_torch_bf16(c["y"]).to(device)
    ys = copies(y0, S)
    wts = torch.from_numpy(c["weights"]).to(device)
    comb = [torch.empty((T, H), dtype=torch.bfloat16, device=device) for _ in range(S)]
    t_ub = time_steady([lambda i=i: sat.fp8q_unpermute_unpad(ys[i], None, R, H, rmap, wts, T, K, comb[i], sp)
                        for i in range(S)], n, stream)
    t_uq = time_steady([lambda i=i: sat.fp8q_unpermute_unpad(q[i], sf[i], max_rows, H, rmap, None, T, K, comb[i], sp)
                        for i in range(S)], n, stream)
    out[f"unpermute_unpad bf16 [{R}x7168] -> [16384x7168], weighted"] = entry(
        T * K * 2 * H + 2 * T * H + 8 * T * K, t_ub, S)
    out[f"unpermute_unpad fp8 [{R}x7168] -> [16384x7168], unit weights"] = entry(
        T * K * (H + H // 128) + 2 * T * H + 4 * T * K, t_uq, S)
    del ys, y0, comb, q, sf, xs
    torch.cuda.empty_cache()
    # expert-parallel dispatch of the same tokens over 4 ranks of 8 experts: the send-side
    # pack of rank 0's 4096 tokens, and rank 0's receive permute from four source segments
    # (the four ranks' send buffers, read in place as an all-to-all receive buffer would be)
    W, Tr = 4, T // 4
    Eloc = E // W
    packs = [sat.ep_dispatch_pack(xq0[r * Tr:(r + 1) * Tr], xsf0[r * Tr:(r + 1) * Tr], idx[r * Tr:(r + 1) * Tr], W,
                                  Eloc) for r in range(W)]
    torch.cuda.synchronize()
    offs = [p[3].tolist() for p in packs]
    sent0 = offs[0][W]
    pk_ws = torch.empty(sat.fp8q_ep_pack_workspace_bytes(Tr, W), dtype=torch.uint8, device=device)
    pk_out = packs[0][:5]
    xq_r, xsf_r, idx_r = xq0[:Tr], xsf0[:Tr], idx[:Tr]
    t_pack = time_steady([lambda: sat.fp8q_ep_dispatch_pack(xq_r, xsf_r, Tr, H, idx_r, K, W, Eloc, pk_out[0], pk_out[1],
                                                            pk_out[2], pk_out[0].shape[0], pk_out[3], pk_out[4], pk_ws,
                                                            pk_ws.numel(), sp)], n, stream)
    segs = [(p[0][o[0]:o[1]], p[1][o[0]:o[1]], p[2][o[0]:o[1]]) for p, o in zip(packs, offs)]
    Rr = sum(sg[0].shape[0] for sg in segs)
    rq, rsf, roff, rrmap = sat.ep_recv_permute(segs, Eloc, align)
    rws = torch.empty(sat.fp8q_ep_recv_workspace_bytes(Rr, K, Eloc), dtype=torch.uint8, device=device)
    seg_args = [(a, b_, c_, a.shape[0]) for a, b_, c_ in segs]
    t_recv = time_steady([lambda: sat.fp8q_ep_recv_permute_fp8(seg_args, H, K, Eloc, align, rq, rsf, rq.shape[0], roff,
                                                               rrmap, rws, rws.numel(), sp)], n, stream)
    Rl = int(roff[-1].item())
    local_slots = int((rrmap >= 0).sum().item())
    out[f"ep_dispatch_pack rank 0 of 4: [{Tr}x7168] -> {sent0} rows"] = entry(
        Tr * (H + H // 128) + 4 * Tr * K + sent0 * (H + H // 128 + 4 * K) + 4 * (W + 1) + 4 * Tr * W, t_pack, 1)
    out[f"ep_recv_permute rank 0 of 4: {Rr} rows from 4 segments -> {Rl} rows"] = entry(
        Rr * (H + H // 128 + 4 * K) + local_slots * (H + H // 128) + (Rl - local_slots) * (H + H // 128)
        + 4 * (Eloc + 1) + 4 * Rr * K, t_recv, 1)
    del packs, segs, seg_args, rq, rsf, xq, xsf, xq0, xsf0, x0
    torch.cuda.empty_cache()
    # range stress
    d = synthetic.stress()
    x0 = synthetic.to_torch_bf16(d["x"]).to(device)
    R, C = x0.shape
    ne = R * C
    S = 2
    xs = copies(x0, S)
    q = [torch.empty((R, C), dtype=torch.uint8, device=device) for _ in range(S)]
    sf = [torch.empty((R, C // 128), dtype=torch.uint8, device=device) for _ in range(S)]
    qt = [torch.empty((C, R), dtype=torch.uint8, device=device) for _ in range(S)]
    sft = [torch.empty((C, R // 128), dtype=torch.uint8, device=device) for _ in range(S)]
    t_q = time_steady([lambda i=i: sat.fp8q_quantize_rowwise(xs[i], R, C, q[i], sf[i], sp) for i in range(S)], n,
                      stream)
    t_d = time_steady([lambda i=i: sat.fp8q_direct_transpose(q[i], sf[i], R, C, None, 1, qt[i], sft[i], sp)
                       for i in range(S)], n, stream)
    out["quantize_rowwise stress [65536x7168]"] = entry(3 * ne + ne // 128, t_q, S)
    out["direct_transpose stress [65536x7168]"] = entry(2 * ne + 2 * (ne // 128), t_d, S)
    del xs, q, sf, qt, sft, x0
    torch.cuda.empty_cache()
    status = sat.fp8q_last_device_status(sp)
    if status != 0:
        raise RuntimeError(f"device status {sat.STATUS.get(status)} in the workload measurements")
    return out


E2E_CHUNKS = 4  # row chunks of the end-to-end pipeline (4: 3.22 ms, 8: 3.40, 16: 3.66 ms per step in one run)


def e2e_pipelined(sat, x, x_host, q, sf, q_h, sf_h, qt_h, sft_h, reps, device):
    """Mean seconds per step of the end-to-end path (pinned host X in, pinned host Q, SF,
    Q^T, SF^T out) with the copies of neighbouring row chunks overlapping the kernels."""
    import ctypes

    import torch
    cudart = ctypes.CDLL("libcudart.so.12")
    memcpy2d = cudart.cudaMemcpy2DAsync
    memcpy2d.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_size_t,
                         ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p]
    memcpy2d.restype = ctypes.c_int
    d2h = 2  # cudaMemcpyDeviceToHost
    cr = ROWS // E2E_CHUNKS
    sh, sc, sd = torch.cuda.Stream(device), torch.cuda.Stream(device), torch.cuda.Stream(device)
    qt_c = [torch.empty((COLS, cr), dtype=torch.uint8, device=device) for _ in range(E2E_CHUNKS)]
    sft_c = [torch.empty((COLS, cr // 128), dtype=torch.uint8, device=device) for _ in range(E2E_CHUNKS)]
    main = torch.cuda.current_stream(device)

    def step():
        start = torch.cuda.Event()
        start.record(main)
        sh.wait_event(start)
        done = [torch.cuda.Event() for _ in range(E2E_CHUNKS)]
        for i in range(E2E_CHUNKS):
            r0, r1 = i * cr, (i + 1) * cr
            with torch.cuda.stream(sh):
                x[r0:r1].copy_(x_host[r0:r1], non_blocking=True)
            ready = torch.cuda.Event()
            ready.record(sh)
            sc.wait_event(ready)
            sat.fp8q_quantize_rowwise(x[r0:r1], cr, COLS, q[r0:r1], sf[r0:r1], sc.cuda_stream)
            sat.fp8q_direct_transpose(q[r0:r1], sf[r0:r1], cr, COLS, None, 1, qt_c[i], sft_c[i], sc.cuda_stream)
            computed = torch.cuda.Event()
            computed.record(sc)
            sd.wait_event(computed)
            with torch.cuda.stream(sd):
                q_h[r0:r1].copy_(q[r0:r1], non_blocking=True)
                sf_h[r0:r1].copy_(sf[r0:r1], non_blocking=True)
            rc = memcpy2d(qt_h.data_ptr() + r0, ROWS, qt_c[i].data_ptr(), cr, cr, COLS, d2h, sd.cuda_stream)
            rc |= memcpy2d(sft_h.data_ptr() + r0 // 128, ROWS // 128, sft_c[i].data_ptr(), cr // 128, cr // 128,
                           COLS, d2h, sd.cuda_stream)
            if rc:
                raise RuntimeError(f"pitched copy failed ({rc})")
            done[i].record(sd)
        main.wait_event(done[-1])

    for _ in range(2):
        step()
    torch.cuda.synchronize()
    pairs = []
    for _ in range(reps):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(main)
        step()
        b.record(main)
        pairs.append((a, b))
    torch.cuda.synchronize()
    return sum(a.elapsed_time(b) * 1e-3 for a, b in pairs) / len(pairs)


# ------------------------------------------------------------------ our arm
def run_ours(args, rank, world, local_rank):
    import numpy as np
    import torch
    import torch.distributed as dist

    import scaling_aware_transpose_b200 as sat
    from scaling_aware_transpose_b200 import synthetic

    torch.cuda.set_device(local_rank)
    device = torch.device("cuda", local_rank)
    sat.lib()  # fail loudly here if the library is missing
    x_bits = synthetic.dense(seed=rank)["x"]
    x_host = synthetic.to_torch_bf16(x_bits).pin_memory()
    xs = [x_host.to(device) for _ in range(SETS)]
    qs = [torch.empty((ROWS, COLS), dtype=torch.uint8, device=device) for _ in range(SETS)]
    sfs = [torch.empty((ROWS, COLS // 128), dtype=torch.uint8, device=device) for _ in range(SETS)]
    qts = [torch.empty((COLS, ROWS), dtype=torch.uint8, device=device) for _ in range(SETS)]
    sfts = [torch.empty((COLS, ROWS // 128), dtype=torch.uint8, device=device) for _ in range(SETS)]
    x, q, sf, qt, sft = xs[0], qs[0], sfs[0], qts[0], sfts[0]
    flush = torch.empty(FLUSH_BYTES, dtype=torch.uint8, device=device)
    stream = torch.cuda.current_stream(device)
    sp = stream.cuda_stream

    def quant(i=0):
        sat.fp8q_quantize_rowwise(xs[i], ROWS, COLS, qs[i], sfs[i], sp)

    def direct(i=0):
        sat.fp8q_direct_transpose(qs[i], sfs[i], ROWS, COLS, None, 1, qts[i], sfts[i], sp)

    def step(k, evs=None):
        a, b = k % SETS, (k - LAG) % SETS
        if evs:
            evs[0].record(stream)
        quant(a)
        if evs:
            evs[1].record(stream)
            evs[2].record(stream)
        direct(b)
        if evs:
            evs[3].record(stream)

    for i in range(SETS):
        quant(i)
    W = max(3, args.warmup)
    for k in range(W):
        step(k)
    torch.cuda.synchronize()
    if sat.fp8q_last_device_status(sp) != 0:
        raise RuntimeError("device status set during warm-up")

    K = args.steps
    t_start, t_end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    if world > 1:
        dist.barrier()
    torch.cuda.synchronize()
    torch.cuda._sleep(2_000_000)  # the host queues the first launches while the GPU waits
    with ClockSampler(local_rank) as clocks:
        t_start.record(stream)
        for k in range(K):
            step(W + k)
        t_end.record(stream)
        torch.cuda.synchronize()
    if world > 1:
        dist.barrier()
    total = t_start.elapsed_time(t_end) * 1e-3
    total_max = reduce_max(total, dist, device)
    # per-kernel durations: each kernel alone, the same number of back-to-back launches
    # over the same rotating sets in one event pair (an event between two kernels costs
    # the second one its launch overlap, about 3 us, so none is placed there)
    def steady(fn, n):
        fn(0)
        torch.cuda.synchronize()
        torch.cuda._sleep(2_000_000)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(stream)
        for i in range(n):
            fn(i % SETS)
        b.record(stream)
        torch.cuda.synchronize()
        return a.elapsed_time(b) * 1e-3 / n
    t_q_steady = reduce_max(steady(quant, K), dist, device)
    t_d_steady = reduce_max(steady(direct, K), dist, device)
    # the same two kernels with an event pair around each one (the previous convention)
    evs = [[torch.cuda.Event(enable_timing=True) for _ in range(4)] for _ in range(min(K, 50))]
    torch.cuda._sleep(2_000_000)
    for k, e in enumerate(evs):
        step(k, e)
    torch.cuda.synchronize()
    t_q_ev = statistics.median(e[0].elapsed_time(e[1]) * 1e-3 for e in evs)
    t_d_ev = statistics.median(e[2].elapsed_time(e[3]) * 1e-3 for e in evs)
    status = sat.fp8q_last_device_status(sp)
    if status != 0:
        raise RuntimeError(f"device status {sat.STATUS.get(status)} after the timed region")

    # every set's outputs are the same bytes: check set 0 against the others
    torch.cuda.synchronize()
    same_sets = all(torch.equal(qts[i], qt) and torch.equal(sfts[i], sft) and torch.equal(qs[i], q)
                    for i in range(1, SETS))

    # ---- extra, untimed-by-the-headline measurements
    # the earlier convention: a 256 MiB device write before each kernel, outside the
    # events (it leaves L2 full of dirty lines whose write-back the kernel then pays)
    t_q_dirty = time_on_stream(quant, min(K, 50), stream, lambda: flush.fill_(1))
    t_d_dirty = time_on_stream(direct, min(K, 50), stream, lambda: flush.fill_(2))
    # chained step: the transpose right after the quantize of the same set (Q still in L2),
    # back to back over the rotating sets
    t_chain = steady(lambda i: (quant(i), direct(i)), min(K, 100))
    # naive three-pass path, back to back over the same rotating sets (its workspace is
    # shared; each call moves about 590 MB)
    ws = torch.empty(sat.fp8q_naive_workspace_bytes(ROWS, COLS), dtype=torch.uint8, device=device)
    t_naive = steady(lambda i: sat.fp8q_naive_transpose(qs[i], sfs[i], ROWS, COLS, None, 1, qts[i], sfts[i], ws,
                                                        ws.numel(), sp), min(K, 50))
    for i in range(SETS):  # restore the sets' outputs for the checks below
        direct(i)

    # same two kernels after a flush that leaves no dirty lines (write, then read the
    # flush buffer): the kernel does not pay for writing back data it never touched
    def clean_flush():
        flush.fill_(5)
        flush.view(torch.int32).max()
    t_q_clean = time_on_stream(quant, min(K, 50), stream, clean_flush)
    t_d_clean = time_on_stream(direct, min(K, 50), stream, clean_flush)

    # single-pass quantizer: the same four outputs from one read of X (byte-identical to
    # the two-kernel step); also with packed UE8M0 scales and the zero-tile option.  Back
    # to back over the rotating X sets, each with its own outputs.
    rc_out = [(torch.empty_like(q), torch.empty_like(sf), torch.empty_like(qt), torch.empty_like(sft))
              for _ in range(SETS)]
    pk_sf = torch.empty(sat.packed_sf_shape(ROWS, COLS), dtype=torch.int32, device=device)
    pk_sft = torch.empty(sat.packed_sf_shape(COLS, ROWS), dtype=torch.int32, device=device)
    rowcol = lambda i: sat.fp8q_quantize_rowwise_colwise(xs[i], ROWS, COLS, 0, *rc_out[i], sp)
    rowcol_pk = lambda i: sat.fp8q_quantize_rowwise_colwise(xs[i], ROWS, COLS, sat.ZERO_TILE_MIN_SCALE |
                                                            sat.SF_PACKED_UE8M0, rc_out[i][0], pk_sf, rc_out[i][2],
                                                            pk_sft, sp)
    t_rc = steady(rowcol, min(K, 100))
    t_rc_pk = steady(rowcol_pk, min(K, 100))
    t_rc_dirty = time_on_stream(lambda: rowcol(0), min(K, 50) + 3, stream, lambda: flush.fill_(10))
    # MX granularity: 1x32 tiles and 32x32 transpose blocks on the same X, back to back
    # over the rotating sets
    mx = [(torch.empty_like(q), torch.empty((ROWS, COLS // 32), dtype=torch.uint8, device=device),
           torch.empty_like(qt), torch.empty((COLS, ROWS // 32), dtype=torch.uint8, device=device))
          for _ in range(SETS)]
    t_mxq = steady(lambda i: sat.fp8q_quantize_rowwise_mx32(xs[i], ROWS, COLS, mx[i][0], mx[i][1], sp), min(K, 100))
    t_mxd = steady(lambda i: sat.fp8q_direct_transpose_mx32(mx[i][0], mx[i][1], ROWS, COLS, mx[i][2], mx[i][3], sp),
                   min(K, 100))
    del mx
    rowcol(0)
    torch.cuda.synchronize()
    rc_q, rc_sf, rc_qt, rc_sft = rc_out[0]
    same_rc = all(torch.equal(a_, b_) for a_, b_ in ((rc_q, q), (rc_sf, sf), (rc_qt, qt), (rc_sft, sft)))

    # ---- end to end through the C ABI from pinned host buffers
    q_h = torch.empty_like(q, device="cpu").pin_memory()
    sf_h = torch.empty_like(sf, device="cpu").pin_memory()
    qt_h = torch.empty_like(qt, device="cpu").pin_memory()
    sft_h = torch.empty_like(sft, device="cpu").pin_memory()
    e2e = []
    for i in range(min(K, 20) + 2):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(stream)
        x.copy_(x_host, non_blocking=True)
        quant()
        direct()
        q_h.copy_(q, non_blocking=True)
        sf_h.copy_(sf, non_blocking=True)
        qt_h.copy_(qt, non_blocking=True)
        sft_h.copy_(sft, non_blocking=True)
        b.record(stream)
        if i >= 2:
            e2e.append((a, b))
    torch.cuda.synchronize()
    t_e2e_serial = reduce_max(sum(a.elapsed_time(b) * 1e-3 for a, b in e2e) / len(e2e), dist, device)
    # the same calls, pipelined over 2048-row chunks on three streams: the H2D copy of chunk
    # i+1, the two kernels on chunk i and the D2H copies of chunk i-1 overlap (the host
    # link is full duplex); each chunk's transposed block lands in the dense host Q^T and
    # SF^T through a pitched copy
    t_e2e = reduce_max(e2e_pipelined(sat, x, x_host, q, sf, q_h, sf_h, qt_h, sft_h, min(K, 20), device), dist, device)
    ok_e2e = bool(np.array_equal(qt_h.numpy(), qt.cpu().numpy()) and np.array_equal(sft_h.numpy(), sft.cpu().numpy())
                  and np.array_equal(q_h.numpy(), q.cpu().numpy()) and np.array_equal(sf_h.numpy(), sf.cpu().numpy()))

    if rank != 0:
        return None
    peak, peak_kind = measured_peak_gbs()
    avg_q, avg_d = t_q_steady, t_d_steady
    dominant = "quantize" if avg_q >= avg_d else "direct"
    rf = roofline(BYTES_QUANT if dominant == "quantize" else BYTES_DIRECT, max(avg_q, avg_d), peak, peak_kind,
                  profiled_traffic(dominant))
    rf["kernel"] = {"quantize": "fp8q_quantize_rowwise (quantize_tiles_kernel)",
                    "direct": "fp8q_direct_transpose (direct_transpose_kernel)"}[dominant]
    value = world * K * BYTES_STEP / total_max / 1e9
    line = {
        "metric": METRIC, "value": round(value, 1), "unit": "GB/s", "n_gpus": world, "steps": K, "warmup": W,
        "ms_per_step": round(total_max / K * 1e3, 5), "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "u8", "data": "synthetic",
        "config": {"workload": WORKLOAD, "path": "fp8q_quantize_rowwise -> fp8q_direct_transpose",
                   "bytes_per_step": BYTES_STEP,
                   "l2": f"inputs larger than L2: {SETS} rotating buffer sets ({SETS * BYTES_STEP // 10**6} MB); "
                         f"step k quantizes set k and transposes set k-{LAG}, no flush",
                   "seed": "rank", "parallelism": f"replicas x{world} (no collective)"},
        "roofline": rf,
        "kernels": {
            "quantize_rowwise": {"us": round(avg_q * 1e6, 2), "GB/s": round(BYTES_QUANT / avg_q / 1e9, 1),
                                 "frac_of_peak": round(BYTES_QUANT / avg_q / 1e9 / peak, 4),
                                 "frac_of_8000": round(BYTES_QUANT / avg_q / 1e9 / 8000, 4),
                                 "traffic": profiled_traffic("quantize")},
            "direct_transpose": {"us": round(avg_d * 1e6, 2), "GB/s": round(BYTES_DIRECT / avg_d / 1e9, 1),
                                 "frac_of_peak": round(BYTES_DIRECT / avg_d / 1e9 / peak, 4),
                                 "frac_of_8000": round(BYTES_DIRECT / avg_d / 1e9 / 8000, 4),
                                 "traffic": profiled_traffic("direct")},
            "per_kernel_timing": f"{K} back-to-back launches of one kernel over the {SETS} rotating sets, "
                                 "one event pair (quantize_rowwise, direct_transpose above)",
            "step_sum_vs_loop": round((avg_q + avg_d) / (total / K), 4),
            "event_pair_per_kernel": {"quantize_us": round(t_q_ev * 1e6, 2), "direct_us": round(t_d_ev * 1e6, 2),
                                      "how": "the headline loop with an event pair around each kernel"},
            "dirty_l2_flush": {"quantize_us": round(t_q_dirty * 1e6, 2),
                               "quantize_GB/s": round(BYTES_QUANT / t_q_dirty / 1e9, 1),
                               "direct_us": round(t_d_dirty * 1e6, 2),
                               "direct_GB/s": round(BYTES_DIRECT / t_d_dirty / 1e9, 1)},
            "rotating_sets_outputs_identical": same_sets,
            "naive_transpose_3pass": {"us": round(t_naive * 1e6, 2),
                                      "GB/s_of_direct_bytes": round(BYTES_DIRECT / t_naive / 1e9, 1),
                                      "direct_speedup": round(t_naive / avg_d, 2)},
            "chained_step": {"us": round(t_chain * 1e6, 2), "GB/s": round(BYTES_STEP / t_chain / 1e9, 1),
                             "how": "quantize then transpose of the same set (Q read back from L2), back to back "
                                    "over the rotating sets"},
            "quantize_rowwise_colwise_single_pass": {
                "us": round(t_rc * 1e6, 2), "bytes": BYTES_ROWCOL, "GB/s": round(BYTES_ROWCOL / t_rc / 1e9, 1),
                "frac_of_peak": round(BYTES_ROWCOL / t_rc / 1e9 / peak, 4),
                "frac_of_8000": round(BYTES_ROWCOL / t_rc / 1e9 / 8000, 4),
                "dirty_l2_flush_us": round(t_rc_dirty * 1e6, 2),
                "packed_ue8m0_zero_tile_us": round(t_rc_pk * 1e6, 2),
                "vs_two_kernel_step": round((avg_q + avg_d) / t_rc, 3),
                "outputs_equal_two_kernel_step": same_rc,
                "traffic": profiled_traffic("rowwise_colwise")},
            "mx32": {"quantize_us": round(t_mxq * 1e6, 2), "quantize_GB/s": round(BYTES_MX_QUANT / t_mxq / 1e9, 1),
                     "quantize_frac_of_peak": round(BYTES_MX_QUANT / t_mxq / 1e9 / peak, 4),
                     "direct_us": round(t_mxd * 1e6, 2), "direct_GB/s": round(BYTES_MX_DIRECT / t_mxd / 1e9, 1),
                     "direct_frac_of_peak": round(BYTES_MX_DIRECT / t_mxd / 1e9 / peak, 4)},
            "clean_l2_flush": {"quantize_us": round(t_q_clean * 1e6, 2),
                               "quantize_GB/s": round(BYTES_QUANT / t_q_clean / 1e9, 1),
                               "direct_us": round(t_d_clean * 1e6, 2),
                               "direct_GB/s": round(BYTES_DIRECT / t_d_clean / 1e9, 1)},
        },
        "gpu_launches": 2 * K,
        "e2e": {"value": round(BYTES_STEP / t_e2e / 1e9, 2), "unit": "GB/s", "h2d_bytes_per_step": 2 * N_ELEM,
                "d2h_bytes_per_step": 2 * N_ELEM + 2 * (N_ELEM // 128), "ms_per_step": round(t_e2e * 1e3, 3),
                "path": f"{E2E_CHUNKS} row chunks, H2D / kernels / D2H on three streams",
                "serial_ms_per_step": round(t_e2e_serial * 1e3, 3), "result_matches_device": ok_e2e},
        "clocks": clocks.summary(),
    }
    if not args.no_extras:
        del flush
        torch.cuda.empty_cache()
        line["workloads"] = measure_workloads(min(K, 20), device, stream, peak)
    if world == 1 and not args.no_cpu_baseline:
        line["cpu_baseline"] = cpu_baseline(x_bits, budget_s=args.cpu_budget)
    return line


# ------------------------------------------------------------------ reference arm
def run_reference(args):
    import oracle
    from scaling_aware_transpose_b200 import synthetic
    x_bits = synthetic.dense(seed=0)["x"][: args.ref_rows]
    rows = x_bits.shape[0]
    W = max(3, args.warmup)
    for _ in range(W):
        q, sf = oracle.quantize_rowwise(x_bits)
        oracle.direct_transpose(q, sf)
    t0 = time.perf_counter()
    for _ in range(args.steps):
        q, sf = oracle.quantize_rowwise(x_bits)
        oracle.direct_transpose(q, sf)
    total = time.perf_counter() - t0
    step_bytes = BYTES_STEP * rows // ROWS
    value = args.steps * step_bytes / total / 1e9
    sample = f"{rows}x{COLS} rows of the workload per step (quantize + direct transpose)"
    return {
        "impl": "reference", "metric": METRIC, "value": round(value, 3), "unit": "GB/s", "n_gpus": 1,
        "steps": args.steps, "warmup": W, "ms_per_step": round(total / args.steps * 1e3, 3),
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "u8", "data": "synthetic",
        "config": {"workload": WORKLOAD, "path": "CPU oracle: quantize_rowwise -> direct_transpose",
                   "bytes_per_step": step_bytes, "sample": sample},
        "cpu_baseline": {"value": round(value, 3), "unit": "GB/s", "cores": oracle.num_threads(),
                         "kind": "oracle", "sample": sample},
        "e2e": {"value": round(value, 3), "unit": "GB/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
        "gpu_launches": 0,
    }


# ------------------------------------------------------------------ ncu driver
def run_profile(args):
    """Launches only one kernel, --warmup + --steps times back to back on the dense workload
    (no flush, no timing): the command line that the committed ncu summaries capture."""
    import torch

    import scaling_aware_transpose_b200 as sat
    from scaling_aware_transpose_b200 import synthetic
    torch.cuda.set_device(0)
    if args.profile in ("quantize", "direct", "naive", "rowwise_colwise"):
        x = synthetic.to_torch_bf16(synthetic.dense(seed=0)["x"]).cuda()
        q, sf = sat.quantize_rowwise(x)
        qt, sft = sat.direct_transpose(q, sf)
        ws = torch.empty(sat.fp8q_naive_workspace_bytes(ROWS, COLS), dtype=torch.uint8, device="cuda")
        calls = {
            "quantize": lambda: sat.fp8q_quantize_rowwise(x, ROWS, COLS, q, sf),
            "direct": lambda: sat.fp8q_direct_transpose(q, sf, ROWS, COLS, None, 1, qt, sft),
            "naive": lambda: sat.fp8q_naive_transpose(q, sf, ROWS, COLS, None, 1, qt, sft, ws, ws.numel()),
            "rowwise_colwise": lambda: sat.fp8q_quantize_rowwise_colwise(x, ROWS, COLS, 0, q, sf, qt, sft),
        }
    elif args.profile in ("mx32", "mx32_quantize"):
        x = synthetic.to_torch_bf16(synthetic.dense(seed=0)["x"]).cuda()
        mq, msf = sat.quantize_rowwise_mx32(x)
        mqt, msft = sat.direct_transpose_mx32(mq, msf)
        calls = {"mx32": lambda: sat.fp8q_direct_transpose_mx32(mq, msf, ROWS, COLS, mqt, msft),
                 "mx32_quantize": lambda: sat.fp8q_quantize_rowwise_mx32(x, ROWS, COLS, mq, msf)}
    elif args.profile == "direct_stress":
        xs_ = synthetic.to_torch_bf16(synthetic.stress(seed=0)["x"]).cuda()
        q, sf = sat.quantize_rowwise(xs_)
        del xs_
        qt, sft = sat.direct_transpose(q, sf)
        R, H = q.shape
        calls = {"direct_stress": lambda: sat.fp8q_direct_transpose(q, sf, R, H, None, 1, qt, sft)}
    elif args.profile == "direct_grouped":
        d = synthetic.moe()
        x = synthetic.to_torch_bf16(d["x"]).cuda()
        idx = torch.from_numpy(d["topk_idx"]).cuda()
        pq, psf, off, _ = sat.permute_pad_quant(x, idx, d["num_experts"], 128)
        del x
        qt = torch.empty(pq.numel(), dtype=torch.uint8, device="cuda")
        sft = torch.empty(psf.numel(), dtype=torch.uint8, device="cuda")
        R, H = pq.shape
        calls = {"direct_grouped": lambda: sat.fp8q_direct_transpose(pq, psf, R, H, off, d["num_experts"], qt, sft)}
    elif args.profile in ("ep_pack", "ep_recv"):
        d = synthetic.moe()
        x = synthetic.to_torch_bf16(d["x"]).cuda()
        idx = torch.from_numpy(d["topk_idx"]).cuda()
        xq, xsf = sat.quantize_rowwise(x)
        del x
        W, Tr = 4, xq.shape[0] // 4
        Eloc = d["num_experts"] // W
        packs = [sat.ep_dispatch_pack(xq[r * Tr:(r + 1) * Tr], xsf[r * Tr:(r + 1) * Tr], idx[r * Tr:(r + 1) * Tr],
                                      W, Eloc) for r in range(W)]
        offs = [p[3].tolist() for p in packs]
        segs = [(p[0][o[0]:o[1]], p[1][o[0]:o[1]], p[2][o[0]:o[1]]) for p, o in zip(packs, offs)]
        calls = {"ep_pack": lambda: sat.ep_dispatch_pack(xq[:Tr], xsf[:Tr], idx[:Tr], W, Eloc),
                 "ep_recv": lambda: sat.ep_recv_permute(segs, Eloc, 128)}
    elif args.profile == "permute_fp8":
        d = synthetic.moe()
        x = synthetic.to_torch_bf16(d["x"]).cuda()
        idx = torch.from_numpy(d["topk_idx"]).cuda()
        xq, xsf = sat.quantize_rowwise(x)
        calls = {"permute_fp8": lambda: sat.permute_pad_fp8(xq, xsf, idx, d["num_experts"], 128)}
    elif args.profile == "swiglu":
        d = synthetic.swiglu()
        g, u = synthetic.to_torch_bf16(d["gate"]).cuda(), synthetic.to_torch_bf16(d["up"]).cuda()
        R, C = g.shape
        q = torch.empty((R, C), dtype=torch.uint8, device="cuda")
        sf = torch.empty((R, C // 128), dtype=torch.uint8, device="cuda")
        qt = torch.empty((C, R), dtype=torch.uint8, device="cuda")
        sft = torch.empty((C, R // 128), dtype=torch.uint8, device="cuda")
        calls = {"swiglu": lambda: sat.fp8q_swiglu_quant(g, u, R, C, q, sf, qt, sft)}
    elif args.profile in ("unpermute", "unpermute_fp8"):
        d = synthetic.moe()
        x = synthetic.to_torch_bf16(d["x"]).cuda()
        idx = torch.from_numpy(d["topk_idx"]).cuda()
        K = idx.shape[1]
        pq, psf, off, rmap = sat.permute_pad_quant(x, idx, d["num_experts"], 128)
        R = int(off[-1].item())
        c = synthetic.moe_combine(rows=R, topk=K)
        y = synthetic.to_torch_bf16(c["y"]).cuda()
        wts = torch.from_numpy(c["weights"]).cuda()
        calls = {"unpermute": lambda: sat.unpermute_unpad(y, rmap, K, wts),
                 "unpermute_fp8": lambda: sat.unpermute_unpad(pq, rmap, K, None, psf)}
    elif args.profile in ("permute_e512", "permute_e4096"):
        # routings too wide for the fused rank kernel: the chunk scan (a CTA per 32 experts)
        # and the eight-warp rank, at 512 and at the 4096-expert maximum
        E = 512 if args.profile == "permute_e512" else 4096
        d = synthetic.moe(num_experts=E)
        x = synthetic.to_torch_bf16(d["x"]).cuda()
        idx = torch.from_numpy(d["topk_idx"]).cuda()
        calls = {args.profile: lambda: sat.permute_pad_quant(x, idx, E, 16)}
    elif args.profile == "unpermute_fp8_k":
        # FP8 combine with hidden % 1024 != 0: the per-top-k kernel instead of the ring
        d = synthetic.moe(hidden=7040)
        x = synthetic.to_torch_bf16(d["x"]).cuda()
        idx = torch.from_numpy(d["topk_idx"]).cuda()
        K = idx.shape[1]
        pq, psf, off, rmap = sat.permute_pad_quant(x, idx, d["num_experts"], 128)
        del x
        calls = {"unpermute_fp8_k": lambda: sat.unpermute_unpad(pq, rmap, K, None, psf)}
    elif args.profile == "router_rows":
        d = synthetic.moe()
        idx = torch.from_numpy(d["topk_idx"]).cuda()
        x = torch.zeros((idx.shape[0], 128), dtype=torch.bfloat16, device="cuda")
        _, _, off, rmap = sat.permute_pad_quant(x, idx, d["num_experts"], 128)
        w, rows = torch.rand(idx.shape, device="cuda"), int(off[-1])
        calls = {"router_rows": lambda: sat.permute_row_weights(w, rmap, rows)}
    elif args.profile.startswith("router"):
        # forward and backward of a training step: the MoE workload's 32 experts, or 256 with
        # sigmoid scores and a selection bias
        wide = args.profile == "router_wide"
        g = torch.Generator(device="cuda").manual_seed(0)
        E, K = (256, 8) if wide else (32, 8)
        logits = torch.randn((16384, E), generator=g, device="cuda") * 1.2
        logits = logits if wide else logits.to(torch.bfloat16)
        opt = {"sigmoid": wide, "loss_coef": 0.01}
        bias = torch.randn(E, generator=g, device="cuda") * 0.1 if wide else None

        def router_step():
            idx, w, counts, _, loss = sat.router_topk(logits, K, bias=bias, **opt)
            sat.router_topk_bwd(logits, idx, w, counts=counts, grad_loss=loss, **opt)
        calls = {args.profile: router_step}
    elif args.profile in ("swiglu_stash", "swiglu_bwd", "swiglu_bwd_quant"):
        d = synthetic.swiglu()
        g, u = synthetic.to_torch_bf16(d["gate"]).cuda(), synthetic.to_torch_bf16(d["up"]).cuda()
        w = torch.linspace(0.0, 1.0, g.shape[0], device="cuda")
        stash = sat.swiglu_quant_stash(g, u, row_weights=w)[2:]
        calls = {"swiglu_stash": lambda: sat.swiglu_quant_stash(g, u, row_weights=w),
                 "swiglu_bwd": lambda: sat.swiglu_bwd(*stash, u, row_weights=w),
                 "swiglu_bwd_quant": lambda: sat.swiglu_bwd_quant(*stash, u, row_weights=w)}
    elif args.profile in ("mxfp4_quantize", "mxfp4_matmul", "mxfp4_token"):
        x = synthetic.to_torch_bf16(synthetic.dense(seed=0)["x"]).cuda()
        a, b = sat.quantize_rowwise_mxfp4(x), sat.quantize_rowwise_mxfp4(x[:4096].contiguous())
        one = sat.quantize_rowwise_mxfp4(x[:1].contiguous())
        calls = {"mxfp4_quantize": lambda: sat.quantize_rowwise_mxfp4(x),
                 "mxfp4_matmul": lambda: sat.matmul_mxfp4(*a, *b),
                 "mxfp4_token": lambda: sat.matmul_mxfp4(*one, *b)}
    elif args.profile in ("mxfp4_permute", "mxfp4_permute_few", "mxfp4_experts"):
        d = synthetic.moe(tokens=4096)
        x = synthetic.to_torch_bf16(d["x"]).cuda()
        idx, E = torch.from_numpy(d["topk_idx"]).cuda(), d["num_experts"]
        q, sf, off, _ = sat.permute_pad_mxfp4(x, idx, E, 128)
        w = sat.quantize_rowwise_mxfp4(torch.randn((E * 2048, x.shape[1]), device="cuda").to(torch.bfloat16))
        out = torch.zeros((q.shape[0], 2048), dtype=torch.bfloat16, device="cuda")
        calls = {"mxfp4_permute": lambda: sat.permute_pad_mxfp4(x, idx, E, 128),
                 "mxfp4_permute_few": lambda: sat.permute_pad_mxfp4(x[:64], idx[:64], E, 128),
                 "mxfp4_experts": lambda: sat.matmul_mxfp4(q, sf, *w, group_offsets=off, out=out)}
    else:  # permute
        d = synthetic.moe()
        x = synthetic.to_torch_bf16(d["x"]).cuda()
        idx = torch.from_numpy(d["topk_idx"]).cuda()
        calls = {"permute": lambda: sat.permute_pad_quant(x, idx, d["num_experts"], 128)}
    torch.cuda.synchronize()
    for _ in range(args.warmup + args.steps):
        calls[args.profile]()
    torch.cuda.synchronize()
    st = sat.fp8q_last_device_status()
    print(json.dumps({"profile": args.profile, "launches": args.warmup + args.steps, "status": st}))
    return 0 if st == 0 else 1


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--impl", choices=["ours", "reference"], default="ours")
    ap.add_argument("--no-cpu-baseline", action="store_true", help="skip the oracle timing leg")
    ap.add_argument("--no-extras", action="store_true", help="skip the SwiGLU / MoE / stress workload timings")
    ap.add_argument("--cpu-budget", type=float, default=10.0, help="seconds of oracle time for cpu_baseline")
    ap.add_argument("--ref-rows", type=int, default=1024, help="rows of the workload per reference step")
    ap.add_argument("--profile", choices=["quantize", "direct", "naive", "swiglu", "permute", "rowwise_colwise",
                                          "unpermute", "unpermute_fp8", "mx32", "permute_fp8", "mx32_quantize",
                                          "direct_grouped", "ep_pack", "ep_recv", "direct_stress", "permute_e512",
                                          "permute_e4096", "unpermute_fp8_k", "router", "router_wide", "router_rows",
                                          "mxfp4_permute_few", "swiglu_stash", "swiglu_bwd", "swiglu_bwd_quant", "mxfp4_quantize",
                                          "mxfp4_permute", "mxfp4_matmul", "mxfp4_token", "mxfp4_experts"],
                    default=None,
                    help="launch only this kernel (for ncu captures); prints no bench line")
    args = ap.parse_args(argv)
    if args.profile:
        return run_profile(args)

    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    local_rank = int(os.environ.get("LOCAL_RANK", "0"))

    if args.impl == "reference":
        if rank == 0:
            print(json.dumps(run_reference(args)), flush=True)
        return 0

    import datetime

    import torch.distributed as dist
    if world > 1:
        import torch
        torch.cuda.set_device(local_rank)
        dist.init_process_group("nccl", timeout=datetime.timedelta(seconds=120),
                                device_id=torch.device("cuda", local_rank))
    try:
        line = run_ours(args, rank, world, local_rank)
    finally:
        if world > 1 and dist.is_initialized():
            dist.destroy_process_group()
    if rank == 0 and line is not None:
        print(json.dumps(line), flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
