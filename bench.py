"""Benchmark of the SAFE-DiT attention hot path on B200.

One step = one pass of the whole hot path for one DiT block at the
2560^2-equivalent workload (B=2, H=24, d=96, N=25600, M=128, |S|=0.25N):
  mask classify (the all-valid [B,1,N,N] bool image mask) -> dense mask-free
  self-attention (anchor) -> padded cross-attention -> PCSP scores + top-k ->
  context-cache scatter -> SRSU self-attention -> SRSU cross-attention.
Inputs (236 MB per image tensor) exceed the 126 MB L2, so no flush is needed
between steps.

    python bench.py [--gpus N] [--steps K] [--warmup W] [--impl ours|reference]
    python bench.py --only KERNEL [--workload W] [--launches L]   (one kernel, for profilers)
    python bench.py --operators [both]                            (the row-wise operators' table)

Prints one JSON line (rank 0). `value` is attention TFLOP/s of the step:
algorithmic FLOPs of dense self-attention (4 B H N^2 d) plus SRSU
(4 B H k N d) plus both cross-attentions (4 H d * rows * sum_b len_b) over
the measured step time, summed over ranks (each rank runs its own replica).
"""

from __future__ import annotations

import argparse
import json
import math
import os
import statistics
import subprocess
import sys
import time

import numpy as np
import torch

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

from mask_free_b200 import synth  # noqa: E402

METRIC = "attention TFLOP/s + ms/call (dense, SRSU) at N=4096/25600; % bf16 tensor peak"
WORKLOAD = "2560^2-equivalent SRSU step: B=2, H=24, d=96, N=25600, M=128 (len U[8,128]), k=6400 (0.25N)"


def max_over_ranks(ms: float, dist=None, device=None) -> float:
    """Largest per-rank device time (ms): the job is as slow as its slowest
    rank. Identity for a single process."""
    if dist is None or not dist.is_initialized() or dist.get_world_size() == 1:
        return ms
    t = torch.tensor([ms], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def job_throughput(world: int, flops_per_rank_step: float, ms_per_step: float) -> float:
    """Whole-job TFLOP/s: every rank runs its own replica of the step (weak
    scaling), so the job does world x the work of one rank per step time."""
    return world * flops_per_rank_step / (ms_per_step * 1e-3) / 1e12


def peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        j = json.load(open(p))
        return {"hbm": j["hbm_gbs"], "bf16": j["bf16_tflops"], "bf16_sustained": j["bf16_tflops_sustained"],
                "source": "measured"}
    return {"hbm": 6650.0, "bf16": 1590.0, "bf16_sustained": 1400.0, "source": "fallback"}


def flash_source_sha():
    import hashlib
    h = hashlib.sha256()
    for f in ("flash_attn.cuh", "sm100.cuh"):
        h.update(open(os.path.join(ROOT, "mask_free_b200", "csrc", f), "rb").read())
    return h.hexdigest()[:16]


def stored_traffic():
    """DRAM bytes per dense launch at this workload from an ncu capture of the
    same kernel source (profiles/flash_traffic.json), else None."""
    p = os.path.join(ROOT, "profiles", "flash_traffic.json")
    if not os.path.exists(p):
        return None
    j = json.load(open(p))
    if j.get("source_sha") != flash_source_sha():
        return None
    return j.get("dram_bytes_per_launch")


def flops(shape, lens_sum, k):
    B, N, H, d = shape.B, shape.N, shape.H, shape.d
    dense = 4.0 * B * H * N * N * d
    srsu = 4.0 * B * H * k * N * d
    cross = 4.0 * H * d * N * lens_sum
    cross_s = 4.0 * H * d * k * lens_sum
    return dense, srsu, cross, cross_s


class ClockSampler:
    """nvidia-smi clock / throttle sampling during the timed region."""

    FIELDS = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, device_index: int, log_dir: str = None):
        import tempfile
        self.dev = device_index
        self.proc = None
        self.path = os.path.join(log_dir or tempfile.gettempdir(), f"clocks_rank{device_index}.csv")

    def __enter__(self):
        try:
            os.makedirs(os.path.dirname(self.path), exist_ok=True)
            self.f = open(self.path, "w")
            self.proc = subprocess.Popen(["nvidia-smi", f"--id={self.dev}", f"--query-gpu={self.FIELDS}",
                                          "--format=csv,noheader,nounits", "-lms", "100"], stdout=self.f,
                                         stderr=subprocess.DEVNULL)
        except Exception:
            self.proc = None
        return self

    def __exit__(self, *a):
        if self.proc is not None:
            self.proc.terminate()
            try:
                self.proc.wait(timeout=5)
            except Exception:
                self.proc.kill()
            self.f.close()

    def summary(self):
        if self.proc is None or not os.path.exists(self.path):
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["nvidia-smi unavailable"]}
        sm, smax, reasons = [], None, set()
        names = ["active", "hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for line in open(self.path):
            parts = [x.strip() for x in line.split(",")]
            if len(parts) < 9:
                continue
            try:
                sm.append(float(parts[1]))
                smax = float(parts[2])
            except ValueError:
                continue
            for name, val in zip(names[1:], parts[5:9]):
                if val.lower() == "active":
                    reasons.add(name)
        return {"sm_mhz": statistics.median(sm) if sm else None, "sm_max_mhz": smax,
                "reasons": sorted(reasons), "samples": len(sm)}


def make_step_inputs(workload: str, dev):
    s = synth.WORKLOADS[workload]
    g = torch.Generator(device=dev).manual_seed(1000 * s.seed_id)

    def bf(rows):
        return torch.randn((s.B, rows, s.H, s.d), generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)

    lens = synth.uniform_lengths(s.B, s.len_lo, s.len_hi, synth.seed_for(s.seed_id, synth.T_LEN))
    inp = {"Q": bf(s.N), "K": bf(s.N), "V": bf(s.N), "Ky": bf(s.M), "Vy": bf(s.M),
           "valid_len": lens.to(dev), "w": synth.content_weights(lens, s.M, synth.seed_for(s.seed_id, synth.T_W)).to(dev)}
    inp["Kc"] = (inp["K"].float() + 0.05 * torch.randn(inp["K"].shape, generator=g, device=dev)).to(torch.bfloat16)
    inp["Vc"] = (inp["V"].float() + 0.05 * torch.randn(inp["V"].shape, generator=g, device=dev)).to(torch.bfloat16)
    inp["mask"] = torch.ones((s.B, 1, s.N, s.N), dtype=torch.bool, device=dev)
    return s, inp, int(lens.sum())


class Step:
    """One pass of the hot path; all buffers preallocated."""

    def __init__(self, s, inp, dev):
        from mask_free_b200 import ops
        self.ops, self.s, self.inp = ops, s, inp
        B, N, H, d, M, k = s.B, s.N, s.H, s.d, s.M, s.k
        self.O = torch.empty((B, N, H, d), dtype=torch.bfloat16, device=dev)
        self.Ox = torch.empty_like(self.O)
        self.Os = torch.empty((B, k, H, d), dtype=torch.bfloat16, device=dev)
        self.Osx = torch.empty_like(self.Os)
        self.scores = torch.empty((B, N), dtype=torch.float32, device=dev)
        self.S = torch.empty((B, k), dtype=torch.int32, device=dev)
        self.C = torch.empty((B, N - k), dtype=torch.int32, device=dev)
        self.ws = torch.empty(ops.pcsp_workspace_bytes(B, N, H), dtype=torch.uint8, device=dev)
        self.cls = torch.empty(3, dtype=torch.int64, device=dev)
        self.ws_self = torch.empty(max(256, ops.attn_workspace_bytes(B, N, N, H, d)), dtype=torch.uint8, device=dev)
        self.ws_srsu = torch.empty(max(256, ops.srsu_workspace_bytes(B, k, N, H, d)), dtype=torch.uint8, device=dev)
        self.Kc, self.Vc = inp["Kc"].clone(), inp["Vc"].clone()
        self.events = []
        # library kernels per step: classify 3 (init, rows, verdict); dense 1
        # (+1 merge when the last wave is split along the keys); cross with
        # PCSP 3 (cross, head sum, top-k); scatter 1; SRSU 2 (query-row copy,
        # attention; +1 merge); cross on S 1
        self.launches = 3 + 1 + (ops.attn_workspace_bytes(B, N, N, H, d) > 0) + 3 + 1 + 2 + \
            (ops.attn_workspace_bytes(B, k, N, H, d) > 0) + 1

    def __call__(self, timed=False):
        o, i = self.ops, self.inp
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(4)] if timed else None
        if timed:
            self.events.append(ev)
        o.mask_classify(i["mask"], sync=False, result=self.cls)
        if timed:
            ev[0].record()
        o.attn_self(i["Q"], i["K"], i["V"], out=self.O, ws=self.ws_self)
        if timed:
            ev[1].record()
        # cross-attention and, from the same probabilities (Eq. (9)), the PCSP
        # scores and the top-k split
        o.attn_cross_pcsp(i["Q"], i["Ky"], i["Vy"], i["valid_len"], i["w"], out=self.Ox, scores=self.scores,
                          k=self.s.k, S=self.S, C=self.C, ws=self.ws)
        o.ctx_cache_scatter(i["K"], i["V"], self.S, self.Kc, self.Vc, src_compact=False)
        if timed:
            ev[2].record()
        o.srsu_attn(i["Q"], self.S, self.Kc, self.Vc, out=self.Os, ws=self.ws_srsu)
        if timed:
            ev[3].record()
        o.attn_cross(i["Q"], i["Ky"], i["Vy"], i["valid_len"], q_idx=self.S, out=self.Osx)

    def launch_times(self):
        torch.cuda.synchronize()
        dense = [e[0].elapsed_time(e[1]) for e in self.events]
        srsu = [e[2].elapsed_time(e[3]) for e in self.events]
        return dense, srsu


def time_kernel(fn, reps=20, warm=3):
    """Device ms per call: `reps` back-to-back calls captured in a CUDA graph
    and replayed, so that neither the Python binding nor the host half of the
    C ABI (tensor-map encoding, launch) is timed; batch timing of eager calls
    if the calls cannot be captured."""
    for _ in range(warm):
        fn()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    try:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(reps):
                fn()
        g.replay()
        torch.cuda.synchronize()
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        del g
        return a.elapsed_time(b) / reps
    except RuntimeError:
        torch.cuda.synchronize()
    a.record()
    for _ in range(reps):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / reps


_FLUSH = {}


def time_flushed(fn, reps=20, warm=3):
    """Median device ms of one call over `reps` calls, each after a 256 MB
    write that evicts the 126 MB L2 (the call is a CUDA graph replayed
    between CUDA events; the flush in front of it covers the host's enqueue
    time, so the events bracket device work only). For kernels whose inputs
    fit in L2 or come close."""
    dev = torch.cuda.current_device()
    if dev not in _FLUSH:
        _FLUSH[dev] = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    buf = _FLUSH[dev]
    for _ in range(warm):
        fn()
    torch.cuda.synchronize()
    try:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        run = g.replay
    except RuntimeError:
        torch.cuda.synchronize()
        g, run = None, fn
    ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for _ in range(reps)]
    for a, b in ev:
        buf.zero_()
        a.record()
        run()
        b.record()
    torch.cuda.synchronize()
    del g
    return statistics.median(a.elapsed_time(b) for a, b in ev)


def kernel_table(dev, pk):
    """ms/call and TFLOP/s of dense and SRSU at N = 4096 and 25600, the
    memory-bound kernels' GB/s at N = 25600, and the SRSU |S|/N sweep."""
    from mask_free_b200 import ops
    out = {"timing": "device ms per call: CUDA-graph replay of 20 back-to-back calls (inputs above the L2 size); "
                     "kernels whose inputs fit in or near L2 (N = 4096 attention, cross, PCSP, top-k, classify, "
                     "scatter, sensitivity field, SW-CFG): 'ms' is the median of 20 single calls each after a 256 MB "
                     "L2 flush, 'ms_back_to_back' the replay figure"}
    for workload in ("n4096", "n25600"):
        s, inp, lsum = make_step_inputs(workload, dev)
        if workload == "n4096":
            k = s.k
        else:
            k = s.k
        S = torch.sort(torch.randperm(s.N, device=dev)[:k])[0].to(torch.int32).expand(s.B, k).contiguous()
        O = torch.empty_like(inp["Q"])
        Os = torch.empty((s.B, k, s.H, s.d), dtype=torch.bfloat16, device=dev)
        dense_f, srsu_f, cross_f, _ = flops(s, lsum, k)
        ws_d = torch.empty(max(256, ops.attn_workspace_bytes(s.B, s.N, s.N, s.H, s.d)), dtype=torch.uint8, device=dev)
        ws_s = torch.empty(max(256, ops.srsu_workspace_bytes(s.B, k, s.N, s.H, s.d)), dtype=torch.uint8, device=dev)
        f_dense = lambda: ops.attn_self(inp["Q"], inp["K"], inp["V"], out=O, ws=ws_d)
        f_srsu = lambda: ops.srsu_attn(inp["Q"], S, inp["Kc"], inp["Vc"], out=Os, ws=ws_s)
        Ox = torch.empty_like(O)
        f_cross = lambda: ops.attn_cross(inp["Q"], inp["Ky"], inp["Vy"], inp["valid_len"], out=Ox)
        t_d, t_s, t_x = time_kernel(f_dense), time_kernel(f_srsu), time_kernel(f_cross)
        t_x_b2b = t_x
        t_x = time_flushed(f_cross)
        small = workload == "n4096"  # Q, K, V of 37.7 MB each: flush between calls
        t_d_b2b, t_s_b2b = t_d, t_s
        if small:
            t_d, t_s = time_flushed(f_dense), time_flushed(f_srsu)
        tag = f"N{s.N}"
        out[f"dense_{tag}"] = {"ms": t_d, "tflops": dense_f / t_d / 1e9,
                               "pct_bf16_burst": 100 * dense_f / t_d / 1e9 / pk["bf16"],
                               "pct_bf16_sustained": 100 * dense_f / t_d / 1e9 / pk["bf16_sustained"]}
        out[f"srsu_{tag}_k{k}"] = {"ms": t_s, "tflops": srsu_f / t_s / 1e9,
                                   "pct_bf16_burst": 100 * srsu_f / t_s / 1e9 / pk["bf16"],
                                   "pct_bf16_sustained": 100 * srsu_f / t_s / 1e9 / pk["bf16_sustained"]}
        if small:
            out[f"dense_{tag}"]["ms_back_to_back"] = t_d_b2b
            out[f"srsu_{tag}_k{k}"]["ms_back_to_back"] = t_s_b2b
        # context only (the pages' mask-induced dispatch tax, on this machine):
        # torch's own SDPA on the same tensors without a mask and with the
        # all-valid boolean mask that the classifier certifies removable
        # (fused backends only: the unfused one would materialise N x N scores)
        try:
            import torch.nn.functional as F
            from torch.nn.attention import SDPBackend, sdpa_kernel
            qt, kt, vt = (inp[n].transpose(1, 2) for n in ("Q", "K", "V"))
            with sdpa_kernel([SDPBackend.FLASH_ATTENTION, SDPBackend.EFFICIENT_ATTENTION, SDPBackend.CUDNN_ATTENTION]):
                t_free = time_kernel(lambda: F.scaled_dot_product_attention(qt, kt, vt), reps=3, warm=1)
                t_mask = time_kernel(lambda: F.scaled_dot_product_attention(qt, kt, vt, attn_mask=inp["mask"]),
                                     reps=3, warm=1)
            out[f"torch_sdpa_context_N{s.N}"] = {
                "mask_free_ms": t_free, "all_valid_bool_mask_ms": t_mask, "masked_over_mask_free": t_mask / t_free,
                "ours_dense_ms": t_d}
            del qt, kt, vt
        except Exception as e:  # context only: record why it could not run
            out[f"torch_sdpa_context_N{s.N}"] = {"unavailable": f"{type(e).__name__}: {str(e)[:160]}"}
        torch.cuda.synchronize()
        xbytes = 2 * 2 * s.B * s.N * s.H * s.d + 2 * 2 * s.B * s.M * s.H * s.d
        out[f"cross_{tag}"] = {"ms": t_x, "gbs": xbytes / t_x / 1e6, "pct_hbm": 100 * xbytes / t_x / 1e6 / pk["hbm"],
                               "tflops": cross_f / t_x / 1e9, "ms_back_to_back": t_x_b2b}
        if workload == "n25600":
            # memory-bound kernels
            cls = torch.empty(3, dtype=torch.int64, device=dev)
            f_c = lambda: ops.mask_classify(inp["mask"], sync=False, result=cls)
            t_c, t_c_b2b = time_flushed(f_c), time_kernel(f_c)
            mb = inp["mask"].numel()
            out["classify_bool_2x1xNxN"] = {"ms": t_c, "gbs": mb / t_c / 1e6, "pct_hbm": 100 * mb / t_c / 1e6 / pk["hbm"],
                                            "ms_back_to_back": t_c_b2b}
            Kc, Vc = inp["Kc"].clone(), inp["Vc"].clone()
            f_sc = lambda: ops.ctx_cache_scatter(inp["K"], inp["V"], S, Kc, Vc, src_compact=False)
            t_sc, t_sc_b2b = time_flushed(f_sc), time_kernel(f_sc)
            sb = 4 * s.B * k * s.H * s.d * 2
            out["scatter"] = {"ms": t_sc, "gbs": sb / t_sc / 1e6, "pct_hbm": 100 * sb / t_sc / 1e6 / pk["hbm"],
                              "ms_back_to_back": t_sc_b2b}
            # SRSU with K/V of S u C assembled in the kernel (no scatter pass,
            # cache only read) against the two launches scatter + SRSU
            t_a = time_kernel(lambda: ops.srsu_attn_assembled(inp["Q"], S, inp["K"], inp["V"], inp["Kc"], inp["Vc"],
                                                              out=Os, ws=ws_s))
            out[f"srsu_assembled_{tag}_k{k}"] = {
                "ms": t_a, "tflops": srsu_f / t_a / 1e9, "pct_bf16_burst": 100 * srsu_f / t_a / 1e9 / pk["bf16"],
                "scatter_plus_srsu_ms": t_sc_b2b + t_s, "saved_ms": t_sc_b2b + t_s - t_a}
            # row-wise layers of the row-selective block (Eq. (15)) at width
            # H*d = 2304: QKV projection and MLP up (GELU) on the rows of S,
            # MLP down on the compact hidden rows; context: torch's linear
            # (cuBLAS) on the same rows already gathered
            dm = s.H * s.d
            Xh = torch.randn((s.B, s.N, dm), device=dev).to(torch.bfloat16)
            lin = {}
            for name, din, dout, act, rows in (("qkv", dm, 3 * dm, "none", S), ("mlp_up", dm, 4 * dm, "gelu_tanh", S),
                                               ("mlp_down", 4 * dm, dm, "none", None)):
                Wl = (torch.randn((dout, din), device=dev) / math.sqrt(din)).to(torch.bfloat16)
                bl = torch.zeros(dout, device=dev)
                Xin = Xh if rows is not None else torch.randn((s.B, k, din), device=dev).to(torch.bfloat16)
                Yl = torch.empty((s.B, k, dout), dtype=torch.bfloat16, device=dev)
                t_l = time_kernel(lambda: ops.gather_linear(Xin, Wl, S=rows, bias=bl, act=act, out=Yl))
                fl = 2.0 * s.B * k * din * dout
                Xg = Xin if rows is None else torch.stack([Xin[b, rows[b].long()] for b in range(s.B)])
                blh = bl.to(torch.bfloat16)
                t_cb = time_kernel(lambda: torch.nn.functional.linear(Xg, Wl, blh), reps=10)
                lin[name] = {"ms": t_l, "tflops": fl / t_l / 1e9, "pct_bf16_burst": 100 * fl / t_l / 1e9 / pk["bf16"],
                             "d_in": din, "d_out": dout, "act": act, "rows_gathered": rows is not None,
                             "torch_linear_on_gathered_rows_ms": t_cb}
                del Wl, Xin, Yl, Xg, blh
            del Xh
            out[f"block_linear_{tag}_k{k}"] = lin
            sc = torch.empty((s.B, s.N), dtype=torch.float32, device=dev)
            ws = torch.empty(ops.pcsp_workspace_bytes(s.B, s.N, s.H), dtype=torch.uint8, device=dev)
            f_p = lambda: ops.pcsp_topk(inp["Q"], inp["Ky"], inp["valid_len"], inp["w"], scores=sc, ws=ws)
            t_p, t_p_b2b = time_flushed(f_p), time_kernel(f_p)
            pb = 2 * s.B * s.N * s.H * s.d + 4 * s.B * s.H * s.N * 2 + 4 * s.B * s.N
            out["pcsp_scores"] = {"ms": t_p, "gbs": pb / t_p / 1e6, "pct_hbm": 100 * pb / t_p / 1e6 / pk["hbm"],
                                  "ms_back_to_back": t_p_b2b}
            f_xp = lambda: ops.attn_cross_pcsp(inp["Q"], inp["Ky"], inp["Vy"], inp["valid_len"], inp["w"], out=Ox,
                                               scores=sc, ws=ws)
            t_xp, t_xp_b2b = time_flushed(f_xp), time_kernel(f_xp)
            xpb = xbytes + 4 * s.B * s.H * s.N * 2 + 4 * s.B * s.N
            out["cross_with_pcsp"] = {"ms": t_xp, "gbs": xpb / t_xp / 1e6, "pct_hbm": 100 * xpb / t_xp / 1e6 / pk["hbm"],
                                      "vs_separate_calls": (t_x + t_p) / t_xp, "ms_back_to_back": t_xp_b2b}
            Sk = torch.empty((s.B, k), dtype=torch.int32, device=dev)
            Ck = torch.empty((s.B, s.N - k), dtype=torch.int32, device=dev)
            f_t = lambda: ops.topk_partition(sc, k, S=Sk, C=Ck)
            out["topk"] = {"ms": time_flushed(f_t), "ms_back_to_back": time_kernel(f_t)}
            # sensitivity field (Eq. (11)) of the PCSP scores on the 160 x 160
            # latent grid, and SW-CFG (Eq. (20), (21)) of one CFG pair with 16
            # prediction values per token (2 x 2 patch x 4 latent channels)
            side = int(math.isqrt(s.N))
            if side * side == s.N:
                sf = torch.empty_like(sc)
                wsf = torch.empty(ops.sensitivity_workspace_bytes(s.B, s.N), dtype=torch.uint8, device=dev)
                f_f = lambda: ops.sensitivity_field(sc, side, side, 2.0, out=sf, ws=wsf)
                t_f = time_flushed(f_f)
                out["sensitivity_field"] = {"ms": t_f, "grid": f"{side}x{side}", "sigma": 2.0,
                                            "gbs": 5 * 4 * s.B * s.N / t_f / 1e6, "ms_back_to_back": time_kernel(f_f)}
                for dt, tag in ((torch.float32, "f32"), (torch.bfloat16, "bf16")):
                    fc = torch.randn((1, s.N, 16), device=dev).to(dt)
                    fu = torch.randn((1, s.N, 16), device=dev).to(dt)
                    fo = torch.empty_like(fc)
                    f_g = lambda: ops.sw_cfg(fc, fu, sf[:1], 4.0, 7.5, out=fo)
                    t_g = time_flushed(f_g)
                    gb = 3 * fc.numel() * fc.element_size() + 4 * s.N
                    out[f"sw_cfg_{tag}"] = {"ms": t_g, "gbs": gb / t_g / 1e6, "pct_hbm": 100 * gb / t_g / 1e6 / pk["hbm"],
                                            "ms_back_to_back": time_kernel(f_g)}
            # SRSU wall time against |S|/N
            sweep = {}
            for rho in (0.1, 0.2, 0.3, 0.5, 1.0):
                kk = max(1, math.ceil(rho * s.N))
                Sr = torch.sort(torch.randperm(s.N, device=dev)[:kk])[0].to(torch.int32).expand(s.B, kk).contiguous()
                Osr = torch.empty((s.B, kk, s.H, s.d), dtype=torch.bfloat16, device=dev)
                wsr = torch.empty(max(256, ops.srsu_workspace_bytes(s.B, kk, s.N, s.H, s.d)), dtype=torch.uint8,
                                  device=dev)
                sweep[str(rho)] = time_kernel(lambda: ops.srsu_attn(inp["Q"], Sr, inp["Kc"], inp["Vc"], out=Osr,
                                                                    ws=wsr), reps=10)
            out["srsu_rho_sweep_ms"] = sweep
            out["srsu_t_rho_over_t_1"] = {r: v / sweep["1.0"] for r, v in sweep.items()}
        del inp
        torch.cuda.empty_cache()
    out.update(sequence_n36864(dev, pk))
    out.update(block_step_n25600(dev, pk))
    return out


def sequence_n36864(dev, pk):
    """The 3072^2-equivalent workload (N = 36864, M = 256, k = 7373): each
    call kind alone, and the 20-call sequence as the schedule runs it
    (anchors at calls 0, 5, 10, 15: dense self-attention, full cache refresh
    and cross-attention over all rows, Eq. (18), (19); other calls: scatter
    of the rows of S, SRSU and cross-attention on S, Eq. (15)-(17)). One
    CUDA event pair around each call; the sequence runs twice and the second
    pass is reported."""
    from mask_free_b200 import ops
    s, inp, lsum = make_step_inputs("n36864_seq", dev)
    k = s.k
    S = torch.sort(torch.randperm(s.N, device=dev)[:k])[0].to(torch.int32).expand(s.B, k).contiguous()
    O = torch.empty_like(inp["Q"])
    Ox = torch.empty_like(O)
    Os = torch.empty((s.B, k, s.H, s.d), dtype=torch.bfloat16, device=dev)
    Osx = torch.empty_like(Os)
    dense_f, srsu_f, cross_f, cross_s_f = flops(s, lsum, k)
    ws_d = torch.empty(max(256, ops.attn_workspace_bytes(s.B, s.N, s.N, s.H, s.d)), dtype=torch.uint8, device=dev)
    ws_s = torch.empty(max(256, ops.srsu_workspace_bytes(s.B, k, s.N, s.H, s.d)), dtype=torch.uint8, device=dev)
    Kc, Vc = inp["Kc"], inp["Vc"]
    t_d = time_kernel(lambda: ops.attn_self(inp["Q"], inp["K"], inp["V"], out=O, ws=ws_d), reps=5)
    t_s = time_kernel(lambda: ops.srsu_attn(inp["Q"], S, Kc, Vc, out=Os, ws=ws_s), reps=10)
    t_x = time_kernel(lambda: ops.attn_cross(inp["Q"], inp["Ky"], inp["Vy"], inp["valid_len"], out=Ox))
    xbytes = 2 * 2 * s.B * s.N * s.H * s.d + 2 * 2 * s.B * s.M * s.H * s.d
    res = {
        "dense_N36864": {"ms": t_d, "tflops": dense_f / t_d / 1e9, "pct_bf16_burst": 100 * dense_f / t_d / 1e9 / pk["bf16"]},
        f"srsu_N36864_k{k}": {"ms": t_s, "tflops": srsu_f / t_s / 1e9,
                              "pct_bf16_burst": 100 * srsu_f / t_s / 1e9 / pk["bf16"]},
        "cross_N36864_M256": {"ms": t_x, "gbs": xbytes / t_x / 1e6, "pct_hbm": 100 * xbytes / t_x / 1e6 / pk["hbm"]},
    }

    def call(t):
        if t % 5 == 0:
            ops.attn_self(inp["Q"], inp["K"], inp["V"], out=O, ws=ws_d)
            ops.ctx_cache_scatter(inp["K"], inp["V"], None, Kc, Vc)
            ops.attn_cross(inp["Q"], inp["Ky"], inp["Vy"], inp["valid_len"], out=Ox)
        else:
            ops.ctx_cache_scatter(inp["K"], inp["V"], S, Kc, Vc, src_compact=False)
            ops.srsu_attn(inp["Q"], S, Kc, Vc, out=Os, ws=ws_s)
            ops.attn_cross(inp["Q"], inp["Ky"], inp["Vy"], inp["valid_len"], q_idx=S, out=Osx)

    for rep in range(2):
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(21)]
        torch.cuda.synchronize()
        ev[0].record()
        for t in range(20):
            call(t)
            ev[t + 1].record()
        torch.cuda.synchronize()
    per = [ev[t].elapsed_time(ev[t + 1]) for t in range(20)]
    anchors = [per[t] for t in range(20) if t % 5 == 0]
    others = [per[t] for t in range(20) if t % 5 != 0]
    seq_f = 4 * (dense_f + cross_f) + 16 * (srsu_f + cross_s_f)
    res["sequence_N36864_20_calls"] = {
        "total_ms": sum(per), "anchor_calls_ms": sum(anchors), "srsu_calls_ms": sum(others),
        "anchor_call_ms_mean": statistics.mean(anchors), "srsu_call_ms_mean": statistics.mean(others),
        "dense_every_call_ms_estimate": 20 * (t_d + t_x), "tflops": seq_f / sum(per) / 1e9,
        "calls": "anchors 0, 5, 10, 15: dense + full refresh + cross; others: scatter + SRSU + cross on S"}
    del inp, O, Ox, Os, Osx, Kc, Vc, ws_d, ws_s
    torch.cuda.empty_cache()
    return res


def block_step_n25600(dev, pk):
    """The row-selective block B^S of Eq. (15) at the 2560^2 workload,
    composed of the library's calls, beside the dense block on all N rows.
    Row-selective: q, k, v projections of the rows of S of the hidden state
    (each H d -> H d), scatter of k, v into the context cache, SRSU over
    S u C, cross-attention on S, MLP up (GELU, H d -> 4 H d) and down on the
    rows of S. Dense: the same layers on all N rows with dense
    self-attention. Normalisations, modulation and residual adds (elementwise)
    are not included. Weights are synthetic. Device time of one CUDA-graph
    replay of 5 back-to-back steps."""
    from mask_free_b200 import ops
    s, inp, lsum = make_step_inputs("n25600", dev)
    B, N, H, d, k = s.B, s.N, s.H, s.d, s.k
    D = H * d
    S = torch.sort(torch.randperm(N, device=dev)[:k])[0].to(torch.int32).expand(B, k).contiguous()
    X = torch.randn((B, N, D), device=dev).to(torch.bfloat16)
    W = {n: (torch.randn(sh, device=dev) / math.sqrt(sh[1])).to(torch.bfloat16)
         for n, sh in (("q", (D, D)), ("k", (D, D)), ("v", (D, D)), ("up", (4 * D, D)), ("down", (D, 4 * D)))}
    Kc, Vc = inp["Kc"], inp["Vc"]
    bufs = {}

    def buf(name, shape):
        if name not in bufs:
            bufs[name] = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        return bufs[name]

    ws_s = torch.empty(max(256, ops.attn_workspace_bytes(B, k, N, H, d)), dtype=torch.uint8, device=dev)
    ws_d = torch.empty(max(256, ops.attn_workspace_bytes(B, N, N, H, d)), dtype=torch.uint8, device=dev)

    def selective():
        q = ops.gather_linear(X, W["q"], S=S, out=buf("q", (B, k, D))).view(B, k, H, d)
        kk = ops.gather_linear(X, W["k"], S=S, out=buf("k", (B, k, D))).view(B, k, H, d)
        v = ops.gather_linear(X, W["v"], S=S, out=buf("v", (B, k, D))).view(B, k, H, d)
        ops.ctx_cache_scatter(kk, v, S, Kc, Vc, src_compact=True)
        o = ops.srsu_attn(q, S, Kc, Vc, q_compact=True, out=buf("o", (B, k, H, d)), ws=ws_s)
        ops.attn_cross(q, inp["Ky"], inp["Vy"], inp["valid_len"], out=buf("ox", (B, k, H, d)))
        h1 = ops.gather_linear(o.view(B, k, D), W["up"], act="gelu_tanh", out=buf("h1", (B, k, 4 * D)))
        ops.gather_linear(h1, W["down"], out=buf("y", (B, k, D)))

    def dense():
        q = ops.gather_linear(X, W["q"], out=buf("qd", (B, N, D))).view(B, N, H, d)
        kk = ops.gather_linear(X, W["k"], out=buf("kd", (B, N, D))).view(B, N, H, d)
        v = ops.gather_linear(X, W["v"], out=buf("vd", (B, N, D))).view(B, N, H, d)
        o = ops.attn_self(q, kk, v, out=buf("od", (B, N, H, d)), ws=ws_d)
        ops.attn_cross(q, inp["Ky"], inp["Vy"], inp["valid_len"], out=buf("oxd", (B, N, H, d)))
        h1 = ops.gather_linear(o.view(B, N, D), W["up"], act="gelu_tanh", out=buf("h1d", (B, N, 4 * D)))
        ops.gather_linear(h1, W["down"], out=buf("yd", (B, N, D)))

    selective()
    dense()
    t_sel = time_kernel(selective, reps=5)
    t_den = time_kernel(dense, reps=3)
    lin = lambda rows: 2.0 * B * rows * (3 * D * D + 2 * 4 * D * D)
    f_sel = lin(k) + 4.0 * B * H * k * N * d + 4.0 * H * d * k * lsum
    f_den = lin(N) + 4.0 * B * H * N * N * d + 4.0 * H * d * N * lsum
    res = {"block_step_N25600": {
        "row_selective_ms": t_sel, "row_selective_tflops": f_sel / t_sel / 1e9,
        "dense_block_ms": t_den, "dense_block_tflops": f_den / t_den / 1e9,
        "dense_over_row_selective": t_den / t_sel, "k": k,
        "layers": "q, k, v projections (2304 -> 2304 each), attention, MLP 2304 -> 9216 (GELU) -> 2304"}}
    del X, W, bufs, inp, Kc, Vc
    torch.cuda.empty_cache()
    return res


ONLY_KERNELS = ("self", "srsu", "cross", "pcsp", "topk", "scatter", "classify", "linear")


def run_only(kernel: str, workload: str, launches: int):
    """Launch one kernel of the hot path `launches` times on one workload and
    nothing else, for a profiler's launch list or capture. Inputs are drawn
    on the device (standard normals in bf16, like the step), so the process
    holds only the tensors of that one call (n4096: ~0.2 GB). `linear` is the
    row-selective block's QKV layer: the k rows of S of a [B, N, H*d] hidden
    state, H*d -> 3*H*d."""
    from mask_free_b200 import ops
    s = synth.WORKLOADS[workload]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(s.seed_id)

    def bf(rows):
        return torch.randn((s.B, rows, s.H, s.d), generator=g, device=dev).to(torch.bfloat16)

    lens = synth.uniform_lengths(s.B, s.len_lo, s.len_hi, 1).to(dev)
    S = torch.sort(torch.randperm(s.N, device=dev, generator=g)[:s.k])[0].to(torch.int32)
    S = S.expand(s.B, s.k).contiguous()
    if kernel in ("self", "srsu", "cross", "pcsp", "scatter"):
        Q, K, V = bf(s.N), bf(s.N), bf(s.N)
    if kernel in ("cross", "pcsp"):
        Ky, Vy = bf(s.M), bf(s.M)
    if kernel == "linear":
        dm = s.H * s.d
        X = torch.randn((s.B, s.N, dm), generator=g, device=dev).to(torch.bfloat16)
        Wt = (torch.randn((3 * dm, dm), generator=g, device=dev) / dm ** 0.5).to(torch.bfloat16)
    for _ in range(launches):
        if kernel == "self":
            ops.attn_self(Q, K, V)
        elif kernel == "srsu":
            ops.srsu_attn(Q, S, K, V)
        elif kernel == "cross":
            ops.attn_cross(Q, Ky, Vy, lens)
        elif kernel == "pcsp":
            ops.pcsp_topk(Q, Ky, lens, None)
        elif kernel == "topk":
            ops.topk_partition(torch.randn((s.B, s.N), generator=g, device=dev), s.k)
        elif kernel == "scatter":
            ops.ctx_cache_scatter(K, V, S, Q, Q.clone(), src_compact=False)
        elif kernel == "linear":
            ops.gather_linear(X, Wt, S=S)
        elif kernel == "classify":
            ops.mask_classify(torch.ones((s.B, 1, s.N, s.N), dtype=torch.bool, device=dev))
    torch.cuda.synchronize()
    assert ops.device_status() == 0
    print(json.dumps({"only": kernel, "workload": workload, "launches": launches, "status": "ok"}))


MX_RATE = {"mxfp8": 2, "mxfp4": 4, "nvfp4": 4}  # nominal rate of a format's products over bf16's
# layers whose kernel is timed by itself: rows, d_in, d_out, activation
MX_LAYERS = ((51200, 2304, 6912, "none"), (12800, 2304, 9216, "gelu_tanh"), (12800, 9216, 6912, "none"),
             (2458, 9216, 2304, "none"))


def operator_limit(case, work, pk):
    """Microseconds for a pass's bytes at the measured copy rate, or for a
    layer's products at the measured bf16 rate times the format's, whichever is
    longer. Not a lower bound where inputs stay in L2 between passes."""
    us = work["bytes"] / pk["hbm"] / 1e3
    if case["op"] == "linear":
        us = max(us, work["flops"] / (pk["bf16"] * MX_RATE[case["fmt"]]) / 1e6)
    return us


def time_passes(fn, seconds=0.5):
    """(us a pass, passes) of eager passes back to back for about `seconds`, the
    host's work included."""
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]

    def batch(n):
        torch.cuda.synchronize()
        ev[0].record()
        for _ in range(n):
            fn()
        ev[1].record()
        torch.cuda.synchronize()
        return ev[0].elapsed_time(ev[1]) * 1e3 / n

    batch(3)
    n = max(5, int(seconds * 1e6 / batch(5)))
    return batch(n), n


def time_one_cool(fn):
    """Device us of a single call after an L2 flush, on a GPU that has idled for a
    second (behind seconds at the power limit the clock stays low)."""
    torch.cuda.synchronize()
    time.sleep(1.0)
    return time_flushed(fn) * 1e3


def run_operators(which):
    """One JSON line for each measured case of the row-wise operators
    (perf/operators.py) and for each of MX_LAYERS: us a pass back to back,
    device us of a single pass (time_one_cool), and with `which` "both" the
    plain forms' pass; then one with the clocks of the whole run."""
    from mask_free_b200 import ops
    from perf import operators as P
    pk, dev = peaks(), torch.device("cuda", torch.cuda.current_device())
    r1 = lambda v: round(v, 1)
    with ClockSampler(dev.index) as clk:
        for case in P.listed():
            P.own = True
            state = P.prepare(case, 1)
            one = time_one_cool(lambda: P.run(state))
            us, n = time_passes(lambda: P.run(state))
            line = {"case": case["name"], "limit_us": round(operator_limit(case, P.work(case), pk), 3), "pass_us": r1(us),
                    "passes": n, "device_us": r1(one)}
            P.own = False
            if which == "both":
                line["plain_us"] = r1(time_passes(lambda: P.run(state), 0.1)[0])
            print(json.dumps(line), flush=True)
            del state
            torch.cuda.empty_cache()
        gen = torch.Generator(device=dev).manual_seed(1)
        for fmt in MX_RATE:
            for M, d_in, d_out, act in MX_LAYERS:
                X, W = (ops.mx_quantize(torch.randn((n, d_in), generator=gen, device=dev), fmt,
                                        scale=0.003 if fmt == "nvfp4" else 1.0) for n in (M, d_out))
                out = torch.empty((M, d_out), dtype=torch.bfloat16, device=dev)
                bias = torch.randn(d_out, generator=gen, device=dev)
                fn = lambda: ops.mx_linear(X, W, bias, act, out=out)
                one, (us, n) = time_one_cool(fn), time_passes(fn, 2.0)
                flop = 2.0 * M * d_in * d_out
                print(json.dumps({"layer": f"{fmt} {M} x {d_in} x {d_out} {act}", "device_us": r1(one),
                                  "pflops": round(flop / one / 1e9, 2), "back_to_back_us": r1(us), "calls": n,
                                  "pflops_back_to_back": round(flop / us / 1e9, 2)}), flush=True)
    print(json.dumps({"clocks": clk.summary(), "peaks": pk["source"]}), flush=True)


def host_info():
    """Host cores and CPU model of the box the oracle runs on."""
    model = None
    try:
        for line in open("/proc/cpuinfo"):
            if line.startswith("model name"):
                model = line.split(":", 1)[1].strip()
                break
    except OSError:
        pass
    try:
        usable = len(os.sched_getaffinity(0))
    except AttributeError:
        usable = os.cpu_count()
    return {"nproc": usable, "cpu_model": model}


def blas_threads():
    from threadpoolctl import threadpool_info
    return max([i.get("num_threads", 1) for i in threadpool_info()] + [1])


class OracleSample:
    """The fp64 oracle (as it stands) on a bounded sample of the workload:
    dense self-attention query rows of the N = 25600 step, all 48 (b, h)
    pairs, against all keys."""

    def __init__(self):
        s = synth.WORKLOADS["n25600"]
        rng = np.random.default_rng(0)
        shape = (s.B, s.N, s.H, s.d)
        self.s = s
        self.Q = rng.standard_normal((s.B, 64, s.H, s.d)).astype(np.float32).astype(np.float64)
        self.K = rng.standard_normal(shape).astype(np.float32).astype(np.float64)
        self.V = rng.standard_normal(shape).astype(np.float32).astype(np.float64)

    def run(self, budget_s):
        import oracle as O
        s = self.s
        rows_done, t0 = 0, time.perf_counter()
        while time.perf_counter() - t0 < budget_s:
            O.attention(self.Q, self.K, self.V, 1 / math.sqrt(s.d))
            rows_done += self.Q.shape[1]
        el = time.perf_counter() - t0
        fl = 4.0 * s.B * s.H * rows_done * s.N * s.d
        threads = blas_threads()
        hi = host_info()
        return {"value": fl / el / 1e12, "unit": "TFLOP/s", "cores": threads, "kind": "oracle",
                "nproc": hi["nproc"], "cpu_model": hi["cpu_model"],
                "sample": f"fp64 oracle dense self-attention, {rows_done} query rows x 48 (b,h) at N=25600, "
                          f"d=96, {el:.1f} s; numpy with {threads} BLAS threads on {hi['nproc']} host cores",
                "seconds": el}


def oracle_per_call(rows: int = 512, heads: int = 4):
    """The fp64 oracle per kind of call on every attention workload: dense
    self-attention, SRSU (rows of S against all keys), cross-attention and
    the PCSP scores, each timed on `rows` query rows of `heads` (b = 0, h <
    heads) pairs and extrapolated to a full call (x rows of the call / rows x
    B H / heads; the oracle's cost is linear in both). A bounded sample of
    each workload: about 10 s of host time in all."""
    import oracle as O
    out = {}
    for wl in ("n4096", "n25600", "n36864_seq"):
        s = synth.WORKLOADS[wl]
        rng = np.random.default_rng(1)
        f64 = lambda *sh: rng.standard_normal(sh).astype(np.float32).astype(np.float64)
        K, V = f64(1, s.N, heads, s.d), f64(1, s.N, heads, s.d)
        Ky, Vy = f64(1, s.M, heads, s.d), f64(1, s.M, heads, s.d)
        Q = f64(1, rows, heads, s.d)
        lens = np.array([s.len_hi])
        w = np.full((1, s.M), 1.0 / s.M)
        scale = 1 / math.sqrt(s.d)
        # K/V rows of this sample stand for all N keys; Q rows for the rows of the call
        Qfull = np.zeros((1, s.N, heads, s.d))
        Qfull[:, :rows] = Q
        sel = np.arange(rows)[None, :]
        kinds = {
            "dense": (lambda: O.attention(Q, K, V, scale), s.N),
            "srsu": (lambda: O.srsu_attention(Qfull, sel, K, V, scale), s.k),
            "cross": (lambda: O.cross_attention(Q, Ky, Vy, lens, scale), s.N),
            "pcsp": (lambda: O.pcsp_scores(Q, Ky, lens, w, scale), s.N),
        }
        res = {}
        for kind, (fn, call_rows) in kinds.items():
            t0 = time.perf_counter()
            fn()
            el = time.perf_counter() - t0
            res[kind] = {"sample_s": el, "extrapolated_full_call_s": el * (call_rows / rows) * (s.B * s.H / heads)}
        out[wl] = res
    hi = host_info()
    return {"sample": f"{rows} query rows x {heads} (b,h) pairs per kind and workload (longest text length), "
                      f"extrapolated to the full call; numpy fp64 with {blas_threads()} BLAS threads",
            "nproc": hi["nproc"], "cpu_model": hi["cpu_model"], "per_call": out}


def run_reference(args, rank, world):
    if rank != 0:
        return
    sample = OracleSample()
    budget = max(2.0, 60.0 / max(1, args.steps + args.warmup))
    vals, last = [], None
    for i in range(args.warmup + args.steps):
        last = sample.run(budget)
        if i >= args.warmup:
            vals.append(last["value"])
    v = statistics.median(vals)
    cb = dict(last, value=v)
    ms = None
    print(json.dumps({
        "metric": METRIC, "value": v, "unit": "TFLOP/s", "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": ms, "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "f64", "data": "synthetic", "impl": "reference",
        "config": {"workload": WORKLOAD, "sample": cb["sample"]},
        "cpu_baseline": cb, "e2e": {"value": v, "unit": "TFLOP/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }), flush=True)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--warmup", type=int, default=3)
    ap.add_argument("--impl", default="ours", choices=["ours", "reference"])
    ap.add_argument("--no-kernel-table", action="store_true")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--clock-log", default=None, help="directory for the raw clock samples (default: a temp dir)")
    ap.add_argument("--only", default=None, choices=ONLY_KERNELS,
                    help="launch one kernel and nothing else (for profilers); no JSON bench line")
    ap.add_argument("--workload", default="n4096", choices=sorted(synth.WORKLOADS), help="workload of --only")
    ap.add_argument("--launches", type=int, default=3, help="launches of --only")
    ap.add_argument("--operators", default=None, nargs="?", const="kernels", choices=["kernels", "both"],
                    help="time the row-wise operators' cases and nothing else (both: their plain forms too)")
    args = ap.parse_args()
    if args.operators is not None:
        run_operators(args.operators)
        return
    if args.only is not None:
        run_only(args.only, args.workload, args.launches)
        return
    args.warmup = max(3, args.warmup)

    world = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    dist = None
    if world > 1:
        import datetime
        import torch.distributed as dist
        torch.cuda.set_device(local)
        dist.init_process_group("nccl", timeout=datetime.timedelta(seconds=120))
    if args.impl == "reference":
        run_reference(args, rank, world)
        if dist is not None:
            dist.destroy_process_group()
        return

    from mask_free_b200 import ops
    ops.lib()
    dev = torch.device("cuda", local)
    torch.cuda.set_device(dev)
    pk = peaks()
    s, inp, lsum = make_step_inputs("n25600", dev)
    step = Step(s, inp, dev)
    f_dense, f_srsu, f_cross, f_cross_s = flops(s, lsum, s.k)
    f_step = f_dense + f_srsu + f_cross + f_cross_s

    for _ in range(args.warmup):
        step()
    torch.cuda.synchronize()
    if dist is not None:
        dist.barrier()
    torch.cuda.synchronize()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with ClockSampler(local, args.clock_log) as clk:
        t0.record()
        for _ in range(args.steps):
            step(timed=True)
        t1.record()
        torch.cuda.synchronize()
    if dist is not None:
        dist.barrier()
    torch.cuda.synchronize()
    ms_total = max_over_ranks(t0.elapsed_time(t1), dist, dev)
    ms_step = ms_total / args.steps
    value = job_throughput(world, f_step, ms_step)

    # end to end through the public API with host buffers: every step copies
    # its inputs from pinned host memory and its results back. Two device
    # buffer sets and two copy streams let the copies of one step overlap
    # the compute of its neighbours; each step still starts only after its
    # own inputs have arrived, and the clock stops after the last results
    # are on the host. (The all-valid attention mask is a device-resident
    # tensor of the model, shared by both sets, and is not re-sent.)
    host = {n: inp[n].cpu().pin_memory() for n in ("Q", "K", "V", "Ky", "Vy", "valid_len", "w")}
    inp2 = {n: (t if n == "mask" else t.clone()) for n, t in inp.items()}
    sets = [(inp, step), (inp2, Step(s, inp2, dev))]
    outs = [[st.O, st.Ox, st.Os, st.Osx, st.S] for _, st in sets]
    host_out = [[torch.empty(o.shape, dtype=o.dtype, pin_memory=True) for o in outs[0]] for _ in range(2)]
    h2d = sum(t.numel() * t.element_size() for t in host.values())
    d2h = sum(t.numel() * t.element_size() for t in host_out[0])
    comp, s_in, s_out = torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()
    ev_in, ev_done, ev_out = ([torch.cuda.Event() for _ in range(2)] for _ in range(3))
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e_steps = max(4, args.steps)  # as many steps as the device-side measurement (fill and drain included)

    def pipeline(n):
        for i in range(n):
            b = i % 2
            ins, st = sets[b]
            with torch.cuda.stream(s_in):
                if i >= 2:
                    s_in.wait_event(ev_done[b])  # step i-2 has finished reading this set
                for n_, t in host.items():
                    ins[n_].copy_(t, non_blocking=True)
                ev_in[b].record(s_in)
            comp.wait_event(ev_in[b])
            if i >= 2:
                comp.wait_event(ev_out[b])  # step i-2's results have left this set
            st()
            ev_done[b].record(comp)
            with torch.cuda.stream(s_out):
                s_out.wait_event(ev_done[b])
                for o, ho in zip(outs[b], host_out[b]):
                    ho.copy_(o, non_blocking=True)
                ev_out[b].record(s_out)

    # untimed warm-up of the same pipeline (the first copies from freshly
    # pinned pages run well below the link rate)
    pipeline(args.warmup)
    torch.cuda.synchronize()
    if dist is not None:
        dist.barrier()
    torch.cuda.synchronize()
    e0.record(s_in)
    pipeline(e_steps)
    e1.record(s_out)
    torch.cuda.synchronize()
    ms_e2e = max_over_ranks(e0.elapsed_time(e1) / e_steps, dist, dev)
    # the host link alone: one step's input and result copies, both
    # directions at once, no compute (the bound the pipelined steps approach)
    link = []
    for _ in range(3):
        c0, c1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        c0.record(s_in)
        with torch.cuda.stream(s_in):
            for n_, t in host.items():
                sets[0][0][n_].copy_(t, non_blocking=True)
        s_out.wait_event(c0)
        with torch.cuda.stream(s_out):
            for o, ho in zip(outs[0], host_out[0]):
                ho.copy_(o, non_blocking=True)
        s_in.wait_stream(s_out)
        c1.record(s_in)
        torch.cuda.synchronize()
        link.append(c0.elapsed_time(c1))
    e2e = {"value": job_throughput(world, f_step, ms_e2e), "unit": "TFLOP/s", "h2d_bytes_per_step": h2d,
           "d2h_bytes_per_step": d2h, "ms_per_step": ms_e2e, "steps": e_steps,
           "overlap": "copies of step i overlap the compute of steps i-1 / i+1 (two buffer sets)",
           "copies_alone_ms": min(link)}
    del sets, inp2, outs

    dense_list, srsu_list = step.launch_times()
    dense_ms, srsu_ms = statistics.mean(dense_list), statistics.mean(srsu_list)
    # the burst bf16 peak is the denominator (the larger, so the smaller
    # fraction); the fraction of the sustained peak, measured over a
    # seconds-long GEMM loop under the power cap, is printed beside it
    achieved = f_dense / (dense_ms * 1e-3) / 1e12
    achieved_srsu = f_srsu / (srsu_ms * 1e-3) / 1e12
    roofline = {"bound": "tensor", "achieved": achieved, "peak": pk["bf16"], "unit": "TFLOP/s",
                "frac": achieved / pk["bf16"], "traffic": stored_traffic(),
                "kernel": "flash_fwd_kernel<96> (dense self-attention, N=25600)",
                "peak_note": f"{pk['source']} burst bf16 peak ({'of measured' if pk['source'] == 'measured' else 'of fallback'}); "
                             f"frac of the sustained peak {achieved / pk['bf16_sustained']:.3f}",
                "units_per_launch": "4*B*H*N^2*d = %.4g FLOP" % f_dense,
                "launch_ms_in_step": dense_ms}
    roofline_srsu = {"bound": "tensor", "achieved": achieved_srsu, "peak": pk["bf16"], "unit": "TFLOP/s",
                     "frac": achieved_srsu / pk["bf16"], "traffic": None,
                     "kernel": "flash_fwd_kernel<96> (SRSU, N=25600, k=6400)",
                     "units_per_launch": "4*B*H*k*N*d = %.4g FLOP" % f_srsu, "launch_ms_in_step": srsu_ms}
    kernels = {"dense_in_step_ms": dense_ms, "srsu_in_step_ms": srsu_ms, "srsu_in_step_tflops": achieved_srsu}
    launches = step.launches * args.steps
    del step
    torch.cuda.empty_cache()
    if not args.no_kernel_table:
        kernels.update(kernel_table(dev, pk))
    cpu = None
    if rank == 0 and world == 1 and not args.no_cpu_baseline:
        cpu = OracleSample().run(12.0)
        cpu["per_call"] = oracle_per_call()
    if rank == 0:
        print(json.dumps({
            "metric": METRIC, "value": value, "unit": "TFLOP/s", "n_gpus": world, "steps": args.steps,
            "warmup": args.warmup, "ms_per_step": ms_step, "higher_is_better": True, "scaling": "weak",
            "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
            "config": {"workload": WORKLOAD, "parallelism": f"replicas x{world}" if world > 1 else "single GPU",
                       "l2": "inputs exceed L2 (236 MB per image tensor); no flush",
                       "flops_per_step": f_step},
            "roofline": roofline, "roofline_srsu": roofline_srsu, "cpu_baseline": cpu, "e2e": e2e,
            "gpu_launches": launches, "clocks": clk.summary(), "kernels": kernels,
        }), flush=True)
    if dist is not None:
        dist.barrier()
        dist.destroy_process_group()


if __name__ == "__main__":
    main()
