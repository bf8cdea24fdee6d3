"""Benchmark of the selective-scan hot path: one training step = ss_fwd_save
(forward, keeping the backward's restart states) + ss_bwd_saved (backward)
over one batch of the Mamba-2.8B-layer workload (Bsz=4, L=4096, Dch=5120,
N=16, bf16 I/O, f32 state and gradients), through the C ABI.

    python bench.py [--gpus N] [--steps K] [--warmup W] [--impl ours|reference]

Prints one JSON line (rank 0).  ``value`` is whole-job throughput in B*L*D
elements per second of forward+backward with inputs resident in HBM;
``e2e`` is the same metric with host<->device copies of each step's inputs
and results inside the timed region.  ``--impl reference`` times the CPU
oracle (the plain f64 reference the tests compare against) on a bounded
sample of the same workload on this host's cores.  Under torchrun every rank
runs an independent replica (the scan shards over batch and channels with no
exchange); rank 0 reports.
"""

from __future__ import annotations

import argparse
import csv
import io
import json
import os
import statistics
import subprocess
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from mamba_selective_scan_fwd_gb300.inputs import WORKLOADS, make_inputs  # noqa: E402

METRIC = "selective-scan fwd+bwd elements/s (B·L·D) and HBM GB/s vs GB300 peak"
UNIT = "elements/s"
WORKLOAD = WORKLOADS[3]  # mamba2.8b-layer-bf16: the workload the metric is quoted on
# the other full-size workloads, each timed as a block of its own: the
# Mamba-130M layer forward (bf16) and training step (f32), and the long sequence
PER_WORKLOAD = (1, 2, 4)


def pick_workload(name):
    """The workload named on the command line (every one runs forward + backward here)."""
    for w in WORKLOADS:
        if w.name == name:
            return w
    raise SystemExit(f"unknown workload {name!r}; one of {[w.name for w in WORKLOADS]}")

# Algorithmic bytes per element (B*L*D unit) for bf16 I/O, f32 gradients:
#   forward  = u, delta, z read + y write (4 x 2 B) = 8 B  (+ B, C, A, D, bias, last_state: per-(b,t) / per-d terms)
#   backward = u, delta, z, dy read (4 x 2 B) + du, ddelta, dz write (3 x 4 B) = 20 B  (+ B, C, dB, dC, dA, ...)
# The small per-(b, t, n) and per-(d, n) terms are added exactly below.


IO_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def algorithmic_bytes(w):
    e = IO_BYTES[w.io]
    bld, bln, dn, d = w.Bsz * w.L * w.Dch, w.Bsz * w.L * w.N, w.Dch * w.N, w.Dch
    fwd = 4 * bld * e + 2 * bln * e + 4 * (dn + 2 * d) + 4 * w.Bsz * w.Dch * w.N
    bwd = 4 * bld * e + 3 * bld * 4 + 2 * bln * (e + 4) + 8 * (dn + 2 * d)
    return fwd, bwd


# FP32 operations (multiplies, adds and fused multiply-adds, one FP32-pipe
# result each) of one state update (t, d, n), as the method's arithmetic needs
# them.  Forward: the exponent delta_eff * A, the input term (delta_eff u) * B,
# the recurrence a h + x and the readout h C.  Backward, recomputing the
# states from the saved ones as the method prescribes: those first three, then
# lam = g C + carry, carry' = a lam, sum_n lam B, q = carry' h_prev,
# sum_n A q, dA += delta_eff q, dB += lam (delta_eff u), dC += g h.
F32_OPS_FWD = 4
F32_OPS_BWD = 11


def mufu_counts(w):
    """MUFU operations of one call of each direction on workload w (softplus on,
    z given): the scan's ex2 per (t, d, n), which the roofline counts, and all
    of them -- per (t, d) the forward's softplus (ex2, rcp) and gate sigmoid
    (ex2, rcp), the backward's softplus with its derivative (ex2, two rcp) and
    gate sigmoid (ex2, rcp).  The chunk summaries of time-cut units, which
    walk their decays once more, are not counted."""
    return {"scan_ex2_per_direction": w.bld * w.N, "fwd_all": w.bld * (w.N + 4), "bwd_all": w.bld * (w.N + 5)}


# DRAM bytes (read + write) of the timed kernels' main passes on this workload
# (the sum over the launches of one pass: one per plan segment), from one ncu
# capture (profiles/ holds the summaries and the commands).  The digest names the
# kernel sources they hold for: a change of those makes the figure stale, and it is
# reported as null.  (The capture was taken at 2f86bc4c97822ea2; since then api.cu
# gained two host functions, device_status_word and tensor_map_encoder, and no
# kernel, launch or plan changed.)
TRAFFIC = {
    # both launches of the main pass (608 one-chunk units; 32 units x 19 chunks)
    ("k_bwd_main", "mamba2.8b-layer-bf16"): 2948585216,  # 1596.0 + 85.5 MB read, 1238.2 + 28.9 MB written
    ("k_fwd_y", "mamba2.8b-layer-bf16"): 1573153792,     # 480.0 + 26.8 MB read, 1059.3 + 7.0 MB written
}
TRAFFIC_SRC_DIGEST = "e3773bb4658a0346"

# timed end-to-end runs (their median is reported)
E2E_RUNS = 5


def measured_traffic(kernel, w):
    from mamba_selective_scan_fwd_gb300 import build

    if TRAFFIC_SRC_DIGEST is None or build.source_digest() != TRAFFIC_SRC_DIGEST:
        return None
    return TRAFFIC.get((kernel, w.name))


def load_peaks():
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(path):
        with open(path) as f:
            p = json.load(f)
        return float(p["hbm_gbs"]), "measured"
    return 6800.0, "fallback"


class ClockSampler:
    """nvidia-smi clock / throttle sampling while the timed region runs."""

    FIELDS = ("clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,clocks_event_reasons.hw_slowdown,"
              "clocks_event_reasons.hw_thermal_slowdown,clocks_event_reasons.sw_thermal_slowdown,"
              "clocks_event_reasons.sw_power_cap")

    def __init__(self, gpu_index):
        self.proc = None
        self.gpu = gpu_index

    def start(self):
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", "-i", str(self.gpu), f"--query-gpu={self.FIELDS}", "--format=csv,noheader,nounits",
                 "-lms", "100"], stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
        except OSError:
            self.proc = None

    def stop(self):
        if self.proc is None:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["nvidia-smi unavailable"]}
        self.proc.terminate()
        try:
            out, _ = self.proc.communicate(timeout=5)
        except subprocess.TimeoutExpired:
            self.proc.kill()
            out, _ = self.proc.communicate()
        sm, smax, reasons = [], [], set()
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for row in csv.reader(io.StringIO(out)):
            if len(row) < 8:
                continue
            try:
                sm.append(float(row[0]))
                smax.append(float(row[1]))
            except ValueError:
                continue
            for name, val in zip(names, row[4:8]):
                if val.strip().lower() == "active":
                    reasons.add(name)
        return {"sm_mhz": statistics.median(sm) if sm else None, "sm_max_mhz": max(smax) if smax else None,
                "reasons": sorted(reasons), "samples": len(sm)}


def dist_setup(backend="nccl"):
    """One process per GPU (torchrun env).  Replicas only: the process group
    carries the barrier and the max-over-ranks timing, never data."""
    import torch

    world = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    if world > 1:
        import torch.distributed as dist

        if backend == "nccl":
            torch.cuda.set_device(local)
            dist.init_process_group("nccl", device_id=torch.device("cuda", local))
        else:
            dist.init_process_group(backend)
    elif backend == "nccl" and torch.cuda.is_available():
        torch.cuda.set_device(0)
    return world, rank, local


def barrier(world):
    if world > 1:
        import torch.distributed as dist

        dist.barrier()


def max_over_ranks(x, world, device="cuda"):
    if world == 1:
        return x
    import torch
    import torch.distributed as dist

    t = torch.tensor([x], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def job_throughput(units_per_rank, world, ms):
    """Whole-job rate: the units every replica processed over the slowest rank's time."""
    return world * units_per_rank / (ms / 1e3)


def measure_decode(dev, hbm_peak, peak_kind, steps=50):
    """One ss_decode_step per token on a Mamba-2.8B-layer decoding batch whose
    state (Bsz x Dch x N f32) is larger than the L2: HBM-bound, reported
    against the measured copy bandwidth."""
    import torch

    import mamba_selective_scan_fwd_gb300 as ss

    Bsz, Dch, N = 512, 5120, 16
    g = torch.Generator(device=dev).manual_seed(7)
    bf = torch.bfloat16
    u = torch.randn((Bsz, Dch), generator=g, device=dev).to(bf)
    delta = (0.5 * torch.randn((Bsz, Dch), generator=g, device=dev)).to(bf)
    z = torch.randn((Bsz, Dch), generator=g, device=dev).to(bf)
    Bm = torch.randn((Bsz, N), generator=g, device=dev).to(bf)
    Cm = torch.randn((Bsz, N), generator=g, device=dev).to(bf)
    A = -torch.arange(1, N + 1, device=dev, dtype=torch.float32).repeat(Dch, 1).contiguous()
    D = torch.ones(Dch, device=dev)
    bias = torch.full((Dch,), -4.0, device=dev)
    state = torch.randn((Bsz, Dch, N), generator=g, device=dev)
    y = torch.empty((Bsz, Dch), dtype=bf, device=dev)

    def step():
        ss.ss_decode_step(u, delta, A, Bm, Cm, D, z, bias, True, state, y=y)

    for _ in range(3):
        step()
    torch.cuda.synchronize(dev)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(steps):
        step()
    e1.record()
    torch.cuda.synchronize(dev)
    ms = e0.elapsed_time(e1) / steps
    # state read + written, u / delta / z read and y written (bf16), B / C, A, D, bias
    nbytes = 2 * Bsz * Dch * N * 4 + 4 * Bsz * Dch * 2 + 2 * Bsz * N * 2 + Dch * N * 4 + 2 * Dch * 4
    ach = nbytes / (ms / 1e3) / 1e9
    return {"workload": f"mamba2.8b-layer-decode-bf16 (Bsz={Bsz}, Dch={Dch}, N={N}, state {Bsz * Dch * N * 4 >> 20} MiB)",
            "ms_per_token": round(ms, 5), "tokens_per_s": round(Bsz / (ms / 1e3), 1),
            "roofline": {"bound": "hbm", "achieved": round(ach, 1), "peak": hbm_peak, "unit": "GB/s",
                         "frac": round(ach / hbm_peak, 4), "peak_kind": f"{peak_kind} HBM copy",
                         "algorithmic_bytes": nbytes}}


IO_KEYS = ("u", "delta", "B", "C", "z", "dy")


def config_of(w, world):
    """The ``config`` dict of a workload's line (the same in both arms)."""
    fwd_b, bwd_b = algorithmic_bytes(w)
    step_b = fwd_b + (bwd_b if w.backward else 0)
    return {"workload": w.name, "Bsz": w.Bsz, "L": w.L, "Dch": w.Dch, "N": w.N, "io": w.io,
            "step": "ss_fwd_save + ss_bwd_saved" if w.backward else "ss_fwd",
            "terms": "D, z, delta_bias, softplus, last_state",
            "l2": f"no flush: each step moves {step_b / 1e6:.0f} MB, above the 129 MB L2",
            "parallelism": "replicas" if world > 1 else "single GPU"}


class Runner:
    """Device-resident inputs, outputs and workspaces of one workload, and its calls."""

    def __init__(self, w, x, dev, stream, pin=False):
        import torch

        import mamba_selective_scan_fwd_gb300 as ss
        from mamba_selective_scan_fwd_gb300 import binding

        self.ss, self.w, self.dev, self.stream = ss, w, dev, stream
        io_dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[w.io]
        self.host = {}
        for k, v in x.items():
            if v is None:
                continue
            t = torch.from_numpy(v)
            if k in IO_KEYS:
                t = t.to(io_dt)
            self.host[k] = t.pin_memory() if pin else t
        self.d = {k: v.to(dev) for k, v in self.host.items()}
        for k in ("D", "z", "delta_bias", "dy"):
            self.d.setdefault(k, None)
        dt = binding.dtype_id(self.d["u"])
        dims = (w.Bsz, w.L, w.Dch, w.N, dt)
        self.plan = ss.plan_info(*dims)
        self.staging = "tma" if ss.staging_uses_tma(*dims) else "asynchronous copies"
        u8 = torch.uint8
        self.ws_f = torch.empty(max(ss.fwd_workspace_bytes(*dims), 256), dtype=u8, device=dev)
        self.y = torch.empty((w.Bsz, w.L, w.Dch), dtype=io_dt, device=dev)
        self.last = torch.empty((w.Bsz, w.Dch, w.N), dtype=torch.float32, device=dev)
        self.grads = {}
        if w.backward:
            self.ws_b = torch.empty(ss.bwd_saved_workspace_bytes(*dims), dtype=u8, device=dev)
            self.saved = torch.empty(ss.saved_bytes(*dims), dtype=u8, device=dev)
            self.ws_r = None  # the recomputing backward's workspace, made on first use

    def _args(self, d):
        return (d["u"], d["delta"], d["A"], d["B"], d["C"], d["D"], d["z"], d["delta_bias"], self.w.softplus)

    def fwd(self):
        self.ss.ss_fwd(*self._args(self.d), y=self.y, last_state=self.last, workspace=self.ws_f, stream=self.stream)

    def fwd_save(self):
        self.ss.ss_fwd_save(*self._args(self.d), y=self.y, last_state=self.last, saved=self.saved,
                            workspace=self.ws_f, stream=self.stream)

    def bwd_saved(self):
        self.grads.update(self.ss.ss_bwd_saved(*self._args(self.d), self.d["dy"], self.saved, out=self.grads,
                                               workspace=self.ws_b, stream=self.stream))

    def bwd(self):
        import torch

        if self.ws_r is None:
            w = self.w
            dims = (w.Bsz, w.L, w.Dch, w.N, 0 if w.io == "f32" else 2 if w.io == "bf16" else 1)
            self.ws_r = torch.empty(self.ss.bwd_workspace_bytes(*dims), dtype=torch.uint8, device=self.dev)
        self.grads.update(self.ss.ss_bwd(*self._args(self.d), self.d["dy"], out=self.grads, workspace=self.ws_r,
                                         stream=self.stream))

    def first(self):
        """The step's first call: the saving forward (or the forward of a forward-only step)."""
        return self.fwd_save() if self.w.backward else self.fwd()

    def step(self):
        self.first()
        if self.w.backward:
            self.bwd_saved()

    def step_recompute(self):
        self.fwd()
        self.bwd()

    def launches(self):
        return self.plan["fwd_kernels"] + (self.plan["bwd_saved_kernels"] if self.w.backward else 0)


def time_steps(fn, K, dev, stream, world):
    """Device time of exactly K calls of fn between two events on the launching stream (max over ranks)."""
    import torch

    barrier(world)
    torch.cuda.synchronize(dev)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record(stream)
    for _ in range(K):
        fn()
    e1.record(stream)
    torch.cuda.synchronize(dev)
    barrier(world)
    return max_over_ranks(e0.elapsed_time(e1), world)


def attribute(r, K):
    """K more steps with events around each call and between the library's own
    launches (it records them there): per-call and per-kernel average ms."""
    import torch

    from mamba_selective_scan_fwd_gb300 import binding

    plan, stream = r.plan, r.stream
    nf, nb = plan["fwd_kernels"], (plan["bwd_saved_kernels"] if r.w.backward else 0)
    evs = [[torch.cuda.Event(enable_timing=True) for _ in range(3)] for _ in range(K)]
    kev_f = [[torch.cuda.Event(enable_timing=True) for _ in range(nf + 1)] for _ in range(K)]
    kev_b = [[torch.cuda.Event(enable_timing=True) for _ in range(nb + 1)] for _ in range(K)]
    for e in [e for row in kev_f + kev_b for e in row]:
        e.record(stream)  # creates the event handles the library records
    torch.cuda.synchronize(r.dev)
    for i in range(K):
        evs[i][0].record(stream)
        binding.profile_events(kev_f[i])
        r.first()
        evs[i][1].record(stream)
        if r.w.backward:
            binding.profile_events(kev_b[i])
            r.bwd_saved()
        evs[i][2].record(stream)
    binding.profile_events([])
    torch.cuda.synchronize(r.dev)
    t_fwd = sum(e[0].elapsed_time(e[1]) for e in evs) / K
    t_bwd = sum(e[1].elapsed_time(e[2]) for e in evs) / K if r.w.backward else 0.0
    # kernel j of a call runs between its events j and j + 1
    k_fwd = [sum(row[j].elapsed_time(row[j + 1]) for row in kev_f) / K for j in range(nf)]
    k_bwd = [sum(row[j].elapsed_time(row[j + 1]) for row in kev_b) / K for j in range(nb)]
    return t_fwd, t_bwd, k_fwd, k_bwd


def analyse(w, plan, ms_per_step, t_fwd, t_bwd, k_fwd, k_bwd, peaks):
    """Rooflines of the step, of its dominant kernel and of the forward's main pass.

    A kernel's (or direction's) roofline time is the slowest of three floors:
    its algorithmic bytes at the measured HBM copy bandwidth, its B*L*D*N
    scan exponentials at the measured MUFU ex2 rate, and its algorithmic FP32
    operations (F32_OPS_* per state update) at the measured FP32-pipe rate
    (SMs x results per clock per SM x the sampled SM clock).  The binding
    floor names the bound; the others are kept beside it."""
    fwd_bytes, bwd_bytes = algorithmic_bytes(w)
    # the backward's main kernel writes everything but dB / dC and dA / dD / ddelta_bias (the reductions do)
    bwd_main_bytes = bwd_bytes - 2 * w.Bsz * w.L * w.N * 4 - 4 * (w.Dch * w.N + 2 * w.Dch)
    hbm_peak = peaks["hbm_gbs"]
    clk = f"{peaks['sm_mhz']:g} MHz (median sampled)"
    exp_peak = peaks["sms"] * peaks["ex2_per_clk_per_sm"] * peaks["sm_mhz"] * 1e6  # ex2 / s
    fma_peak = peaks["sms"] * peaks["fma_per_clk_per_sm"] * peaks["sm_mhz"] * 1e6  # f32 results / s
    exps = w.bld * w.N

    def roof(bytes_, f32ops, t_ms):
        floors = {"hbm": bytes_ / (hbm_peak * 1e9), "fp32": f32ops / fma_peak, "mufu": exps / exp_peak}
        bound = max(floors, key=floors.get)
        t_s = t_ms / 1e3
        hbm = {"achieved": round(bytes_ / t_s / 1e9, 1), "peak": hbm_peak, "unit": "GB/s",
               "frac": round(bytes_ / t_s / 1e9 / hbm_peak, 4)}
        if bound == "hbm":
            r = dict(hbm, bound="hbm", peak_kind=f"{peaks['hbm_kind']} HBM copy")
        elif bound == "fp32":
            pk = fma_peak / 1e9
            r = {"bound": "alu", "achieved": round(f32ops / t_s / 1e9, 1), "peak": round(pk, 1), "unit": "Gop/s",
                 "frac": round(f32ops / t_s / 1e9 / pk, 4),
                 "peak_kind": (f"FP32 pipe (measured): {peaks['sms']} SMs x {peaks['fma_per_clk_per_sm']:.1f} "
                               f"f32 results/clk x {clk}"),
                 "algorithmic_f32_ops": f32ops}
        else:
            pk = exp_peak / 1e9
            r = {"bound": "alu", "achieved": round(exps / t_s / 1e9, 1), "peak": round(pk, 1), "unit": "Gexp2/s",
                 "frac": round(exps / t_s / 1e9 / pk, 4),
                 "peak_kind": (f"MUFU ex2 (measured): {peaks['sms']} SMs x {peaks['ex2_per_clk_per_sm']:.2f}/clk x "
                               f"{clk}")}
        r.update({"roofline_ms": round(floors[bound] * 1e3, 4), "algorithmic_bytes": bytes_,
                  "floors_ms": {k: round(v * 1e3, 4) for k, v in floors.items()}})
        if bound != "hbm":
            r["hbm"] = hbm
        return r

    # launch order of a call: the summary passes of the chunked segments (in the
    # backward followed by their carry passes), then each segment's main pass
    # (then, in the backward, the two reductions)
    segs = plan["segments"]
    tag = [f"{u} units x {k} chunk{'s' if k > 1 else ''}" for u, k in segs]
    first = "y + saved states" if w.backward else "y"
    chunked = [i for i, (_, k) in enumerate(segs) if k > 1]
    fwd_names = [f"k_fwd chunk summary ({tag[i]})" for i in chunked] + [f"k_fwd {first} ({t})" for t in tag]
    bwd_names = ([f"k_bwd reverse summary ({tag[i]})" for i in chunked] +
                 [f"k_bwd_carry ({tag[i]})" for i in chunked] +
                 [f"k_bwd main ({t})" for t in tag] + ["k_bwd_reduce_bc", "k_bwd_reduce_params"])
    # a direction's main pass: one launch per segment
    main_f = range(len(chunked), len(chunked) + len(segs))
    main_b = range(2 * len(chunked), 2 * len(chunked) + len(segs))
    t_main_f = sum(k_fwd[j] for j in main_f)
    launches = f"{len(segs)} launch{'es' if len(segs) > 1 else ''}"
    f32_fwd, f32_bwd = F32_OPS_FWD * exps, F32_OPS_BWD * exps
    r_fwd = roof(fwd_bytes, f32_fwd, t_main_f)
    r_fwd.update({"kernel": f"k_fwd main pass ({'ss_fwd_save' if w.backward else 'ss_fwd'}; {launches})",
                  "ms": round(t_main_f, 4), "traffic": measured_traffic("k_fwd_y", w)})
    out = {"hbm_gbs": round((fwd_bytes + (bwd_bytes if w.backward else 0)) / (ms_per_step / 1e3) / 1e9, 1),
           "ns_per_element": round(ms_per_step * 1e6 / w.bld, 5)}
    t_roof = roof(fwd_bytes, f32_fwd, t_fwd)["roofline_ms"]
    if w.backward:
        t_main_b = sum(k_bwd[j] for j in main_b)
        r_bwd = roof(bwd_main_bytes, f32_bwd, t_main_b)
        r_bwd.update({"kernel": f"k_bwd main pass (ss_bwd_saved; {launches})", "ms": round(t_main_b, 4),
                      "traffic": measured_traffic("k_bwd_main", w)})
        t_roof += roof(bwd_bytes, f32_bwd, t_bwd)["roofline_ms"]
        out.update({"roofline": r_bwd, "roofline_fwd": r_fwd})
    else:
        out["roofline"] = r_fwd
    out["roofline_step_frac"] = round(t_roof / ms_per_step, 4)
    out["fwd_ms"] = round(t_fwd, 4)
    if w.backward:
        out["bwd_ms"] = round(t_bwd, 4)
    names = fwd_names + (bwd_names if w.backward else [])
    out["kernel_ms"] = {n: round(v, 4) for n, v in zip(names, k_fwd + k_bwd)}
    return out


def measure_unit_rates():
    """MUFU ex2 and FP32-pipe (f32 FMA) results per clock per SM, measured by
    the library's probe kernels (the first run of each warms up; the second is
    reported)."""
    from mamba_selective_scan_fwd_gb300 import binding

    binding.measure_ex2_rate(1024)
    ex2 = binding.measure_ex2_rate(4096)
    binding.measure_fma_rate(1024)
    return ex2, binding.measure_fma_rate(4096)


def run_workload(w, dev, stream, world, K, warmup, peaks, cpu_seconds, rank):
    """One per-workload block: the step's throughput and rooflines, and the oracle's rate."""
    import torch

    x = make_inputs(w, with_dy=w.backward)
    r = Runner(w, x, dev, stream)
    for _ in range(warmup):
        r.step()
    total = time_steps(r.step, K, dev, stream, world)
    ms = total / K
    t_fwd, t_bwd, k_fwd, k_bwd = attribute(r, K)
    block = {"config": config_of(w, world), "steps": K, "ms_per_step": round(ms, 4),
             "value": round(job_throughput(w.bld * K, world, total), 1), "unit": UNIT, "staging": r.staging,
             "chunks": r.plan["chunks"]}
    block.update(analyse(w, r.plan, ms, t_fwd, t_bwd, k_fwd, k_bwd, peaks))
    del r
    torch.cuda.empty_cache()
    if rank == 0 and cpu_seconds > 0:
        block["cpu_baseline"] = cpu_baseline(w, x, budget_s=cpu_seconds)
    return block


def run_ours(args):
    import torch

    import mamba_selective_scan_fwd_gb300 as ss

    world, rank, local = dist_setup("nccl")
    dev = torch.device("cuda", local if world > 1 else 0)
    ss.set_copies_only(args.staging == "copies")
    w = pick_workload(args.workload)
    x = make_inputs(w, with_dy=w.backward)
    stream = torch.cuda.current_stream(dev)
    r = Runner(w, x, dev, stream, pin=True)

    for _ in range(args.warmup):
        r.step()
    torch.cuda.synchronize(dev)

    # ---- device-resident timing: exactly K steps between two events on the
    # launching stream, nothing else in between; clocks sampled meanwhile
    K = args.steps
    clocks = ClockSampler(local if world > 1 else 0)
    clocks.start()
    time.sleep(0.3)
    total_ms = time_steps(r.step, K, dev, stream, world)
    clk = clocks.stop()
    ms_per_step = total_ms / K
    value = job_throughput(w.bld * K, world, total_ms)
    t_fwd, t_bwd, k_fwd, k_bwd = attribute(r, K)

    # ---- the recomputing pair (ss_fwd + ss_bwd: the backward recomputes the
    # restart states itself) on the same inputs (a forward-only workload has none)
    recompute_ms = None
    if w.backward:
        for _ in range(3):
            r.step_recompute()
        recompute_ms = time_steps(r.step_recompute, K, dev, stream, world) / K

    # ---- end to end through the public API with host buffers.  Every step copies
    # its inputs from pinned host memory and its outputs back; two sets of device
    # input / output buffers and one copy stream per direction let step i's
    # input copy run during step i - 1's compute and its output copy during
    # step i + 1's (the restart states and workspaces stay on the compute
    # stream).  The output copy bounds it (1178 MB per step); splitting each
    # copy over two streams per direction was no faster.
    ss, host, d = r.ss, r.host, r.d
    in_keys = [k for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "dy") if k in host]
    h2d = sum(host[k].numel() * host[k].element_size() for k in in_keys)
    out_host = {"y": torch.empty(r.y.shape, dtype=r.y.dtype).pin_memory(),
                "last_state": torch.empty(r.last.shape, dtype=r.last.dtype).pin_memory()}
    for k, v in r.grads.items():
        if v is not None:
            out_host[k] = torch.empty(v.shape, dtype=v.dtype).pin_memory()
    d2h = sum(v.numel() * v.element_size() for v in out_host.values())
    e2e_steps = max(2, min(args.e2e_steps, K))
    sets = []
    for _ in range(2):
        di = {k: (None if v is None else torch.empty_like(v)) for k, v in d.items()}
        sets.append({"d": di, "y": torch.empty_like(r.y), "last": torch.empty_like(r.last), "g": {}})
    s_in, s_out = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
    ev = {k: [torch.cuda.Event() for _ in range(2)] for k in ("in", "done", "out")}

    def e2e_run(nsteps, start_ev=None):
        if start_ev is not None:
            s_in.wait_event(start_ev)
        for i in range(nsteps):
            j = i % 2
            bs = sets[j]
            with torch.cuda.stream(s_in):
                if i >= 2:
                    s_in.wait_event(ev["done"][j])  # step i - 2 is done reading this set's inputs
                for k in in_keys:
                    bs["d"][k].copy_(host[k], non_blocking=True)
                ev["in"][j].record(s_in)
            stream.wait_event(ev["in"][j])
            if i >= 2:
                stream.wait_event(ev["out"][j])  # step i - 2's outputs have left this set
            di = bs["d"]
            fargs = (di["u"], di["delta"], di["A"], di["B"], di["C"], di["D"], di["z"], di["delta_bias"], w.softplus)
            if w.backward:
                ss.ss_fwd_save(*fargs, y=bs["y"], last_state=bs["last"], saved=r.saved, workspace=r.ws_f,
                               stream=stream)
                bs["g"].update(ss.ss_bwd_saved(*fargs, di["dy"], r.saved, out=bs["g"], workspace=r.ws_b,
                                               stream=stream))
            else:
                ss.ss_fwd(*fargs, y=bs["y"], last_state=bs["last"], workspace=r.ws_f, stream=stream)
            ev["done"][j].record(stream)
            with torch.cuda.stream(s_out):
                s_out.wait_event(ev["done"][j])
                out_host["y"].copy_(bs["y"], non_blocking=True)
                out_host["last_state"].copy_(bs["last"], non_blocking=True)
                for k, v in bs["g"].items():
                    if v is not None:
                        out_host[k].copy_(v, non_blocking=True)
                ev["out"][j].record(s_out)
        stream.wait_event(ev["out"][(nsteps - 1) % 2])

    e2e_run(2)
    torch.cuda.synchronize(dev)
    # five timed runs of e2e_steps steps: the host link is shared with other
    # work on the machine and its throughput varies from run to run (seen: 2x),
    # so the median is reported and every run is listed
    e2e_runs = []
    for _ in range(E2E_RUNS):
        barrier(world)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(stream)
        e2e_run(e2e_steps, start_ev=e0)
        e1.record(stream)
        torch.cuda.synchronize(dev)
        barrier(world)
        e2e_runs.append(max_over_ranks(e0.elapsed_time(e1), world))
    e2e_ms = sorted(e2e_runs)[E2E_RUNS // 2]
    e2e_value = job_throughput(w.bld * e2e_steps, world, e2e_ms)
    staging, plan, launches = r.staging, r.plan, r.launches()
    gstatus = ss.device_status(stream)
    del sets, r
    torch.cuda.empty_cache()

    # ---- peaks: the measured HBM copy bandwidth, MUFU ex2 rate and FP32-pipe rate
    hbm_peak, peak_kind = load_peaks()
    ex2, fma = measure_unit_rates()
    peaks = {"hbm_gbs": hbm_peak, "hbm_kind": peak_kind, "ex2_per_clk_per_sm": ex2, "fma_per_clk_per_sm": fma,
             "sms": torch.cuda.get_device_properties(dev).multi_processor_count,
             "sm_mhz": clk.get("sm_mhz") or 2070.0}
    stats = analyse(w, plan, ms_per_step, t_fwd, t_bwd, k_fwd, k_bwd, peaks)

    line = {
        "metric": METRIC, "value": round(value, 1), "unit": UNIT, "n_gpus": world, "steps": K,
        "warmup": args.warmup, "ms_per_step": round(ms_per_step, 4), "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "f32", "data": "synthetic", "config": config_of(w, world),
        "chunks": plan["chunks"], "staging": staging,
    }
    line.update(stats)
    line.update({
        "step_recompute_ms": None if recompute_ms is None else round(recompute_ms, 4),
        "mufu_ops": mufu_counts(w), "ex2_per_clk_per_sm": round(ex2, 3), "fma_per_clk_per_sm": round(fma, 2),
        "clocks": clk,
        "e2e": {"value": round(e2e_value, 1), "unit": UNIT, "h2d_bytes_per_step": h2d, "d2h_bytes_per_step": d2h,
                "steps": e2e_steps, "runs": [round(job_throughput(w.bld * e2e_steps, world, v), 1) for v in e2e_runs],
                "of_runs": "median"},
        "gpu_launches": K * launches,  # the timed region only
        "device_status": ss.status_string(gstatus),
    })
    if not args.no_decode:
        line["decode"] = measure_decode(dev, hbm_peak, peak_kind)
    if not args.no_per_workload:
        pw = {}
        for wi in PER_WORKLOAD:
            w2 = WORKLOADS[wi]
            pw[w2.name] = run_workload(w2, dev, stream, world, max(3, min(K, 20)), 3, peaks,
                                       args.cpu_seconds_per_workload, rank)
        line["per_workload"] = pw
    if rank == 0 and not args.no_cpu_baseline:
        line["cpu_baseline"] = cpu_baseline(w, x, budget_s=args.cpu_seconds)
    if rank == 0:
        print(json.dumps(line), flush=True)
    if world > 1:
        import torch.distributed as dist

        dist.destroy_process_group()


def _oracle_sample(orc, w, x, rows):
    """The oracle's forward (and backward, for a training step) on a row sample of
    the workload; returns seconds."""
    t0 = time.perf_counter()
    orc.fwd(x["u"], x["delta"], x["A"], x["B"], x["C"], x["D"], x["z"], x["delta_bias"], w.softplus, rows=rows)
    if w.backward:
        orc.bwd(x["u"], x["delta"], x["A"], x["B"], x["C"], x["D"], x["z"], x["delta_bias"], w.softplus, dy=x["dy"],
                rows=rows, want_dBdC=True)
    return time.perf_counter() - t0


def cpu_baseline(w, x, budget_s=15.0):
    """The oracle, as it stands, on a bounded row sample of the workload (all host cores).

    Row batches of growing size run until about ``budget_s`` seconds of oracle
    work have been timed; the rate is rows x L over the summed time."""
    import numpy as np

    import oracle

    orc = oracle.get()
    cores = oracle.default_threads()
    # f64 copies once, outside the timed sample
    x64 = {k: (None if v is None else np.ascontiguousarray(v, dtype=np.float64)) for k, v in x.items()}
    rng = np.random.default_rng(0)
    perm = rng.permutation(w.Bsz * w.Dch)
    _oracle_sample(orc, w, x64, perm[:cores])  # untimed: first-call overheads
    done, spent, n = 0, 0.0, cores
    while spent < budget_s and done < perm.size:
        rows = perm[done:done + n]
        spent += _oracle_sample(orc, w, x64, rows)
        done += rows.size
        n = min(2 * n, perm.size - done)
    return {"value": round(done * w.L / spent, 1), "unit": UNIT, "cores": cores, "kind": "oracle",
            "sample": f"{done} of {w.Bsz * w.Dch} (b, d) rows, full L={w.L}, "
                      f"{'forward + backward incl. dB/dC contributions' if w.backward else 'forward'}, f64, "
                      f"{spent:.1f} s"}


def run_reference(args):
    world = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    if rank != 0:
        return
    import numpy as np

    import oracle

    w = pick_workload(args.workload)
    x = make_inputs(w, with_dy=True)
    x64 = {k: (None if v is None else np.ascontiguousarray(v, dtype=np.float64)) for k, v in x.items()}
    orc = oracle.get()
    cores = oracle.default_threads()
    rng = np.random.default_rng(1)
    # size each step's row sample so that warmup + steps fit in about two minutes
    probe = _oracle_sample(orc, w, x64, rng.choice(w.Bsz * w.Dch, cores, replace=False)) / cores
    per_step_budget = 120.0 / max(1, args.steps + args.warmup)
    n = int(max(cores, min(w.Bsz * w.Dch, per_step_budget / max(probe, 1e-6))))
    n = max(1, n // cores * cores) if n >= cores else n
    for _ in range(args.warmup):
        _oracle_sample(orc, w, x64, rng.choice(w.Bsz * w.Dch, n, replace=False))
    total = 0.0
    for _ in range(args.steps):
        total += _oracle_sample(orc, w, x64, rng.choice(w.Bsz * w.Dch, n, replace=False))
    value = args.steps * n * w.L / total
    sample = f"{n} of {w.Bsz * w.Dch} (b, d) rows per step, full L={w.L}, forward + backward, f64 oracle"
    line = {
        "impl": "reference", "metric": METRIC, "value": round(value, 1), "unit": UNIT, "n_gpus": world,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": round(total / args.steps * 1e3, 3),
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64", "data": "synthetic",
        "config": config_of(w, world),
        "cpu_baseline": {"value": round(value, 1), "unit": UNIT, "cores": cores, "kind": "oracle", "sample": sample},
        "e2e": {"value": round(value, 1), "unit": UNIT, "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }
    print(json.dumps(line), flush=True)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--impl", choices=["ours", "reference"], default="ours")
    ap.add_argument("--e2e-steps", type=int, default=8)
    ap.add_argument("--cpu-seconds", type=float, default=15.0)
    ap.add_argument("--cpu-seconds-per-workload", type=float, default=6.0,
                    help="oracle seconds for each per-workload block's cpu_baseline (0: none)")
    ap.add_argument("--no-per-workload", action="store_true", help="time the headline workload only")
    ap.add_argument("--staging", choices=["tma", "copies"], default="tma",
                    help="tile staging of the scan kernels: TMA where the problem allows it (default), or "
                         "per-thread asynchronous copies everywhere (for comparison)")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-decode", action="store_true", help="skip the single-step decoding measurement")
    ap.add_argument("--workload", default=WORKLOAD.name,
                    help="workload to time (default: the one the metric is quoted on)")
    args = ap.parse_args()
    args.warmup = max(3, args.warmup)  # at least three untimed warm-up steps
    if args.impl == "reference":
        run_reference(args)
    else:
        run_ours(args)


if __name__ == "__main__":
    main()
