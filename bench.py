#!/usr/bin/env python
"""Decode-throughput benchmark of the GB300 packed quantized-weight decoder.

One step = one batched launch decoding a whole Llama-3-8B-shaped model
(225 tensors: attention q/k/v/o in gguf:q4_k, FFN gate/up/down in gguf:q6_k,
the [128256,4096] embedding in gguf:q8_0) from HBM-resident payloads into
bf16, i.e. every row of the decode path: validation, block staging, scale
decode, code unpack, FP32 arithmetic, RNE cast and the batched launcher.

Printed (rank 0): one JSON line on stdout, kept below 2500 characters, and
before it, on stderr, one line "[bench] details" with the JSON of everything
measured.  In the line:
  value         dequant GB/s = (payload bytes + output bytes) / step time,
                whole job (all ranks), inputs resident in HBM;
  e2e           the same metric through the public API with host buffers:
                each step copies the payloads host->device from pinned memory,
                decodes, and copies the decoded bf16 weights device->host;
  roofline      the decode kernel against the measured HBM copy bandwidth;
  cpu_baseline  the CPU oracle on a bounded sample of the same workload;
  parity        the timed launch's whole output against the oracle's.
In the details also:
  per_workload  the single-format workloads (q8_0, q4_0, q4_g64, q4_k, q6_k,
                nvfp4, mxfp4, iq4_nl), each timed back to back over buffer
                sets larger than L2 and as one launch after an L2 eviction;
  per_workload_next_formats
                the same for every other gguf and NInfer format, each on one
                [14336,4096] tensor -> bf16;
  fused_matmul  decode fused into its consumer (ndq_matmul_packed) against
                decode-to-bf16 + cuBLAS: one whole-model generation step
                (M = 1) and single tensors at M = 1 and 8.

`--impl reference` times the CPU oracle (the parity reference) on the host
cores instead, on a bounded sample of the same workload per step.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import ctypes
import hashlib
import json
import os
import statistics
import subprocess
import sys
import threading
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import synth  # noqa: E402

WORKLOAD_NAME = ("whole-model batched decode: Llama-3-8B-shaped weights, 225 tensors "
                 "(q/k/v/o gguf:q4_k, gate/up/down gguf:q6_k, embedding [128256,4096] gguf:q8_0) -> bf16, "
                 "one launch per step")
METRIC = "dequant GB/s (bytes in+out) and elements/s per format vs 8 TB/s HBM peak"
ALIGN = 256
# Descriptors per launch-table upload kernel of the batched call: a batched
# decode of n tensors is ceil(n / 128) upload launches and one decode launch.
UPLOAD_CHUNK = 128


def batched_launches(n: int) -> int:
    return -(-n // UPLOAD_CHUNK) + 1


def parse_args():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=400)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--impl", choices=["ours", "reference"], default="ours")
    ap.add_argument("--e2e-steps", type=int, default=5)
    ap.add_argument("--e2e-groups", type=int, default=32, help="tensor groups pipelined in the end-to-end leg")
    ap.add_argument("--no-workloads", action="store_true", help="skip the single-format workload table")
    ap.add_argument("--no-fused", action="store_true", help="skip the fused decode + product figures")
    ap.add_argument("--only-fused", default=None, metavar="FMT,N,K,M[,bf16]",
                    help="time one fused decode + product (weights FMT [N,K], M activation rows; binary32 "
                         "weights, or bfloat16 with ',bf16') for --steps launches and exit (for focused profiling)")
    ap.add_argument("--no-cpu", action="store_true", help="skip the CPU-oracle baseline")
    ap.add_argument("--no-parity", action="store_true",
                    help="skip the oracle comparisons of the timed outputs and the payload digests")
    ap.add_argument("--no-e2e", action="store_true")
    ap.add_argument("--cpu-fraction", type=int, default=1,
                    help="CPU baseline decodes 1/N of every tensor's blocks")
    ap.add_argument("--layers", type=int, default=32,
                    help="decoder layers of the model workload (profiling runs use fewer)")
    ap.add_argument("--no-embedding", action="store_true", help="leave the embedding out of the model workload")
    ap.add_argument("--only", default=None,
                    help="time one single-format workload (a label of synth.WORKLOADS) for --steps steps and exit")
    return ap.parse_args()


# What the line on stdout holds of each part (None: all of it).
LINE_PARTS = {
    "config": None, "clocks": None,
    "roofline": ("bound", "achieved", "peak", "unit", "frac", "traffic", "peak_source"),
    "parity": ("bit_exact", "elements", "mismatches", "tensors"),
    "payload_sha256": ("whole_model",),
    "cpu_baseline": ("value", "unit", "cores", "kind", "elements/s", "seconds", "sample"),
    "e2e": ("value", "unit", "ms_per_step", "steps", "h2d_bytes_per_step", "d2h_bytes_per_step", "gpu_launches_per_step"),
}
LINE_MAX = 2500


def result_line(res):
    """The JSON line for the measured result: its numbers, and of its parts what
    LINE_PARTS names; the tables are left to the details."""
    out = {}
    for k, v in res.items():
        if not isinstance(v, dict):
            out[k] = v
        elif k in LINE_PARTS:
            keep = LINE_PARTS[k]
            out[k] = {x: y for x, y in v.items() if keep is None or x in keep}
    line = json.dumps(out)
    if len(line) >= LINE_MAX:
        raise RuntimeError(f"the result line has {len(line)} characters, {LINE_MAX} or more")
    return line


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def dist_env():
    return (int(os.environ.get("RANK", 0)), int(os.environ.get("WORLD_SIZE", 1)),
            int(os.environ.get("LOCAL_RANK", 0)))


def max_over_ranks(value: float, device) -> float:
    """Largest `value` over all ranks (the slowest rank sets the job time)."""
    import torch
    import torch.distributed as dist

    if not (dist.is_available() and dist.is_initialized()) or dist.get_world_size() == 1:
        return value
    t = torch.tensor([value], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def job_gbs(bytes_per_rank: int, world: int, ms: float) -> float:
    """Whole-job throughput: every rank's bytes over the slowest rank's time."""
    return world * bytes_per_rank / (ms * 1e-3) / 1e9


def measured_peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        with open(p) as f:
            d = json.load(f)
        return float(d["hbm_gbs"]), "measured"
    except Exception:
        return 6800.0, "fallback"


# --------------------------------------------------------------------------
# workload layout
# --------------------------------------------------------------------------
class ModelWorkload:
    def __init__(self, specs):
        self.specs = specs
        self.x_off, self.y_off, self.x_len, self.nel = [], [], [], []
        xo = yo = 0
        for s in specs:
            B, S = synth.GEOMETRY[s.fmt]
            nb = synth._nblocks(s.fmt, s.shape)
            n = int(np.prod(s.shape))
            self.x_off.append(xo)
            self.y_off.append(yo)
            self.x_len.append(nb * S)
            self.nel.append(n)
            xo += (nb * S + ALIGN - 1) // ALIGN * ALIGN
            yo += (n * 2 + ALIGN - 1) // ALIGN * ALIGN
        self.x_total, self.y_total = xo, yo
        self.bytes_in = sum(self.x_len)
        self.bytes_out = 2 * sum(self.nel)
        self.elements = sum(self.nel)

    def fill_host(self, x_host_np):
        t0 = time.time()
        for i, s in enumerate(self.specs):
            x_host_np[self.x_off[i]:self.x_off[i] + self.x_len[i]] = synth.payload(s.fmt, s.shape, s.seed)
        return time.time() - t0


# --------------------------------------------------------------------------
# clocks during the timed region
# --------------------------------------------------------------------------
class ClockSampler:
    QUERY = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
             "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
             "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, gpu_id: str | None):
        self.gpu_id = gpu_id
        self.proc = None
        self.lines: list[str] = []
        self.thread = None

    def start(self):
        cmd = ["nvidia-smi", f"--query-gpu={self.QUERY}", "--format=csv,noheader,nounits", "-lms", "200"]
        if self.gpu_id:
            cmd.insert(1, f"--id={self.gpu_id}")
        try:
            self.proc = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
        except OSError:
            self.proc = None
            return
        self.thread = threading.Thread(target=self._read, daemon=True)
        self.thread.start()
        time.sleep(0.3)

    def _read(self):
        for line in self.proc.stdout:
            self.lines.append(line.strip())

    def stop(self):
        if not self.proc:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["nvidia-smi unavailable"]}
        time.sleep(0.25)
        self.proc.terminate()
        try:
            self.proc.wait(timeout=5)
        except subprocess.TimeoutExpired:
            self.proc.kill()
        self.thread.join(timeout=5)
        sm, smax, reasons, power = [], [], set(), []
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for ln in self.lines:
            f = [c.strip() for c in ln.split(",")]
            if len(f) < 9:
                continue
            try:
                sm.append(float(f[1]))
                smax.append(float(f[2]))
                power.append(float(f[3]))
            except ValueError:
                continue
            for nm, v in zip(names, f[5:9]):
                if v.lower() == "active":
                    reasons.add(nm)
        return {"sm_mhz": statistics.median(sm) if sm else None, "sm_max_mhz": max(smax) if smax else None,
                "reasons": sorted(reasons), "samples": len(sm),
                "power_w_max": max(power) if power else None}


# --------------------------------------------------------------------------
# CPU oracle: timed baseline, parity and payload digests
# --------------------------------------------------------------------------
_OUT_BYTES = {"float32": 4, "float16": 2, "bfloat16": 2, "float64": 8}
_BITS = {"float32": np.uint32, "float64": np.uint64, "float16": np.uint16, "bfloat16": np.uint16}


def oracle_pieces(tensors, fraction: int, cores: int, out: str = "bfloat16", per_core: int = 8):
    """Disjoint block ranges of about equal size covering the first
    1/fraction of every tensor's blocks (at least one block each), so that
    `cores` threads, each running the single-threaded oracle on one range at
    a time, finish together.  tensors: [(fmt, shape, payload)].  Returns
    (pieces [(fmt, shape, x, b0, b1)], bytes in+out, elements)."""
    rows = []
    for fmt, shape, x in tensors:
        B, S = synth.GEOMETRY[fmt]
        take = max(1, synth._nblocks(fmt, shape) // fraction)
        rows.append((fmt, shape, x, take, B, S))
    total = sum(take * B for (_, _, _, take, B, _) in rows)
    target = max(1, total // (cores * per_core))
    pieces, nbytes, nel = [], 0, 0
    for fmt, shape, x, take, B, S in rows:
        step = max(1, target // B)
        for b0 in range(0, take, step):
            b1 = min(take, b0 + step)
            pieces.append((fmt, shape, x, b0, b1))
        nbytes += take * (S + _OUT_BYTES[out] * B)
        nel += take * B
    return pieces, nbytes, nel


def time_oracle(pieces, threads: int, out: str = "bfloat16") -> float:
    """Seconds for the oracle, unchanged, to decode every piece: one thread
    per piece at a time on `threads` host threads (ctypes releases the GIL
    during each call)."""
    import oracle

    oracle.build()

    def run(p):
        fmt, shape, x, b0, b1 = p
        oracle.decode_range(fmt, shape, x, b0, b1, out)

    t0 = time.perf_counter()
    if threads == 1:
        for p in pieces:
            run(p)
    else:
        with cf.ThreadPoolExecutor(threads) as ex:
            list(ex.map(run, pieces))
    return time.perf_counter() - t0


def oracle_figures(tensors, cores: int, out: str, one_core_elements: int = 1 << 24):
    """The oracle timed on `cores` threads over all of `tensors`, and on one
    core over a leading sample of about `one_core_elements` elements."""
    pieces, nbytes, nel = oracle_pieces(tensors, 1, cores, out)
    secs = time_oracle(pieces, cores, out)
    total = sum(int(np.prod(shape)) for (_, shape, _) in tensors)
    frac1 = max(1, total // one_core_elements)
    p1, b1, n1 = oracle_pieces(tensors, frac1, 1, out, per_core=1)
    s1 = time_oracle(p1, 1, out)
    return {"cores": cores, "GB/s": round(nbytes / secs / 1e9, 3), "elements/s": float(f"{nel / secs:.4g}"),
            "seconds": round(secs, 3),
            "1_core": {"GB/s": round(b1 / s1 / 1e9, 3), "elements/s": float(f"{n1 / s1:.4g}"),
                       "seconds": round(s1, 3),
                       "sample": f"first 1/{frac1} of every tensor's blocks ({n1} elements)"}}


def nan_mask(bits: np.ndarray, out: str) -> np.ndarray:
    if out == "float32":
        return (bits & 0x7F800000 == 0x7F800000) & (bits & 0x007FFFFF != 0)
    if out == "float64":
        return (bits & 0x7FF0000000000000 == 0x7FF0000000000000) & (bits & 0x000FFFFFFFFFFFFF != 0)
    if out == "float16":
        return (bits & 0x7C00 == 0x7C00) & (bits & 0x03FF != 0)
    return (bits & 0x7F80 == 0x7F80) & (bits & 0x007F != 0)


def count_mismatches(got: np.ndarray, want: np.ndarray, out: str) -> int:
    """Elements whose bits differ (NaN only needs to be NaN: its payload is
    unspecified)."""
    g, w = got.reshape(-1).view(_BITS[out]), want.reshape(-1).view(_BITS[out])
    if g.shape != w.shape:
        return max(g.size, w.size)
    if np.array_equal(g, w):
        return 0
    gn, wn = nan_mask(g, out), nan_mask(w, out)
    return int(((gn != wn) | (~wn & (g != w))).sum())


def parity_against_oracle(pool, tensors, fetch, out: str, cores: int):
    """Every element of every tensor's GPU output against the oracle's
    decode of the same payload, one tensor at a time (host memory holds one
    decoded tensor); each tensor's blocks are split over the pool.
    tensors: [(fmt, shape, payload)]; fetch(i) returns tensor i's GPU output
    bits as a flat numpy array."""
    import oracle

    oracle.build()
    total = bad = 0
    bad_tensors = []
    for i, (fmt, shape, x) in enumerate(tensors):
        got = fetch(i)
        B, _ = synth.GEOMETRY[fmt]
        pieces, _, _ = oracle_pieces([(fmt, shape, x)], 1, cores, out, per_core=2)

        def check(p, got=got, B=B):
            f, shp, xx, b0, b1 = p
            want = oracle.decode_range(f, shp, xx, b0, b1, out)
            return count_mismatches(got[b0 * B:b1 * B], want, out)

        m = sum(pool.map(check, pieces))
        total += got.size
        bad += m
        if m:
            bad_tensors.append(i)
    return {"bit_exact": bad == 0, "elements": total, "mismatches": bad, "tensors": len(tensors),
            "tensors_with_mismatches": bad_tensors[:16]}


def payload_digests(pool, payloads):
    """SHA-256 of every payload, and of the list of those digests (in order)."""
    digs = list(pool.map(lambda x: hashlib.sha256(memoryview(np.ascontiguousarray(x))).hexdigest(), payloads))
    return digs, hashlib.sha256("".join(digs).encode()).hexdigest()


# --------------------------------------------------------------------------
# our arm
# --------------------------------------------------------------------------
def kernel_source_sha() -> str:
    """Hash of the decode kernel's sources (device code, launcher, shared header)."""
    h = hashlib.sha256()
    for f in ("ndq_device.cuh", "ndq_kernels.cu", "ndq_internal.h"):
        with open(os.path.join(ROOT, "quantized_weight_block_gb300", "csrc", f), "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def profiled_traffic(profile_name: str, algorithmic_bytes: int):
    """DRAM bytes per launch from a committed ncu summary, if it was taken on
    the current kernel source for a launch of these algorithmic bytes;
    otherwise None."""
    p = os.path.join(ROOT, "profiles", profile_name)
    try:
        with open(p) as f:
            d = json.load(f)
        if d.get("kernel_src_sha256") == kernel_source_sha() and d.get("algorithmic_bytes_per_launch") == algorithmic_bytes:
            return d.get("dram_bytes_per_launch")
    except Exception:
        pass
    return None


def host_bits(torch, y):
    """A device tensor's bits as a flat host numpy array."""
    t = y.reshape(-1).cpu()
    if t.element_size() == 2:
        return t.view(torch.int16).numpy().view(np.uint16)
    return t.numpy()


def time_single_workloads(torch, ndq, stream, peak, workloads, pool=None, cores=1, oracle_legs=True):
    """Single-format workloads.

    Steady state: back-to-back launches rotating over enough copies of the
    payload and output that the rotation's working set exceeds 4x L2, so no
    launch finds its data in L2.  Single launch: one launch after L2 was
    evicted by a 512 MB read (L2 left full of clean lines), which adds the
    launch and pipeline-fill latency.  With oracle_legs: the payload's
    SHA-256, the parity of the whole GPU output against the oracle, and the
    oracle itself timed on the same payload (all host cores, and one core on
    a sample).
    """
    l2 = int(getattr(torch.cuda.get_device_properties(torch.cuda.current_device()), "L2_cache_size", 0) or 132 << 20)
    flush = torch.ones(512 << 20, dtype=torch.uint8, device="cuda")
    flush_sink = torch.empty((), dtype=torch.uint8, device="cuda")
    out = {}
    tdt = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
    for label, fmt, shape, seed, od in workloads:
        x_np = synth.payload(fmt, shape, seed)
        nbytes = x_np.size + int(np.prod(shape)) * torch.empty((), dtype=tdt[od]).element_size()
        nsets = int(min(64, max(2, -(-4 * l2 // nbytes))))
        x0 = torch.from_numpy(x_np).cuda()
        xs = [x0] + [x0.clone() for _ in range(nsets - 1)]
        ys = [torch.empty(shape, dtype=tdt[od], device="cuda") for _ in range(nsets)]
        # the C ABI with prepared arguments, so that host overhead per call
        # stays below the kernel time even for the 10 us launches
        call = ndq._lib.ndq_dequantize_packed
        fid, oc = ndq.format_id(fmt), ndq.out_dtype_code(tdt[od])
        sa = (ctypes.c_int64 * len(shape))(*shape)
        sh = int(stream.cuda_stream)
        args = [(fid, sa, len(shape), oc, xs[i].data_ptr(), x_np.size, ys[i].data_ptr(), sh) for i in range(nsets)]

        def launch(i):
            rc = call(*args[i])
            if rc:
                raise ndq.NdqError(rc)

        for i in range(nsets):
            launch(i)
        reps = max(40, 2 * nsets)
        torch.cuda.synchronize()
        a = torch.cuda.Event(enable_timing=True)
        b = torch.cuda.Event(enable_timing=True)
        a.record(stream)
        for r in range(reps):
            launch(r % nsets)
        b.record(stream)
        b.synchronize()
        ms = a.elapsed_time(b) / reps
        single = []
        for r in range(12):
            flush_sink.copy_(flush.max())
            a.record(stream)
            launch(r % nsets)
            b.record(stream)
            b.synchronize()
            single.append(a.elapsed_time(b))
        ms1 = statistics.median(single)
        extra = {}
        if oracle_legs and pool is not None:
            torch.cuda.synchronize()
            tensors = [(fmt, shape, x_np)]
            extra["payload_sha256"] = hashlib.sha256(memoryview(x_np)).hexdigest()
            extra["parity"] = parity_against_oracle(pool, tensors, lambda i: host_bits(torch, ys[0]), od, cores)
            extra["oracle"] = oracle_figures(tensors, cores, od)
        gbs = nbytes / (ms * 1e-3) / 1e9
        out[label] = {"GB/s": round(gbs, 1), "ms": round(ms, 5), "elements/s": float(f"{np.prod(shape) / (ms * 1e-3):.4g}"),
                      "frac_of_8TBs": round(gbs / 8000.0, 4), "frac_of_measured": round(gbs / peak, 4),
                      "bytes": nbytes,
                      "l2": f"back to back over {nsets} buffer sets ({nsets * nbytes / 1e6:.0f} MB > 4x L2)",
                      "single_launch_ms": round(ms1, 5),
                      "single_launch_GB/s": round(nbytes / (ms1 * 1e-3) / 1e9, 1), **extra}
        del xs, ys, x0
    del flush, flush_sink
    return out


def time_fused_matmul(torch, ndq, stream, work, x_dev, y_dev, reps=20):
    """Decode fused into its consumer (ndq_matmul_packed), M = 1 activation
    row: one generation step of the whole model (one fused product per
    weight tensor, 225 launches replayed as a CUDA graph) against the
    unfused path on the same payloads (the batched decode to bf16, then one
    cuBLAS bf16 product per tensor, also as a graph).  Also single tensors
    at M = 1, 4 and 8 with the exact binary32 weights (the lean CUDA-core
    kernels where K <= 4096; the [4096,14336] q6_k down projection at M > 1
    on the tensor cores, the group scales applied after the tensor core's
    per-group sums) and M = 8 with bfloat16 weights."""
    specs = work.specs
    ks = sorted({s.shape[1] for s in specs})
    xs = {k: torch.randn(1, k, device="cuda").to(torch.bfloat16) for k in ks}
    n_out = sum(s.shape[0] for s in specs)
    y_f = torch.empty(n_out, dtype=torch.float32, device="cuda")
    y_u = torch.empty(n_out, dtype=torch.bfloat16, device="cuda")
    views, wviews = [], []
    o = 0
    for i, s in enumerate(specs):
        N, K = s.shape
        views.append((s.fmt, x_dev[work.x_off[i]:work.x_off[i] + work.x_len[i]], N, K, y_f[o:o + N].view(1, N),
                      y_u[o:o + N].view(1, N)))
        wviews.append(y_dev[work.y_off[i] // 2:work.y_off[i] // 2 + work.nel[i]].view(N, K))
        o += N

    def fused():
        for fmt, w, N, K, yf, _ in views:
            ndq.matmul_packed(fmt, w, N, K, xs[K], y=yf)

    # the products of a layer that read the same activations (q, k and v;
    # gate and up) as one batched call each
    groups, cur = [], []
    for i, s in enumerate(specs):
        key = s.name.rsplit(".", 1)[0] + (".qkv" if s.name.endswith((".q", ".k", ".v")) else
                                          ".gu" if s.name.endswith((".gate", ".up")) else f".{i}")
        if cur and cur[0][0] == key:
            cur.append((key, i))
        else:
            if cur:
                groups.append([j for _, j in cur])
            cur = [(key, i)]
    groups.append([j for _, j in cur])

    def fused_grouped():
        for g in groups:
            if len(g) == 1:
                fmt, w, N, K, yf, _ = views[g[0]]
                ndq.matmul_packed(fmt, w, N, K, xs[K], y=yf)
            else:
                K = views[g[0]][3]
                ndq.matmul_packed_batched([(views[j][0], views[j][1], views[j][2], views[j][4]) for j in g], K, xs[K])

    def gemvs():
        for (fmt, w, N, K, _, yu), wb in zip(views, wviews):
            torch.matmul(xs[K], wb.t(), out=yu)

    def decode():
        ndq.dequantize_packed_batched([(s.fmt, s.shape, views[i][1], wviews[i]) for i, s in enumerate(specs)])

    def graph_of(fn):
        fn()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        return g

    def graph_timed(fn, n=10):
        # n calls captured in one CUDA graph and replayed, so that the
        # Python wrapper's host time does not pace the short launches
        g = torch.cuda.CUDAGraph()
        fn()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for _ in range(n):
                fn()
        return timed(g.replay) / n

    def timed(fn, n=reps):
        for _ in range(3):
            fn()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(stream)
        for _ in range(n):
            fn()
        b.record(stream)
        b.synchronize()
        return a.elapsed_time(b) / n

    g_fused, g_gemv = graph_of(fused), graph_of(gemvs)
    t_f = timed(g_fused.replay)
    y_single = y_f.clone()
    g_grouped = graph_of(fused_grouped)
    t_fg = timed(g_grouped.replay)
    same = bool(torch.equal(y_f.view(torch.int32), y_single.view(torch.int32)))
    t_g = timed(g_gemv.replay)
    t_d = timed(decode)
    whole = {"fused_ms": round(t_f, 4), "unfused_ms": round(t_d + t_g, 4), "unfused_decode_ms": round(t_d, 4),
             "unfused_cublas_ms": round(t_g, 4), "speedup": round((t_d + t_g) / t_f, 3),
             "launches": len(specs), "payload_GB/s": round(work.bytes_in / (t_f * 1e-3) / 1e9, 1),
             "weights/s": float(f"{work.elements / (t_f * 1e-3):.4g}"),
             "what": "one generation step (M=1) over all 225 weight tensors, each a CUDA graph of per-tensor launches",
             "grouped": {"fused_ms": round(t_fg, 4), "launches": len(groups), "speedup": round((t_d + t_g) / t_fg, 3),
                         "payload_GB/s": round(work.bytes_in / (t_fg * 1e-3) / 1e9, 1),
                         "outputs_equal_per_tensor_launches": same,
                         "what": "the same step with the products that share activations (q, k, v; gate, up) as one "
                                 "ndq_matmul_packed_batched call each: 4 launches per layer"}}

    single = {}
    for fmt, N, K in (("gguf:q4_k", 4096, 4096), ("gguf:q6_k", 14336, 4096), ("gguf:q6_k", 4096, 14336),
                      ("gguf:q8_0", 128256, 4096)):
        i = next(j for j, s in enumerate(specs) if s.fmt == fmt and s.shape == (N, K))
        w, wb = views[i][1], wviews[i]
        for M, wdt in ((1, torch.float32), (4, torch.float32), (8, torch.float32), (8, torch.bfloat16)):
            x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
            yf = torch.empty(M, N, device="cuda")
            yb = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
            tf = graph_timed(lambda: ndq.matmul_packed(fmt, w, N, K, x, y=yf, weight_dtype=wdt))
            tu = graph_timed(lambda: (ndq.dequantize_packed(fmt, (N, K), w, torch.bfloat16, y=wb),
                                torch.matmul(x, wb.t(), out=yb)))
            wname = "bfloat16" if wdt == torch.bfloat16 else "binary32"
            if M == 1:
                tag = f"binary32 weights, CUDA cores ({'k_gemvl' if K <= 4096 else 'k_gemvm'})"
            elif wdt == torch.bfloat16 and M >= 6:
                tag = "bfloat16 weights, tensor cores (k_mma)"
            elif K % 512 == 0 and K <= 4096:  # (every format here has lean decoders)
                tag = f"{wname} weights, CUDA cores (k_gemvm)"
            elif fmt in ("gguf:q6_k", "gguf:q8_0"):
                tag = "binary32 weights, grouped tensor cores (k_mmag)"
            else:
                tag = "binary32 weights, CUDA cores (k_matvec)"
            single[f"{fmt.split(':')[-1]}[{N},{K}] M={M} {tag}"] = {
                "fused_us": round(tf * 1e3, 1), "unfused_us": round(tu * 1e3, 1), "speedup": round(tu / tf, 3),
                "payload_GB/s": round(w.numel() / (tf * 1e-3) / 1e9, 1)}
    # bfloat16 weights on the tensor cores (tcgen05) for more activation rows
    tensor = {}
    for fmt, N, K in (("gguf:q4_k", 14336, 4096), ("gguf:q6_k", 14336, 4096), ("gguf:q6_k", 4096, 14336)):
        i = next(j for j, s in enumerate(specs) if s.shape == (N, K) and (s.fmt == fmt or fmt == "gguf:q4_k"))
        w, wb = views[i][1], wviews[i]
        if fmt != specs[i].fmt:  # the model has no q4_k FFN tensor: a payload of that shape
            w = torch.from_numpy(synth.payload(fmt, (N, K), 3)).cuda()
        for M in (16, 64, 256, 1024):
            x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
            yf = torch.empty(M, N, device="cuda")
            yb = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
            tf = graph_timed(lambda: ndq.matmul_packed(fmt, w, N, K, x, y=yf, weight_dtype=torch.bfloat16))
            tu = graph_timed(lambda: (ndq.dequantize_packed(fmt, (N, K), w, torch.bfloat16, y=wb),
                                torch.matmul(x, wb.t(), out=yb)))
            tensor[f"{fmt.split(':')[-1]}[{N},{K}] M={M}"] = {
                "fused_us": round(tf * 1e3, 1), "unfused_us": round(tu * 1e3, 1), "speedup": round(tu / tf, 3),
                "TFLOP/s": round(2 * M * N * K / (tf * 1e-3) / 1e12, 1)}
    return {"whole_model_m1": whole, "single": single, "tensor_core_bf16_weights": tensor,
            "l2": "payloads of 5.9 GB per step (whole model); single tensors back to back, 10 launches per CUDA graph "
                  "replay on both sides (the 33-560 MB payload and its decoded copy partly stay in L2)"}


def run_only_fused(args, torch, ndq):
    """One fused decode + product, --warmup untimed then --steps timed launches."""
    fmt, N, K, M, *wt = args.only_fused.split(",")
    N, K, M = int(N), int(K), int(M)
    wdt = torch.bfloat16 if wt and wt[0] == "bf16" else torch.float32
    w = torch.from_numpy(synth.payload(fmt, (N, K), 3)).cuda()
    x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    y = torch.empty(M, N, device="cuda")
    stream = torch.cuda.current_stream()
    for _ in range(args.warmup):
        ndq.matmul_packed(fmt, w, N, K, x, y=y, weight_dtype=wdt)
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(stream)
    for _ in range(args.steps):
        ndq.matmul_packed(fmt, w, N, K, x, y=y, weight_dtype=wdt)
    b.record(stream)
    b.synchronize()
    ms = a.elapsed_time(b) / args.steps
    print(json.dumps({"fused": args.only_fused, "us_per_launch": round(ms * 1e3, 2),
                      "weights/s": float(f"{N * K / (ms * 1e-3):.4g}"),
                      "payload_GB/s": round(w.numel() / (ms * 1e-3) / 1e9, 1), "steps": args.steps,
                      "l2": "back-to-back launches on one payload"}), flush=True)


def run_only(args, torch, ndq):
    """One single-format workload, --warmup untimed then --steps timed
    launches (used for focused profiling of one format)."""
    every = synth.WORKLOADS + synth.NEXT_WORKLOADS
    match = [w for w in every if w[0] == args.only]
    if not match:
        raise SystemExit(f"unknown workload {args.only!r}; choose from {[w[0] for w in every]}")
    label, fmt, shape, seed, od = match[0]
    tdt = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}[od]
    x_np = synth.payload(fmt, shape, seed)
    x = torch.from_numpy(x_np).cuda()
    y = torch.empty(shape, dtype=tdt, device="cuda")
    stream = torch.cuda.current_stream()
    for _ in range(args.warmup):
        ndq.dequantize_packed(fmt, shape, x, tdt, y=y)
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(stream)
    for _ in range(args.steps):
        ndq.dequantize_packed(fmt, shape, x, tdt, y=y)
    b.record(stream)
    b.synchronize()
    ms = a.elapsed_time(b) / args.steps
    nbytes = x_np.size + y.numel() * y.element_size()
    print(json.dumps({"workload": label, "ms_per_step": round(ms, 5), "GB/s": round(nbytes / (ms * 1e-3) / 1e9, 1),
                      "steps": args.steps, "l2": "back-to-back launches (no flush)"}), flush=True)


def end_to_end(args, torch, ndq, work, x_host, x_dev, y_dev, stream, world, step_bytes):
    """Host payloads in, host bf16 weights out, through the public API.

    The model is split into groups of consecutive tensors of about equal
    bytes.  Per group: a host->device copy on one stream, the batched decode
    on a second (after that copy), a device->host copy of the decoded weights
    on a third (after the decode), so the two link directions and the decode
    overlap.  Every byte of every payload and every decoded weight crosses the
    link once per step.
    """
    # Pinned buffers of this leg are allocated here, after everything else: a
    # pinned buffer allocated earlier in the process was measured to lose
    # most of its host->device bandwidth once later pinned buffers exist.
    x_src = x_host
    x_host = torch.empty(work.x_total, dtype=torch.uint8, pin_memory=True)
    x_host.copy_(x_src)
    y_host = torch.empty(work.y_total // 2, dtype=torch.bfloat16, pin_memory=True)
    ngroups = args.e2e_groups
    target = work.x_total / ngroups
    groups, cur, acc = [], [], 0
    for i in range(len(work.specs)):
        cur.append(i)
        acc += work.x_len[i]
        if acc >= target * (len(groups) + 1) or i == len(work.specs) - 1:
            groups.append(cur)
            cur = []
    s_h2d, s_dec, s_d2h = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()
    gdescs, gws = [], []
    for g in groups:
        items = []
        for i in g:
            s = work.specs[i]
            xv = x_dev[work.x_off[i]:work.x_off[i] + work.x_len[i]]
            yv = y_dev[work.y_off[i] // 2:work.y_off[i] // 2 + work.nel[i]].view(s.shape)
            items.append(ndq.make_desc(s.fmt, s.shape, xv, yv))
        gdescs.append((ndq.ndq_tensor_desc * len(items))(*items))
        nb = ndq.ndq_batched_workspace_bytes(len(items))
        gws.append((torch.empty(max(16, nb), dtype=torch.uint8, device="cuda"), nb))

    def span(idx, off, ln):
        lo = min(off[i] for i in idx)
        hi = max(off[i] + ln(i) for i in idx)
        return lo, hi

    xr = [span(g, work.x_off, lambda i: work.x_len[i]) for g in groups]
    yr = [span(g, work.y_off, lambda i: 2 * work.nel[i]) for g in groups]

    def one_step():
        start = torch.cuda.Event()
        start.record(stream)
        for st in (s_h2d, s_dec, s_d2h):
            st.wait_event(start)
        for gi, g in enumerate(groups):
            lo, hi = xr[gi]
            with torch.cuda.stream(s_h2d):
                x_dev[lo:hi].copy_(x_host[lo:hi], non_blocking=True)
                eh = torch.cuda.Event()
                eh.record(s_h2d)
            s_dec.wait_event(eh)
            ws, nb = gws[gi]
            rc = ndq._lib.ndq_dequantize_packed_batched(gdescs[gi], len(g), ws.data_ptr(), nb,
                                                        int(s_dec.cuda_stream))
            if rc:
                raise ndq.NdqError(rc)
            ed = torch.cuda.Event()
            ed.record(s_dec)
            s_d2h.wait_event(ed)
            ylo, yhi = yr[gi]
            with torch.cuda.stream(s_d2h):
                y_host[ylo // 2:yhi // 2].copy_(y_dev[ylo // 2:yhi // 2], non_blocking=True)
        for st in (s_h2d, s_dec, s_d2h):
            ev = torch.cuda.Event()
            ev.record(st)
            stream.wait_event(ev)

    for _ in range(2):  # warm: first touches of pinned pages are slower
        one_step()
    torch.cuda.synchronize()
    # link bandwidth alone, for the log
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(stream)
    x_dev.copy_(x_host, non_blocking=True)
    b.record(stream)
    b.synchronize()
    h2d_gbs = work.x_total / (a.elapsed_time(b) * 1e-3) / 1e9
    a.record(stream)
    y_host.copy_(y_dev, non_blocking=True)
    b.record(stream)
    b.synchronize()
    d2h_gbs = work.y_total / (a.elapsed_time(b) * 1e-3) / 1e9
    log(f"[bench] pinned host<->device alone: H2D {h2d_gbs:.1f} GB/s, D2H {d2h_gbs:.1f} GB/s")

    if world > 1:
        torch.distributed.barrier()
    e_steps = max(1, args.e2e_steps)
    a.record(stream)
    for _ in range(e_steps):
        one_step()
    b.record(stream)
    b.synchronize()
    e_ms = max_over_ranks(a.elapsed_time(b) / e_steps, "cuda")
    del y_host, x_host
    return {"value": round(job_gbs(step_bytes, world, e_ms), 2), "unit": "GB/s",
            "ms_per_step": round(e_ms, 3), "steps": e_steps,
            "h2d_bytes_per_step": work.x_total, "d2h_bytes_per_step": work.y_total,
            "link_alone_GB/s": {"h2d": round(h2d_gbs, 1), "d2h": round(d2h_gbs, 1)},
            "gpu_launches_per_step": sum(batched_launches(len(g)) for g in groups),
            "path": f"pinned host payloads -> H2D copy -> ndq_dequantize_packed_batched -> D2H copy of the bf16 "
                    f"weights, {len(groups)} groups of tensors pipelined over 3 streams"}


def run_ours(args, rank, world, local_rank):
    import torch

    import quantized_weight_block_gb300 as ndq

    torch.cuda.set_device(local_rank)
    if world > 1:
        import torch.distributed as dist

        dist.init_process_group("nccl", device_id=torch.device("cuda", local_rank))
    peak, peak_src = measured_peaks()
    if args.only:
        return run_only(args, torch, ndq)
    if args.only_fused:
        return run_only_fused(args, torch, ndq)
    specs = synth.llama3_8b_tensors()
    if args.layers != 32 or args.no_embedding:
        specs = [t for t in specs if (t.name.startswith("layers.") and int(t.name.split(".")[1]) < args.layers)
                 or (t.name == "embed" and not args.no_embedding)]
    work = ModelWorkload(specs)

    # host payloads (pinned, for the end-to-end leg and the CPU baseline)
    x_host = torch.empty(work.x_total, dtype=torch.uint8, pin_memory=True)
    gen_s = work.fill_host(x_host.numpy())
    log(f"[bench] generated {work.bytes_in / 1e9:.2f} GB of payloads in {gen_s:.1f}s")

    x_dev = torch.empty(work.x_total, dtype=torch.uint8, device="cuda")
    y_dev = torch.empty(work.y_total // 2, dtype=torch.bfloat16, device="cuda")
    x_dev.copy_(x_host)
    items = []
    for i, s in enumerate(work.specs):
        xv = x_dev[work.x_off[i]:work.x_off[i] + work.x_len[i]]
        yv = y_dev[work.y_off[i] // 2:work.y_off[i] // 2 + work.nel[i]].view(s.shape)
        items.append(ndq.make_desc(s.fmt, s.shape, xv, yv))
    descs = (ndq.ndq_tensor_desc * len(items))(*items)
    ws_bytes = ndq.ndq_batched_workspace_bytes(len(items))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream()
    sh = int(stream.cuda_stream)
    lib = ndq._lib

    def step():
        rc = lib.ndq_dequantize_packed_batched(descs, len(items), ws.data_ptr(), ws_bytes, sh)
        if rc:
            raise ndq.NdqError(rc)

    for _ in range(args.warmup):
        step()
    torch.cuda.synchronize()

    props = torch.cuda.get_device_properties(local_rank)
    uuid = getattr(props, "uuid", None)
    sampler = ClockSampler(("GPU-" + str(uuid)) if uuid else None)
    sampler.start()
    if world > 1:
        torch.distributed.barrier()
    torch.cuda.synchronize()
    ev0, ev1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    ev0.record(stream)
    for _ in range(args.steps):
        step()
    ev1.record(stream)
    ev1.synchronize()
    torch.cuda.synchronize()
    if world > 1:
        torch.distributed.barrier()
    clocks = sampler.stop()
    ms = max_over_ranks(ev0.elapsed_time(ev1) / args.steps, "cuda")
    step_bytes = work.bytes_in + work.bytes_out
    value = job_gbs(step_bytes, world, ms)
    if ndq.get_device_fault():
        raise RuntimeError("device fault word set during the timed region")

    cores = os.cpu_count() or 1
    pool = cf.ThreadPoolExecutor(cores)
    x_np = x_host.numpy()
    model_tensors = [(s.fmt, s.shape, x_np[work.x_off[i]:work.x_off[i] + work.x_len[i]])
                     for i, s in enumerate(work.specs)]
    # ---- outside the timed region: the timed launch's whole output against
    # the oracle, and the payloads' digests ----
    parity = digests = None
    if not args.no_parity and rank == 0:
        t0 = time.time()
        digs, combined = payload_digests(pool, [t[2] for t in model_tensors])
        digests = {"whole_model": combined, "tensors": len(digs),
                   "what": "SHA-256 of the concatenated hex SHA-256 digests of every payload, in tensor order",
                   "first": digs[0], "embedding": digs[-1]}

        def fetch(i):
            return host_bits(torch, y_dev[work.y_off[i] // 2:work.y_off[i] // 2 + work.nel[i]])

        parity = parity_against_oracle(pool, model_tensors, fetch, "bfloat16", cores)
        parity["what"] = ("every element of every tensor decoded by the last timed launch, against the oracle's "
                          "decode of the same payload (bf16 bits; NaN only needs to be NaN)")
        log(f"[bench] parity {parity['bit_exact']} ({parity['mismatches']} mismatches) in {time.time() - t0:.1f}s")

    # ---- end to end through the public API with host buffers ----
    e2e = None
    if not args.no_e2e:
        e2e = end_to_end(args, torch, ndq, work, x_host, x_dev, y_dev, stream, world, step_bytes)

    per_workload = per_workload_next = fused = None
    if not args.no_workloads and rank == 0:
        legs = not args.no_parity
        per_workload = time_single_workloads(torch, ndq, stream, peak, synth.WORKLOADS, pool, cores, legs)
        per_workload_next = time_single_workloads(torch, ndq, stream, peak, synth.NEXT_WORKLOADS, pool, cores, legs)
    if not args.no_fused and rank == 0 and not (args.layers != 32 or args.no_embedding):
        fused = time_fused_matmul(torch, ndq, stream, work, x_dev, y_dev)

    cpu = None
    if not args.no_cpu and rank == 0:
        pieces, nbytes, nel = oracle_pieces(model_tensors, args.cpu_fraction, cores)
        secs = time_oracle(pieces, cores)
        frac1 = max(1, work.elements // (1 << 26))
        p1, b1, n1 = oracle_pieces(model_tensors, frac1, 1, per_core=1)
        s1 = time_oracle(p1, 1)
        cpu = {"value": round(nbytes / secs / 1e9, 4), "unit": "GB/s", "cores": cores, "kind": "oracle",
               "elements/s": float(f"{nel / secs:.4g}"), "seconds": round(secs, 2),
               "sample": f"first 1/{args.cpu_fraction} of every tensor's blocks of the same whole-model "
                         f"payloads ({nel} elements, {nbytes / 1e9:.3f} GB in+out), decoded to bf16, "
                         f"{cores} threads over {len(pieces)} disjoint block ranges of about equal size",
               "1_core": {"value": round(b1 / s1 / 1e9, 4), "unit": "GB/s", "elements/s": float(f"{n1 / s1:.4g}"),
                          "seconds": round(s1, 2),
                          "sample": f"first 1/{frac1} of every tensor's blocks ({n1} elements), one thread"}}
    pool.shutdown()

    # (the committed traffic record is for the full model's launch only)
    traffic = profiled_traffic("k_decode_whole_model.json", step_bytes)
    res = {
        "metric": METRIC, "value": round(value, 2), "unit": "GB/s", "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": round(ms, 4), "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "f32", "data": "synthetic (seeded payloads, recipe in synth/)",
        "config": {"workload": WORKLOAD_NAME, "tensors": len(work.specs), "elements": work.elements,
                   "bytes_in": work.bytes_in, "bytes_out": work.bytes_out, "out_dtype": "bf16",
                   "elements/s": float(f"{world * work.elements / (ms * 1e-3):.4g}"),
                   "frac_of_8TBs": round(value / world / 8000.0, 4),
                   "l2": f"inputs larger than L2 ({step_bytes / 1e9:.1f} GB moved per step)",
                   "parallelism": f"replicas x{world}" if world > 1 else "single GPU"},
        "roofline": {"bound": "hbm", "achieved": round(step_bytes / (ms * 1e-3) / 1e9, 1), "peak": peak,
                     "unit": "GB/s", "frac": round(step_bytes / (ms * 1e-3) / 1e9 / peak, 4),
                     "traffic": traffic, "peak_source": peak_src,
                     "kernel": "k_decode (batched; step time includes the launch-table upload kernels, 225 x 64 B)"},
        "parity": parity, "payload_sha256": digests,
        "cpu_baseline": cpu, "e2e": e2e, "gpu_launches": batched_launches(len(items)) * args.steps, "clocks": clocks,
        "per_workload": per_workload, "per_workload_next_formats": per_workload_next, "fused_matmul": fused,
    }
    if world > 1:
        torch.distributed.destroy_process_group()
    if rank == 0:
        log("[bench] details " + json.dumps(res))
        print(result_line(res), flush=True)


# --------------------------------------------------------------------------
# reference arm: the CPU oracle
# --------------------------------------------------------------------------
def run_reference(args, rank, world):
    if rank != 0:
        return
    import oracle

    oracle.build()
    # a bounded sample with the same field distributions: for every tensor,
    # 1/fraction of its rows (at least one), generated from the tensor's seed;
    # 1/16 keeps the 225 calls' fixed cost small against the decode itself
    # (at 1/4096 it was nearly all of a step)
    fraction = 16
    specs = synth.llama3_8b_tensors()
    sample = []
    for s in specs:
        rows = max(1, s.shape[0] // fraction)
        shp = (rows,) + tuple(s.shape[1:])
        sample.append((s.fmt, shp, synth.payload(s.fmt, shp, s.seed)))
    cores = os.cpu_count() or 1
    # disjoint block ranges of about equal size, so that every host thread
    # stays busy to the end of each step (not one thread on the largest tensor)
    pieces, nbytes, nel = oracle_pieces(sample, 1, cores)

    def one(p):
        fmt, shp, x, b0, b1 = p
        oracle.decode_range(fmt, shp, x, b0, b1, "bfloat16")

    ex = cf.ThreadPoolExecutor(cores)

    def step():
        list(ex.map(one, pieces))

    for _ in range(args.warmup):
        step()
    t0 = time.perf_counter()
    for _ in range(args.steps):
        step()
    secs = (time.perf_counter() - t0) / args.steps
    ex.shutdown()
    value = nbytes / secs / 1e9
    res = {
        "impl": "reference", "metric": METRIC, "value": round(value, 4), "unit": "GB/s", "n_gpus": world,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": round(secs * 1e3, 3),
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f32",
        "data": "synthetic (seeded payloads, recipe in synth/)",
        "config": {"workload": WORKLOAD_NAME, "tensors": len(specs), "elements": nel, "bytes": nbytes,
                   "out_dtype": "bf16"},
        "cpu_baseline": {"value": round(value, 4), "unit": "GB/s", "cores": cores, "kind": "oracle",
                         "sample": f"1/{fraction} of every tensor's rows (same field distributions and seeds), "
                                   f"{nel} elements per step, {cores} threads over {len(pieces)} disjoint block "
                                   f"ranges of about equal size"},
        "e2e": {"value": round(value, 4), "unit": "GB/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }
    print(json.dumps(res), flush=True)


def main():
    args = parse_args()
    rank, world, local = dist_env()
    if args.impl == "reference":
        run_reference(args, rank, world)
    else:
        run_ours(args, rank, world, local)


if __name__ == "__main__":
    main()
