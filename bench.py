"""FlashHead throughput on one MI355X: calls/s and achieved HBM GB/s of the
retrieval head at (v=128256, d=2048, c=8016, p=512, bf16, batch 1), beside
the dense head z = E h on the same inputs and the CPU oracle.

One step is one fh_forward call (stage-1 scores, probe selection,
gather-score of the p*b retrieved tokens, argmax epilogue) over one batch of
B synthetic queries.  Inputs are resident in HBM before timing starts.  The
engine is replicated R times (default 16) and consecutive steps rotate over
the replicas and over 256 queries, so that the bytes a call touches are not
still in the 256 MB Infinity Cache from the previous call: the working set
between two uses of one replica is R * (|C| + |E rows read|), several times
the cache.

Output: one JSON line (see the keys below).  --gpus N > 1 is not supported:
this benchmark runs on one GPU.
"""

from __future__ import annotations

import argparse
import ctypes
import hashlib
import json
import os
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

HBM_PEAK_GBS = 8000.0  # MI355X HBM3E, published peak


def parse():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=2000)
    ap.add_argument("--warmup", type=int, default=100)
    ap.add_argument("--shape", default="llama32_1b")
    ap.add_argument("--B", type=int, default=1)
    ap.add_argument("--p", type=int, default=512)
    ap.add_argument("--quant", default="none", choices=["none", "int4", "int8"])
    ap.add_argument("--mode", type=int, default=0)
    ap.add_argument("--temperature", type=float, default=1.0)
    ap.add_argument("--replicas", type=int, default=16)
    ap.add_argument("--dense-steps", type=int, default=200)
    ap.add_argument("--cpu-seconds", type=float, default=12.0)
    ap.add_argument("--no-cpu", action="store_true")
    ap.add_argument("--no-dense", action="store_true")
    ap.add_argument("--path", default="auto", choices=["auto", "multi"],
                    help="auto: one launch per batch-1 call; multi: one per stage")
    ap.add_argument("--cluster", action="store_true",
                    help="time the offline balanced spherical k-means (fh_cluster) at --shape "
                         "instead of the head, one JSON line of its own")
    ap.add_argument("--cluster-iters", type=int, default=5)
    ap.add_argument("--cluster-runs", type=int, default=2)
    ap.add_argument("--sweep", action="store_true",
                    help="latency and agreement with the dense head over B in {1,8,32,64} x p in "
                         "{128,256,512,1024} at --shape / --quant; one JSON line")
    ap.add_argument("--adaptive", type=float, default=None, metavar="TAU",
                    help="with --sweep: also rows of the adaptive probe count (mass TAU at "
                         "--temperature, p_max = --p) on the same queries")
    ap.add_argument("--alpha", type=float, default=None,
                    help="--sweep: query scale on its source token's embedding (default: the "
                         "shape's); smaller is harder for the probes")
    ap.add_argument("--spread", type=float, default=None,
                    help="--sweep: within-cluster noise scale of the embeddings (default 0.3; "
                         "1.3 puts tokens at cosine ~0.6 to their cluster, the pages' quality bound)")
    ap.add_argument("--spec", type=int, default=0, metavar="K",
                    help="time the speculative verification of K draft positions (fh_spec_verify) "
                         "beside K single-position drafts and the dense head at B=K; one JSON line")
    ap.add_argument("--serve", action="store_true",
                    help="time one decode step after the last layer at --shape, --B and --mode: norm, "
                         "int8 dense head, rules on logits (W8A8Head.step), each part and the same step "
                         "on the head in its own dtype; one JSON line")
    ap.add_argument("--burst", action="store_true",
                    help="time the plain one-shot read probe (fhb_read_probe) at the sizes of a "
                         "batch-1 call's phases, the whole call and the dense head; one JSON line")
    ap.add_argument("--copy-calibration", action="store_true",
                    help="only run a plain elementwise copy of known size (to scale the "
                         "FETCH_SIZE / WRITE_SIZE counters of a rocprofv3 --pmc run) and exit")
    return ap.parse_args()


COPY_BYTES = 512 << 20  # per launch of the calibration copy, read and written


def copy_calibration():
    """A plain device copy (torch's elementwise negation, read once, written
    once) of COPY_BYTES, five launches."""
    import torch
    src = torch.ones(COPY_BYTES // 4, dtype=torch.float32, device="cuda")
    dst = torch.empty_like(src)
    for _ in range(5):
        torch.neg(src, out=dst)
    torch.cuda.synchronize()
    print(json.dumps({"copy_kernel": "neg", "bytes_read_per_launch": COPY_BYTES,
                      "bytes_written_per_launch": COPY_BYTES, "launches": 5}), flush=True)


# One-shot read sizes (bytes) of the Llama-3.2-1B-shape head, as the roofline
# table counts them: a batch-1 call's stage 1 and stage 2, the call, the dense head.
BURST_SIZES = (("stage 1", 32_869_696), ("stage 2", 33_593_344), ("batch-1 call", 66_497_152),
               ("dense head", 525_340_672))


def load_bench_lib():
    """bench.py's own library (the plain read probe, fhb_read_probe), built
    beside libflashhead.so by lm_output_head_amd.build."""
    path = os.path.join(ROOT, "lm_output_head_amd", "libflashhead_bench.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build with `python -m lm_output_head_amd.build`")
    lib = ctypes.CDLL(path)
    lib.fhb_read_probe.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32,
                                   ctypes.c_void_p, ctypes.c_void_p]
    lib.fhb_read_probe.restype = ctypes.c_int
    return lib


def burst_main(args):
    """How fast the part streams a buffer of each size in one launch: the
    library's plain read probe over 16 rotating buffers (their 8.4 GB exceed the
    256 MB Infinity Cache, so every launch reads from HBM), timed back to back
    and with a HIP event pair around each launch on its stream.  The timed
    loops call the C ABI with the pointers marshalled beforehand, so that the
    host keeps ahead of launches of a few microseconds."""
    import ctypes

    import torch

    lib = load_bench_lib()
    nbuf, steps = 16, max(50, min(args.steps, 400))
    big = max(n for _, n in BURST_SIZES)
    bufs = [torch.full((big // 4,), i + 1, dtype=torch.int32, device="cuda") for i in range(nbuf)]
    found = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream()
    ptrs = [ctypes.c_void_p(b.data_ptr()) for b in bufs]
    fptr, sptr = ctypes.c_void_p(found.data_ptr()), ctypes.c_void_p(stream.cuda_stream)
    probe = lib.fhb_read_probe
    rows = []
    for what, n in BURST_SIZES:
        for i in range(20):
            assert probe(ptrs[i % nbuf], n, 0, fptr, sptr) == 0
        torch.cuda.synchronize()
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record(stream)
        for i in range(steps):
            probe(ptrs[i % nbuf], n, 0, fptr, sptr)
        t1.record(stream)
        t1.synchronize()
        b2b = t0.elapsed_time(t1) * 1e3 / steps
        ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
              for _ in range(steps)]
        for i, (a0, a1) in enumerate(ev):
            a0.record(stream)
            probe(ptrs[i % nbuf], n, 0, fptr, sptr)
            a1.record(stream)
        torch.cuda.synchronize()
        evu = sum(a0.elapsed_time(a1) for a0, a1 in ev) * 1e3 / steps
        rows.append({"what": what, "bytes": n, "us_back_to_back": round(b2b, 2),
                     "gbs_back_to_back": round(n / b2b / 1e3, 1), "us_per_launch_events": round(evu, 2),
                     "gbs_events": round(n / evu / 1e3, 1), "frac_of_8tbs_back_to_back": round(n / b2b / 8e6, 3)})
    assert int(found.item()) == 0  # the key is absent: every launch read its whole buffer
    print(json.dumps({"metric": "one-shot HBM read probe", "unit": "us per launch", "n_gpus": 1,
                      "steps": steps, "data": "16 rotating device buffers", "peak_gbs": 8000.0,
                      "kernel": "k_read_probe (one 16-byte load per thread, 1024-thread "
                                "workgroups; a search for a 32-bit value absent from the buffers)",
                      "sizes": rows}), flush=True)


def stream_bandwidth(sizes, nbuf=16, steps=100):
    """Back-to-back plain reads (the bench library's read probe) over nbuf
    rotating buffers of each size: the part's streaming rate in GB/s."""
    import ctypes

    import torch

    lib = load_bench_lib()
    stream = torch.cuda.current_stream()
    found = torch.zeros(1, dtype=torch.int32, device="cuda")
    fptr, sptr = ctypes.c_void_p(found.data_ptr()), ctypes.c_void_p(stream.cuda_stream)
    out = {}
    for n in sizes:
        nb = (n // 16) * 16  # the probe reads whole 16-byte words
        bufs = [torch.full((n // 4,), i + 1, dtype=torch.int32, device="cuda") for i in range(nbuf)]
        ptrs = [ctypes.c_void_p(b.data_ptr()) for b in bufs]
        for i in range(nbuf):
            assert lib.fhb_read_probe(ptrs[i], nb, 0, fptr, sptr) == 0
        torch.cuda.synchronize()
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record(stream)
        for i in range(steps):
            lib.fhb_read_probe(ptrs[i % nbuf], nb, 0, fptr, sptr)
        t1.record(stream)
        t1.synchronize()
        us = t0.elapsed_time(t1) * 1e3 / steps
        out[n] = round(nb / us / 1e3, 1)
        del bufs
    assert int(found.item()) == 0
    torch.cuda.empty_cache()
    return out


CLUSTER_SOURCES = ("fh_cluster.hip",)  # the offline clustering, its own translation unit
# the operators around the dense head: no code of theirs runs in a head call
SERVE_SOURCES = ("fh_norm.hip", "fh_w8a8.hip", "fh_rules.hip", "fh_serve.cpp", "fh_serve.hpp",
                 "fh_choice.hpp")


def kernel_source_hash(cluster: bool = False) -> str:
    """Hash of the kernel sources a measurement depends on: the head's (every
    file under csrc/ but the clustering's and the operators' around the dense
    head), or the clustering's."""
    h = hashlib.sha256()
    csrc = os.path.join(ROOT, "lm_output_head_amd", "csrc")
    for name in sorted(os.listdir(csrc)):
        if (name in CLUSTER_SOURCES) != cluster or name in SERVE_SOURCES:
            continue
        with open(os.path.join(csrc, name), "rb") as f:
            h.update(name.encode() + f.read())
    return h.hexdigest()[:16]


def algorithmic_bytes(shape, B, p, quant, elem, union=None):
    """Bytes each kernel must move per launch (the minimum the method reads
    and writes), by kernel name.  `union` is the mean number of distinct
    clusters probed by a batch (B > 1): the cluster-major stage 2 reads each
    of them once."""
    v, d, c, b = shape.v, shape.d, shape.c, shape.b
    if quant == "int4":
        c_bytes = c * d // 2 + c * (d // 32) * 2
    elif quant == "int8":
        c_bytes = c * d + c * (d // 32) * 2
    else:
        c_bytes = c * d * elem
    score = c_bytes + B * d * elem + B * c * 4
    select = B * c * 4 + B * p * 4
    # stage 2: the embedding rows of the retrieved tokens, their C2T entries,
    # the probe lists and h; writes nothing but per-workgroup partials (not
    # counted), the retrieved ids/logits are optional outputs (off here)
    gather = B * p * b * d * elem + B * p * b * 4 + B * p * 4 + B * d * elem
    dense = v * d * elem + B * d * elem
    # cluster-major stage 2: the union's rows and C2T entries, h, the probe
    # bitsets and their prefix counts
    W = (c + 31) // 32
    u = union if union is not None else B * p
    gather_cm = int(round(u * b * (d * elem + 4))) + B * d * elem + 2 * W * B * 4
    call = score + select + (gather_cm if (B > 1 and union is not None) else gather)
    return {"score": score, "score_int4": score, "score_int8": score, "score_mfma": score, "score_int4_mfma": score,
            "select": select, "gather": gather, "gather_cm": gather_cm, "dense": dense,
            "dense_mfma": dense, "batch1": score + select + gather, "batched": select + gather,
            "call": call}


def traffic_from_profiles(kernel: str, src_hash: str, workload_key: str,
                          name: str = "pmc_traffic.json"):
    """HBM bytes per launch measured by rocprofv3 PMC counters, if a summary
    for the current kernel sources and this workload exists under profiles/."""
    path = os.path.join(ROOT, "profiles", name)
    if not os.path.exists(path):
        return None
    try:
        with open(path) as f:
            rec = json.load(f)
    except (OSError, ValueError):
        return None
    if rec.get("source_hash") != src_hash or rec.get("workload_key") != workload_key:
        return None
    k = rec.get("kernels", {}).get(kernel)
    return None if k is None else k.get("bytes_per_launch")


def kernel_us_from_profiles(kernel: str, src_hash: str, workload_key: str, nbytes: int) -> dict:
    """The rocprofv3 kernel-trace mean of `kernel` for this workload, if the
    summary under profiles/ was taken from the current kernel sources."""
    path = os.path.join(ROOT, "profiles", "kernel_times.json")
    try:
        with open(path) as f:
            rec = json.load(f)
    except (OSError, ValueError):
        return {}
    if rec.get("source_hash") != src_hash:
        return {}
    us = rec.get("workloads", {}).get(workload_key, {}).get(kernel)
    if not us:
        return {}
    return {"rocprof_kernel_us": us, "rocprof_frac": round(nbytes / (us * 1e-6) / 1e9 / HBM_PEAK_GBS, 4)}


def cpu_info():
    """The host's CPU model, its BLAS libraries and the thread variables."""
    model = None
    try:
        with open("/proc/cpuinfo") as f:
            for line in f:
                if line.startswith("model name"):
                    model = line.split(":", 1)[1].strip()
                    break
    except OSError:  # pragma: no cover
        pass
    blas = []
    try:
        from threadpoolctl import threadpool_info
        blas = [{"api": i.get("internal_api"), "version": i.get("version"),
                 "threads": i.get("num_threads"), "library": os.path.basename(i.get("filepath", ""))}
                for i in threadpool_info()]
    except Exception:  # pragma: no cover
        pass
    env = {k: os.environ.get(k) for k in ("OMP_NUM_THREADS", "OPENBLAS_NUM_THREADS",
                                          "MKL_NUM_THREADS") if os.environ.get(k) is not None}
    return {"cpu_model": model, "logical_cpus": len(os.sched_getaffinity(0)), "blas": blas,
            "thread_env": env}


def _oracle_rate(head, pb, p, mode, temperature, seconds):
    n = 0
    t0 = time.perf_counter()
    while True:
        q = n % pb.H.shape[0]
        head.forward(pb.H[q:q + 1], p, mode, temperature, 0x5EED + n)
        n += 1
        el = time.perf_counter() - t0
        if el >= seconds:
            return n, el


def cpu_fp32_two_stage(pb, p, seconds):
    """A plain float32 numpy two-stage head (scores, top-p by argpartition,
    gathered rows, argmax) on host cores: what BLAS-speed CPU code does on
    the same workload, greedy top-p only.  Its tokens are certified against
    the float64 oracle on the timed sample."""
    import numpy as np

    import oracle
    E32 = np.ascontiguousarray(pb.E, dtype=np.float32)
    C32 = np.ascontiguousarray(pb.C, dtype=np.float32)
    c2t = np.asarray(pb.C2T)
    H32 = np.asarray(pb.H, dtype=np.float32)

    def call(h):
        s = C32 @ h
        probes = np.argpartition(-s, p - 1)[:p]
        ids = c2t[probes].reshape(-1)
        z = E32[ids] @ h
        return int(ids[int(np.argmax(z))])

    toks, n = [], 0
    t0 = time.perf_counter()
    while True:
        toks.append(call(H32[n % H32.shape[0]]))
        n += 1
        el = time.perf_counter() - t0
        if el >= seconds:
            break
    head = oracle.OracleHead(pb.E, pb.C, pb.C2T)
    m = min(n, H32.shape[0], 32)
    ref = head.forward(pb.H[:m], p).fin.token
    agree = int(sum(int(ref[i]) == toks[i] for i in range(m)))
    return {"value": round(n / el, 3), "unit": "calls/s",
            "sample": f"{n} single-query calls in {el:.1f} s (float32 numpy, E and C widened to float32)",
            "tokens_equal_to_oracle": f"{agree}/{m}"}


def cpu_baseline(pb, p, quant, mode, temperature, seconds):
    """The oracle as it stands, on host cores, over a bounded query sample;
    beside it the same oracle on one thread, a float32 numpy two-stage head
    (greedy top-p), and the host's CPU model and BLAS."""
    import oracle
    try:
        from threadpoolctl import threadpool_info, threadpool_limits
        cores = max([i.get("num_threads", 1) for i in threadpool_info()] + [1])
    except Exception:  # pragma: no cover
        threadpool_limits = None
        cores = os.cpu_count() or 1
    head = oracle.OracleHead(pb.E, pb.C, pb.C2T, quant)
    n, el = _oracle_rate(head, pb, p, mode, temperature, seconds)
    res = {"value": round(n / el, 3), "unit": "calls/s", "cores": int(cores), "kind": "oracle",
           "sample": f"{n} single-query calls of the same workload in {el:.1f} s "
                     f"(float64 numpy oracle, BLAS threads={cores})"}
    if threadpool_limits is not None:
        with threadpool_limits(limits=1):
            n1, el1 = _oracle_rate(head, pb, p, mode, temperature, seconds / 2)
        res["single_thread"] = {"value": round(n1 / el1, 3), "unit": "calls/s",
                                "sample": f"{n1} calls in {el1:.1f} s on one BLAS thread"}
    if quant == "none" and mode == 0:
        res["fp32_two_stage"] = cpu_fp32_two_stage(pb, p, seconds / 2)
    res["dense"] = cpu_dense(pb, seconds / 4)
    res["host"] = cpu_info()
    return res


def cpu_dense(pb, seconds):
    """The dense head on the host: z = E h in float32 numpy (E widened to
    float32: numpy has no bfloat16, so it reads twice the bf16 bytes), then
    the argmax, one query per call."""
    import numpy as np
    E32 = np.ascontiguousarray(pb.E, dtype=np.float32)
    H32 = np.ascontiguousarray(pb.H, dtype=np.float32)
    n = 0
    t0 = time.perf_counter()
    while True:
        int(np.argmax(E32 @ H32[n % H32.shape[0]]))
        n += 1
        el = time.perf_counter() - t0
        if el >= seconds or n >= 200:
            break
    v, d = E32.shape
    return {"value": round(n / el, 3), "unit": "calls/s",
            "sample": f"{n} single-query calls in {el:.2f} s (float32 numpy E h + argmax)",
            "bytes_per_call_read": v * d * 4, "algorithmic_bf16_bytes": v * d * 2}


def cluster_cpu_baseline(E, c, seconds):
    """The clustering oracle on host cores over bounded samples, scaled to
    one whole clustering: k-means++ steps on the full table (each a pass over
    every row) and one iteration's similarities on a block of rows.  The
    balanced rounds and the update are left out, so this underestimates the
    oracle's time."""
    import numpy as np

    from oracle import cluster_oracle as co
    try:
        from threadpoolctl import threadpool_info
        cores = max([i.get("num_threads", 1) for i in threadpool_info()] + [1])
    except Exception:  # pragma: no cover
        cores = os.cpu_count() or 1
    v = E.shape[0]
    Xn = co.normalize_rows(E)
    u = np.random.default_rng(7).random(c)
    t0 = time.perf_counter()
    m = 1
    D = 1.0 - Xn @ Xn[min(int(u[0] * v), v - 1)]
    while time.perf_counter() - t0 < seconds / 2 and m < c:
        t = co.pp_pick(D * D, u[m])
        D = np.minimum(D, 1.0 - Xn @ Xn[t])
        m += 1
    pp_s = (time.perf_counter() - t0) / m * c
    rows = min(v, 4096)
    C = Xn[:c]
    t1 = time.perf_counter()
    _ = Xn[:rows] @ C.T
    sims_s = (time.perf_counter() - t1) * v / rows
    return pp_s, sims_s, {
        "unit": "s per clustering", "cores": int(cores), "kind": "oracle",
        "sample": f"{m} k-means++ steps over all {v} rows and one {rows}-row similarity block "
                  f"(float64 numpy oracle), scaled to {c} centres and {v} rows; the balanced "
                  f"rounds and the update are not included"}


def cluster_main(args):
    """One JSON line: seconds per balanced spherical k-means of the head's
    embedding table (planted clusters, bf16), with the k-means++ phase's
    achieved HBM bandwidth (it reads the table's rows once per centre)."""
    import numpy as np
    import torch

    from lm_output_head_amd import flashhead as fhb
    from synth import SHAPES, make_problem

    if not torch.cuda.is_available():
        print(json.dumps({"error": "no GPU visible"}))
        sys.exit(1)
    shape = SHAPES[args.shape]
    v, d, c = shape.v, shape.d, shape.c
    print(f"[bench] generating {shape.name} table", file=sys.stderr, flush=True)
    pb = make_problem(shape, nq=1)
    if shape.dtype == "bf16":
        E = torch.from_numpy(pb.E_bits.view(np.int16)).view(torch.bfloat16).cuda()
    else:
        E = torch.from_numpy(np.ascontiguousarray(pb.E, dtype=np.float32)).cuda()
    u = np.random.default_rng(7).random(c)
    C = torch.empty((c, d), dtype=torch.float32, device="cuda")
    c2t = torch.empty((c, v // c), dtype=torch.int32, device="cuda")
    asg = torch.empty(v, dtype=torch.int32, device="cuda")
    runs = []
    for i in range(max(1, args.cluster_runs)):
        print(f"[bench] clustering run {i}", file=sys.stderr, flush=True)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        tm = fhb.fh_cluster(E, c, args.cluster_iters, u, C, c2t, None, asg)
        torch.cuda.synchronize()
        tm["wall_s"] = time.perf_counter() - t0
        runs.append(tm)
    best = min(runs, key=lambda r: r["total_ms"])
    truth = np.empty(v, dtype=np.int64)
    truth[pb.C2T.ravel()] = np.repeat(np.arange(c), v // c)
    from oracle import cluster_oracle as co  # quality figures of the result
    got = asg.cpu().numpy()
    ari = co.adjusted_rand_index(got, truth)
    elem = 2 if shape.dtype == "bf16" else 4
    # one k-means++ distance refresh (k_pp_step): the table's rows in their
    # storage type, the inverse norms, D read and written, one fp64 partial
    # per 4-row workgroup
    step_bytes = v * d * elem + v * 4 * 3 + ((v + 3) // 4) * 8
    step_gbs = step_bytes / (best["pp_step_us"] * 1e-6) / 1e9
    init_gbs = c * step_bytes / (best["init_ms"] * 1e-3) / 1e9
    workload_key = f"cluster/{shape.name}"
    traffic = traffic_from_profiles("k_pp_step", kernel_source_hash(cluster=True), workload_key,
                                    name="cluster_pmc_traffic.json")
    sims_tflops = 2.0 * v * c * d * args.cluster_iters / (best["sims_ms"] * 1e-3) / 1e12
    res = {
        "metric": "balanced k-means s per clustering", "value": round(best["total_ms"] / 1e3, 4),
        "unit": "s", "n_gpus": 1, "steps": len(runs), "warmup": 0,
        "ms_per_step": round(best["total_ms"], 2), "higher_is_better": False, "scaling": "weak",
        "vs_baseline": None, "dtype": "f32", "data": "synthetic planted clusters",
        "config": {"workload": f"{shape.name} table v={v} d={d} c={c} b={v // c}, "
                               f"{args.cluster_iters} iterations, {shape.dtype} input"},
        "phases_ms": {"kmeanspp": round(best["init_ms"], 2), "sims": round(best["sims_ms"], 2),
                      "rounds_and_update": round(best["total_ms"] - best["init_ms"]
                                                 - best["sims_ms"], 2)},
        "rounds": best["rounds"],
        "roofline": {"bound": "hbm", "achieved": round(step_gbs, 1), "peak": HBM_PEAK_GBS,
                     "unit": "GB/s", "frac": round(step_gbs / HBM_PEAK_GBS, 4),
                     "traffic": traffic, "kernel": "k_pp_step",
                     "algorithmic_bytes": step_bytes,
                     "avg_launch_us": round(best["pp_step_us"], 2)},
        "kmeanspp_phase_gbs": round(init_gbs, 1),
        "sims_tflops_f32": round(sims_tflops, 2),
        "quality": {"ari_vs_planted": round(ari, 5)},
    }
    if not args.no_cpu:
        print("[bench] timing the clustering oracle", file=sys.stderr, flush=True)
        pp_s, sims_s, base = cluster_cpu_baseline(pb.E.astype(np.float64), c, args.cpu_seconds)
        base["value"] = round(pp_s + sims_s * args.cluster_iters, 2)
        res["cpu_baseline"] = base
    print(json.dumps(res), flush=True)


def sweep_main(args):
    """The accuracy/latency curve against the dense head: for every (B, p),
    the per-call latency (HIP events over rotated engine replicas, as in the
    default run) and, over all generated queries, the top-1 agreement of
    FlashHead's argmax with the dense head's and the recall of the dense
    argmax's cluster among the probes (greedy calls)."""
    import numpy as np
    import torch

    from lm_output_head_amd import flashhead as fhb
    from synth import SHAPES, make_problem

    if not torch.cuda.is_available():
        print(json.dumps({"error": "no GPU visible"}))
        sys.exit(1)
    shape = SHAPES[args.shape]
    import dataclasses
    if args.alpha is not None:
        shape = dataclasses.replace(shape, alpha=float(args.alpha))
    if args.spread is not None:
        shape = dataclasses.replace(shape, spread=float(args.spread))
    Bs, ps = (1, 8, 32, 64), (128, 256, 512, 1024)
    pb = make_problem(shape)
    bf16 = shape.dtype == "bf16"

    def dev(x):
        a = np.ascontiguousarray(x)
        if bf16:
            return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()
        return torch.from_numpy(a.astype(np.float32)).cuda()

    E0, C0 = dev(pb.E_bits if bf16 else pb.E), dev(pb.C_bits if bf16 else pb.C)
    Hall = dev(pb.H_bits if bf16 else pb.H)
    nq = Hall.shape[0]
    R = max(1, min(args.replicas, 8))
    heads = [fhb.FlashHead(E0 if r == 0 else E0.clone(), C0 if r == 0 else C0.clone(), pb.C2T,
                           quant=args.quant, max_batch=max(Bs)) for r in range(R)]
    stream = torch.cuda.current_stream()
    lib = fhb._abi.load()
    sp = ctypes.c_void_p(stream.cuda_stream)
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    otok = torch.empty(max(Bs), dtype=torch.int32, device="cuda")
    olog = torch.empty(max(Bs), dtype=torch.float32, device="cuda")
    olse = torch.empty(max(Bs), dtype=torch.float32, device="cuda")

    def timed_us(B, call, steps):
        hts = [Hall[(i * B) % nq:(i * B) % nq + B].contiguous() for i in range(max(1, nq // B))]
        hp = [ptr(h) for h in hts]

        def fn(i):
            st = call(heads[i % R].eng, hp[i % len(hp)], B, i)
            if st != 0:
                raise RuntimeError(lib.fh_last_error().decode())
        for i in range(10):
            fn(i)
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(stream)
        for i in range(steps):
            fn(10 + i)
        b.record(stream)
        torch.cuda.synchronize()
        return a.elapsed_time(b) / steps * 1e3

    # dense tokens of every query, and the cluster of every token
    t2c = np.empty(shape.v, dtype=np.int64)
    t2c[pb.C2T.ravel()] = np.arange(shape.v) // shape.b
    dense_tok = np.concatenate([heads[0].dense(Hall[i:i + 64])["token"].cpu().numpy()
                                for i in range(0, nq, 64)])
    shared = bool(args.mode & 4)  # one probe set per batch: agreement depends on B

    def agreement(p, chunk):
        toks, hits = [], []
        for i in range(0, nq, chunk):
            o = heads[0].forward(Hall[i:i + chunk], p, mode=args.mode & 4, want_clusters=True)
            toks.append(o["token"].cpu().numpy())
            cl = o["clusters"].cpu().numpy()
            dt = dense_tok[i:i + chunk]
            hits.append(np.array([t2c[t] in set(cl[j].tolist()) for j, t in enumerate(dt)]))
        return float((np.concatenate(toks) == dense_tok).mean()), float(np.concatenate(hits).mean())

    rows = []
    for p in ps:
        if not shared:
            agree, recall = agreement(p, 64)
        for B in Bs:
            if shared:
                agree, recall = agreement(p, B)
            steps = max(50, 800 // B)
            us = timed_us(B, lambda e, h, b, i: lib.fh_forward(e, h, b, p, args.mode & 4, 1.0, 0x5EED + i,
                                                                ptr(otok), ptr(olog), ptr(olse),
                                                                None, None, None, sp), steps)
            rows.append({"B": B, "p": p, "us_per_call": round(us, 2),
                         "tokens_per_s": round(B / (us * 1e-6), 1),
                         "top1_agreement": round(agree, 4), "cluster_recall": round(recall, 4)})
            print(f"[bench] B={B} p={p} {us:.1f} us agree {agree:.3f}", file=sys.stderr, flush=True)
    adaptive = []
    if args.adaptive is not None:
        tau, T, pmax = float(args.adaptive), float(args.temperature), int(args.p)
        toks, hits, ns = [], [], []
        for i in range(0, nq, 64):
            o = heads[0].forward_adaptive(Hall[i:i + 64], pmax, tau, mode=0, temperature=T,
                                          want_clusters=True)
            toks.append(o["token"].cpu().numpy())
            ns.append(o["nprobe"].cpu().numpy())
            cl = o["clusters"].cpu().numpy()
            dt = dense_tok[i:i + 64]
            hits.append(np.array([t2c[t] in set(cl[j].tolist()) for j, t in enumerate(dt)]))
        ns = np.concatenate(ns)
        agree = float((np.concatenate(toks) == dense_tok).mean())
        recall = float(np.concatenate(hits).mean())
        for B in Bs:
            steps = max(50, 800 // B)
            us = timed_us(B, lambda e, h, b, i: lib.fh_forward_adaptive(
                e, h, b, pmax, 1, tau, 0, T, 0x5EED + i, None, ptr(otok), ptr(olog), ptr(olse),
                None, None, None, sp), steps)
            adaptive.append({"B": B, "p_max": pmax, "tau": tau, "temperature": T,
                             "mean_probes": round(float(ns.mean()), 1),
                             "probes_min_median_max": [int(ns.min()), float(np.median(ns)),
                                                       int(ns.max())],
                             "us_per_call": round(us, 2), "tokens_per_s": round(B / (us * 1e-6), 1),
                             "top1_agreement": round(agree, 4), "cluster_recall": round(recall, 4)})
            print(f"[bench] adaptive B={B} tau={tau} {us:.1f} us mean n {ns.mean():.1f}",
                  file=sys.stderr, flush=True)
    dense = []
    for B in Bs:
        us = timed_us(B, lambda e, h, b, i: lib.fh_dense_forward(e, h, b, 0, 1.0, 0x5EED + i,
                                                                  ptr(otok), ptr(olog), ptr(olse),
                                                                  None, sp), max(50, 400 // B))
        dense.append({"B": B, "us_per_call": round(us, 2), "tokens_per_s": round(B / (us * 1e-6), 1)})
    res = {"metric": "FlashHead latency and top-1 agreement with the dense head, B x p sweep",
           "unit": "us per call", "n_gpus": 1, "dtype": "bf16" if bf16 else "f32",
           "data": f"synthetic seeded clustered embeddings (no trained weights), {nq} queries",
           "config": {"workload": f"{shape.name} sweep", "quant": args.quant, "replicas": R,
                      "alpha": shape.alpha, "spread": shape.spread,
                      "mode": "greedy, probes shared by the batch (top p of the summed scores)"
                      if shared else "greedy (top-p probes, argmax)"},
           "rows": rows, "dense": dense}
    if adaptive:
        res["adaptive"] = adaptive
    print(json.dumps(res), flush=True)
    for h in heads:
        h.close()


def spec_main(args):
    """Speculative decoding with FlashHead drafts: K draft calls at B = 1
    (sampled tokens, their probes kept) and one verification of the K
    positions against the dense head, timed with HIP events on the launch
    stream; beside it, the dense head sampling the same K positions."""
    import numpy as np
    import torch

    from lm_output_head_amd import flashhead as fhb
    from synth import SHAPES, make_problem

    if not torch.cuda.is_available():
        print(json.dumps({"error": "no GPU visible"}))
        sys.exit(1)
    shape = SHAPES[args.shape]
    K, p, T = args.spec, args.p, args.temperature
    pb = make_problem(shape, nq=max(K, 16))
    bf16 = shape.dtype == "bf16"
    tdt = torch.bfloat16 if bf16 else torch.float32

    def dev(x):
        if bf16:
            return torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).view(torch.bfloat16).cuda()
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()

    E, C, H = dev(pb.E_bits if bf16 else pb.E), dev(pb.C_bits if bf16 else pb.C), \
        dev(pb.H_bits if bf16 else pb.H)
    head = fhb.FlashHead(E, C, pb.C2T, quant=args.quant, max_batch=K)
    Hk = H[:K].contiguous()
    st = torch.cuda.current_stream()
    drafts = [head.forward(Hk[i:i + 1], p, mode=2, temperature=T, seed=100 + i, want_clusters=True)
              for i in range(K)]
    draft = {k: torch.cat([d[k] for d in drafts]) for k in ("clusters", "token", "lse")}

    def timed(fn, n):
        for _ in range(5):
            fn()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record(st)
        for _ in range(n):
            fn()
        b.record(st)
        torch.cuda.synchronize()
        return a.elapsed_time(b) * 1e3 / n

    steps = max(20, min(args.steps, 400))
    draft_us = timed(lambda: head.forward(Hk[:1], p, mode=2, temperature=T, seed=1,
                                          want_clusters=True), steps)
    verify_us = timed(lambda: head.spec_verify(Hk, draft, p, T, 7), steps)
    dense_us = timed(lambda: head.dense(Hk, mode=2, temperature=T, seed=7), steps)
    dense1_us = timed(lambda: head.dense(Hk[:1], mode=2, temperature=T, seed=7), steps)
    acc = torch.cat([head.spec_verify(Hk, draft, p, T, s)["accepted"] for s in range(64)])
    rate = float(acc.float().mean())
    elem = 2 if bf16 else 4
    verify_bytes = shape.v * shape.d * elem + K * shape.d * elem + shape.v * 4
    res = {
        "metric": "speculative verification of K FlashHead drafts against the dense head",
        "value": round(verify_us, 2), "unit": "us per verification", "n_gpus": 1, "steps": steps,
        "higher_is_better": False, "dtype": "bf16" if bf16 else "f32",
        "data": "synthetic seeded clustered embeddings (no trained weights)",
        "config": {"workload": f"{shape.name} K={K} p={p} T={T}", "K": K, "p": p,
                   "temperature": T, "quant": args.quant},
        "draft_us_per_position": round(draft_us, 2),
        "dense_sample_us": {"B=1": round(dense1_us, 2), f"B={K}": round(dense_us, 2)},
        "acceptance_rate": round(rate, 4),
        "verify_achieved_gbs": round(verify_bytes / (verify_us * 1e-6) / 1e9, 1),
        "roofline": {"bound": "hbm", "achieved": round(verify_bytes / (verify_us * 1e-6) / 1e9, 1),
                     "peak": HBM_PEAK_GBS, "unit": "GB/s",
                     "frac": round(verify_bytes / (verify_us * 1e-6) / 1e9 / HBM_PEAK_GBS, 4),
                     "traffic": None, "kernel": "spec verification (probe bits, row pass, finish)"},
    }
    print(json.dumps(res), flush=True)
    head.close()


def serve_main(args):
    """One decode step after the last layer: rmsnorm(x + residual) with an
    int8 output, the int8 dense head, the rules on its logits (penalties over
    1000 tokens of history, 16 biases, a grammar mask on every other row) and
    the choice of the token; beside it the step's parts, and the same step
    with the norm's own output into the dense head of the shape's dtype.  Two
    copies of each head are used in turn, so that no call finds the rows of
    the one before in the 256 MB cache."""
    import torch

    from lm_output_head_amd import FlashHead, LogitRules, W8A8Head, logits_apply, rmsnorm
    from synth import SHAPES, make_problem

    if not torch.cuda.is_available():
        print(json.dumps({"error": "no GPU visible"}))
        sys.exit(1)
    shape = SHAPES[args.shape]
    B, v, d, mode, T = args.B, shape.v, shape.d, args.mode & 2, args.temperature
    bf16 = shape.dtype == "bf16"
    pb = make_problem(shape, nq=1)
    if bf16:
        E = torch.from_numpy(pb.E_bits.view("int16")).view(torch.bfloat16).cuda()
        C = torch.from_numpy(pb.C_bits.view("int16")).view(torch.bfloat16).cuda()
    else:
        E, C = torch.from_numpy(pb.E).cuda(), torch.from_numpy(pb.C).cuda()
    E2 = E.clone()
    w8 = [W8A8Head(E), W8A8Head(E2)]
    dense = [FlashHead(E, C, pb.C2T, max_batch=B), FlashHead(E2, C, pb.C2T, max_batch=B)]
    g = torch.Generator(device="cuda").manual_seed(11)

    def rand(*size):
        return torch.randn(*size, generator=g, device="cuda")

    x, res, weight = rand(B, d).to(E.dtype), rand(B, d).to(E.dtype), rand(d).to(E.dtype)
    words = (v + 31) // 32
    rules = LogitRules(
        v, history=torch.randint(0, v, (B, 1000), generator=g, device="cuda", dtype=torch.int32),
        n_prompt=torch.full((B,), 500, device="cuda", dtype=torch.int32),
        repetition=torch.full((B,), 1.1, device="cuda"), presence=torch.full((B,), 0.2, device="cuda"),
        bias_ids=torch.randint(0, v, (B, 16), generator=g, device="cuda", dtype=torch.int32), bias=rand(B, 16),
        mask=torch.randint(-2 ** 31, 2 ** 31 - 1, (1, words), generator=g, device="cuda", dtype=torch.int32),
        mask_row=(torch.arange(B, device="cuda", dtype=torch.int32) % 2) - 1)
    st = torch.cuda.current_stream()

    def timed(fn, n):
        for i in range(10):
            fn(i)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record(st)
        for i in range(n):
            fn(i)
        b.record(st)
        torch.cuda.synchronize()
        return round(a.elapsed_time(b) * 1e3 / n, 2)

    steps = max(20, min(args.steps, 400))
    h = rmsnorm(x, weight, residual=res, want_q=True)
    z = w8[0].matmul(h["q"], h["q_scale"])

    def step_dense(i):
        y = rmsnorm(x, weight, residual=res)
        o = dense[i % 2].dense(y["out"], want_logits=True)
        return logits_apply(o["logits"], rules, mode=mode, temperature=T, seed=i, out=o["logits"])

    step_us = timed(lambda i: w8[i % 2].step(x, weight, residual=res, rules=rules, mode=mode, temperature=T,
                                             seed=i), steps)
    parts = {
        "norm": timed(lambda i: rmsnorm(x, weight, residual=res, want_out=False, want_q=True), steps),
        "int8_product": timed(lambda i: w8[i % 2].matmul(h["q"], h["q_scale"]), steps),
        "int8_head": timed(lambda i: w8[i % 2].forward(h["q"], h["q_scale"], mode, T, i), steps),
        "rules": timed(lambda i: logits_apply(z, rules, mode=mode, temperature=T, seed=i), steps),
    }
    dense_us = timed(step_dense, steps)
    nbytes = v * d + 4 * v + 4 * B * v + B * d * (3 * E.element_size() + 1)
    res_line = {
        "metric": "decode step after the last layer: norm, int8 dense head, rules on logits, token",
        "value": step_us, "unit": "us per step", "n_gpus": 1, "steps": steps, "higher_is_better": False,
        "dtype": "int8 x int8, f32 logits", "data": "synthetic seeded clustered embeddings (no trained weights)",
        "config": {"workload": f"{shape.name} B={B} mode={mode} T={T}", "B": B, "v": v, "d": d},
        "parts_us": parts, f"step_{'bf16' if bf16 else 'f32'}_dense_us": dense_us,
        "roofline": {"bound": "hbm", "achieved": round(nbytes / step_us / 1e3, 1), "peak": HBM_PEAK_GBS,
                     "unit": "GB/s", "frac": round(nbytes / step_us / 1e3 / HBM_PEAK_GBS, 4)},
    }
    print(json.dumps(res_line), flush=True)
    for o in w8 + dense:
        o.close()


def main():
    args = parse()
    if args.gpus != 1:
        print(json.dumps({"error": "this benchmark runs on one GPU; --gpus must be 1",
                          "n_gpus_requested": args.gpus}))
        sys.exit(2)
    if args.copy_calibration:
        copy_calibration()
        return
    if args.burst:
        burst_main(args)
        return
    if args.cluster:
        cluster_main(args)
        return
    if args.spec:
        spec_main(args)
        return
    if args.serve:
        serve_main(args)
        return
    if args.sweep:
        sweep_main(args)
        return

    import numpy as np
    import torch

    from lm_output_head_amd import flashhead as fhb
    from synth import SHAPES, make_problem

    if not torch.cuda.is_available():
        print(json.dumps({"error": "no GPU visible"}))
        sys.exit(1)
    shape = SHAPES[args.shape]
    B, p = args.B, args.p
    print(f"[bench] generating {shape.name} workload", file=sys.stderr, flush=True)
    pb = make_problem(shape)
    bf16 = shape.dtype == "bf16"
    elem = 2 if bf16 else 4
    tdt = torch.bfloat16 if bf16 else torch.float32

    def dev(bits_or_f32):
        a = np.ascontiguousarray(bits_or_f32)
        if bf16:
            return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()
        return torch.from_numpy(a.astype(np.float32)).cuda()

    E0 = dev(pb.E_bits if bf16 else pb.E)
    C0 = dev(pb.C_bits if bf16 else pb.C)
    Hall = dev(pb.H_bits if bf16 else pb.H)
    nq = Hall.shape[0]
    R = max(1, args.replicas)
    heads = []
    for r in range(R):
        E = E0 if r == 0 else E0.clone()
        C = C0 if r == 0 else C0.clone()
        heads.append(fhb.FlashHead(E, C, pb.C2T, quant=args.quant, max_batch=B))
        heads[-1].set_path(args.path)
    # query batches: B consecutive queries, rotating
    hb = [Hall[(i * B) % nq:(i * B) % nq + B].contiguous() for i in range(max(1, nq // B))]
    out_tok = torch.empty(B, dtype=torch.int32, device="cuda")
    out_logit = torch.empty(B, dtype=torch.float32, device="cuda")
    out_lse = torch.empty(B, dtype=torch.float32, device="cuda")
    stream = torch.cuda.current_stream()
    lib = fhb._abi.load()
    sp = ctypes.c_void_p(stream.cuda_stream)
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    hptr = [ptr(h) for h in hb]
    engs = [h.eng for h in heads]
    otok, olog, olse = ptr(out_tok), ptr(out_logit), ptr(out_lse)

    def step(i):
        st = lib.fh_forward(engs[i % R], hptr[i % len(hptr)], B, p, args.mode,
                            args.temperature, 0x5EED + i, otok, olog, olse, None, None, None, sp)
        if st != 0:
            raise RuntimeError(lib.fh_last_error().decode())

    def dense_step(i):
        st = lib.fh_dense_forward(engs[i % R], hptr[i % len(hptr)], B, args.mode & 2,
                                  args.temperature, 0x5EED + i, otok, olog, olse, None, sp)
        if st != 0:
            raise RuntimeError(lib.fh_last_error().decode())

    def timed(fn, steps, warmup):
        for i in range(warmup):
            fn(i)
        torch.cuda.synchronize()
        ev0, ev1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0 = time.perf_counter()
        ev0.record(stream)
        for i in range(steps):
            fn(warmup + i)
        ev1.record(stream)
        torch.cuda.synchronize()
        wall = time.perf_counter() - t0
        return ev0.elapsed_time(ev1) / steps, wall / steps * 1e3

    print(f"[bench] timing {args.steps} FlashHead steps", file=sys.stderr, flush=True)
    ms, wall_ms = timed(step, args.steps, args.warmup)

    # the same steps again with per-kernel HIP events on the launch stream
    n_launch = 4 * args.steps
    for eng in engs:
        fhb.fh_profile_begin(eng, n_launch)
    ms_prof, _ = timed(step, args.steps, 0)
    per = {}
    for eng in engs:
        for name, (n, tot) in fhb.fh_profile_end(eng).items():
            a = per.setdefault(name, [0, 0.0])
            a[0] += n
            a[1] += tot
    kern = {k: {"launches": n, "avg_us": round(tot / n * 1e3, 3)} for k, (n, tot) in per.items()}
    union = None
    if B > 1:
        # distinct clusters per batch, from the engine's own probe lists
        us = []
        for hq in hb[:16]:
            o = heads[0].forward(hq, p, mode=args.mode, temperature=args.temperature, seed=0x5EED,
                                 want_clusters=True)
            us.append(int(torch.unique(o["clusters"]).numel()))
        union = sum(us) / len(us)
    algo = algorithmic_bytes(shape, B, p, args.quant, elem, union)
    dominant = max((k for k in kern if k in algo),
                   key=lambda k: kern[k]["avg_us"] * kern[k]["launches"] * (algo[k] > 1e6))
    dom_bytes = algo[dominant]
    # the kernel's duration: a step of one launch (the batch-1 call) is timed
    # by the events around the whole timed region divided by the steps, which
    # cannot exceed the step; an event pair around each launch also holds the
    # launch's own latency and is kept beside it
    one_launch = len(kern) == 1 and kern[dominant]["launches"] == args.steps
    pair_us = kern[dominant]["avg_us"]
    dom_us = min(pair_us, ms * 1e3) if one_launch else pair_us
    dur_src = ("HIP events around the timed region / steps (one launch per step)" if one_launch
               else "HIP event pair around each launch, on its stream")
    achieved = dom_bytes / (dom_us * 1e-6) / 1e9
    src_hash = kernel_source_hash()
    wkey = f"{shape.name}/B{B}/p{p}/{args.quant}/m{args.mode}"
    traffic = traffic_from_profiles(dominant, src_hash, wkey)
    total_bytes = algo["call"]

    if union is not None:
        res_union = {"distinct_clusters_per_batch": round(union, 1)}
    else:
        res_union = {}
    res = {
        "metric": "FlashHead calls/s & achieved HBM GB/s (v=128256,d=2048,p=512) vs dense head",
        "value": round(1000.0 / ms, 2),
        "unit": "calls/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "bf16" if bf16 else "f32",
        "data": "synthetic seeded clustered embeddings (no trained weights)",
        "config": {"workload": f"flashhead_{shape.name}", "v": shape.v, "d": shape.d,
                   "c": shape.c, "b": shape.b, "p": p, "batch": B, "quant": args.quant,
                   "mode": args.mode, "replicas": R, "path": args.path,
                   "parallelism": "single-gpu"},
        "tokens_per_s": round(1000.0 / ms * B, 2),
        "call_algorithmic_bytes": total_bytes,
        "call_achieved_gbs": round(total_bytes / (ms * 1e-3) / 1e9, 1),
        "call_roofline_frac": round(total_bytes / (ms * 1e-3) / 1e9 / HBM_PEAK_GBS, 4),
        "host_wall_ms_per_step": round(wall_ms, 5),
        "profiled_ms_per_step": round(ms_prof, 5),
        "kernels": kern,
        **res_union,
        "roofline": {"bound": "hbm", "kernel": dominant, "achieved": round(achieved, 1),
                     "peak": HBM_PEAK_GBS, "unit": "GB/s",
                     "frac": round(achieved / HBM_PEAK_GBS, 4), "traffic": traffic,
                     "algorithmic_bytes": dom_bytes, "duration_us": round(dom_us, 3),
                     "duration_source": dur_src, "event_pair_us": pair_us,
                     "source_hash": src_hash, **kernel_us_from_profiles(dominant, src_hash, wkey,
                                                                        dom_bytes)},
    }
    # the same call writing every output fh_forward offers (the probe list,
    # the retrieved ids and logits), as the method's call returns them
    b = shape.b
    o_cl = torch.empty(B * p, dtype=torch.int32, device="cuda")
    o_ids = torch.empty(B * p * b, dtype=torch.int32, device="cuda")
    o_lg = torch.empty(B * p * b, dtype=torch.float32, device="cuda")
    ocl, oids, olg = ptr(o_cl), ptr(o_ids), ptr(o_lg)

    def step_all(i):
        st = lib.fh_forward(engs[i % R], hptr[i % len(hptr)], B, p, args.mode, args.temperature,
                            0x5EED + i, otok, olog, olse, ocl, oids, olg, sp)
        if st != 0:
            raise RuntimeError(lib.fh_last_error().decode())

    # per-call latency: an event pair around each call on the launch stream
    nlat = min(args.steps, 500)
    evs = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
           for _ in range(nlat)]
    for i, (a0, a1) in enumerate(evs):
        a0.record(stream)
        step(i)
        a1.record(stream)
    torch.cuda.synchronize()
    lat = sorted(a0.elapsed_time(a1) * 1e3 for a0, a1 in evs)
    pick = lambda q: round(lat[min(len(lat) - 1, int(q * len(lat)))], 3)  # noqa: E731
    res["latency_us"] = {"p10": pick(0.10), "p50": pick(0.50), "p90": pick(0.90), "calls": nlat,
                         "how": "HIP event pair around each call on its stream, back to back, "
                                "engine replicas rotated"}
    # the roofline against the part's measured streaming rate as well
    print("[bench] measuring the stream bandwidth", file=sys.stderr, flush=True)
    call_sz = int(total_bytes)
    sb = stream_bandwidth([call_sz, 525336576])
    res["roofline"]["stream_gbs"] = sb[525336576]
    res["roofline"]["stream_call_size_gbs"] = sb[call_sz]
    res["roofline"]["frac_vs_stream"] = round(achieved / sb[525336576], 4)
    res["roofline"]["frac_vs_stream_call_size"] = round(achieved / sb[call_sz], 4)
    res["roofline"]["stream_how"] = ("plain one-shot reads (bench library read probe), 16 rotating "
                                     "buffers, back to back, at 525,336,576 B and at the call's bytes")
    print(f"[bench] timing {args.steps} steps with every output", file=sys.stderr, flush=True)
    ms_all, _ = timed(step_all, args.steps, 10)
    res["with_retrieved_outputs"] = {
        "ms_per_step": round(ms_all, 5), "calls_per_s": round(1000.0 / ms_all, 2),
        "extra_output_bytes": B * p * 4 + 2 * B * p * b * 4,
        "outputs": "token, token logit, LSE, probe list, retrieved ids and logits"}
    if not args.no_dense:
        print(f"[bench] timing {args.dense_steps} dense steps", file=sys.stderr, flush=True)
        dms, _ = timed(dense_step, args.dense_steps, 10)
        dense_bytes = algo["dense"]
        res["dense"] = {"calls_per_s": round(1000.0 / dms, 2), "ms_per_call": round(dms, 5),
                        "achieved_gbs": round(dense_bytes / (dms * 1e-3) / 1e9, 1),
                        "speedup_flashhead_vs_dense": round(dms / ms, 3)}
        # sanity reference for the dense baseline: the vendor GEMM (torch ->
        # hipBLASLt / rocBLAS) for the logits plus an argmax, same replicas
        Es = [hd._E for hd in heads]

        def torch_dense(i):
            z = torch.matmul(hb[i % len(hb)], Es[i % R].t())
            return z.argmax(dim=1)

        tms, _ = timed(torch_dense, args.dense_steps, 10)
        res["dense"]["torch_matmul_argmax_ms"] = round(tms, 5)
    for hd in heads:
        hd.sync_status()
        hd.close()
    if not args.no_cpu:
        print("[bench] timing the CPU oracle", file=sys.stderr, flush=True)
        res["cpu_baseline"] = cpu_baseline(pb, p, args.quant, args.mode, args.temperature,
                                           args.cpu_seconds)
    print(json.dumps(res), flush=True)


if __name__ == "__main__":
    main()
