"""Workloads of the low-bit linear layer and the gated unit: what the files profiles/*_linear.md are taken from.

    python -m bit_quantization_block_amd.linear_workloads run PASSES
    python -m bit_quantization_block_amd.linear_workloads times OUT_MD
    python -m bit_quantization_block_amd.linear_workloads kernels KERNEL_TRACE_CSV OUT_MD "COMMAND"
    python -m bit_quantization_block_amd.linear_workloads counters OUT_MD "COMMANDS" COUNTER_CSV...

`run` (under rocprofv3) makes one call of each workload a pass, so that no call finds its own data in a cache. `times` needs
no profiler: each workload's calls one after another between two events, and calls of one layer after another in a graph,
over more weights than the caches hold.
"""
from __future__ import annotations

import csv
import re
import sys
from collections import defaultdict

from . import lq
from .profiling import CYCLES_PER_VALU, SIMDS, kernel_source_digest

# call: of Mx4Linear (with `ckpt` the forward call keeps x), quantize (x to MXFP4 and to a checkpoint), gated, gated_back
WORK = [
    dict(call="forward", m=1, n=11008, k=4096), dict(call="forward", m=16, n=4096, k=11008),
    dict(call="forward", m=64, n=4096, k=4096), dict(call="forward", m=515, n=4099, k=1000, dtype="f32", out="f32"),
    dict(call="forward", m=8192, n=11008, k=4096), dict(call="quantize", m=8192, n=0, k=4096, fmt="int8"),
    dict(call="dgrad", m=77, n=1001, k=520, out="f32"), dict(call="dgrad", m=1024, n=4096, k=4096),
    dict(call="dgrad", m=8192, n=11008, k=4096),
    dict(call="wgrad", m=1001, n=520, k=1000, fmt="e4m3"), dict(call="wgrad", m=1024, n=4096, k=4096, fmt="int8"),
    dict(call="wgrad", m=8192, n=11008, k=4096, fmt="int8"), dict(call="wgrad", m=8192, n=11008, k=4096, fmt="e4m3"),
    dict(call="gated", m=8192, n=11008, dtype="bf16", fmt="int8"), dict(call="gated_back", m=8192, n=11008, dtype="bf16", fmt="int8"),
    dict(call="gated", m=8192, n=11008, dtype="f32", fmt="int8"), dict(call="gated_back", m=8192, n=11008, dtype="f32", fmt="int8"),
]
# weights that no cache holds: rows, n, k
COLD = [(1, 4096, 4096), (1, 11008, 4096), (1, 4096, 11008), (1, 8192, 8192), (4, 11008, 4096), (8, 11008, 4096), (16, 4096, 11008),
        (24, 4096, 4096), (64, 4096, 4096), (128, 4096, 4096), (256, 4096, 4096)]


def label(w: dict) -> str:
    what = {"forward": "y", "dgrad": "dx", "wgrad": "dw", "quantize": "x to MXFP4 and 8 bits", "gated": "gated unit",
            "gated_back": "gated unit back"}[w["call"]]
    size = "x".join(str(w[d]) for d in ("m", "n", "k") if w.get(d))
    types = [w.get("dtype", "bf16")] + ([w["out"]] if "out" in w else []) + ([w["fmt"]] if "fmt" in w else [])
    return f"{what} {size} {' '.join(types)}"


def kernels(w: dict) -> list:
    """[(kernel, workgroups)] of the workload's call."""
    m, n, k, fmt = w["m"], w["n"], w.get("k", 0), w.get("fmt", "int8")
    dtype = w.get("dtype", "bf16")
    if w["call"].startswith("gated"):
        name = "k_swiglu" if w["call"] == "gated" else "k_swiglu_backward"
        return [(f"{name}<{lq.DTYPE[dtype]}, {lq.FORMAT[fmt]}>", -(-n // 512) * min(-(-m // 4), 65535))]
    call = {"forward": "linear"}.get(w["call"], w["call"])
    out = "f32" if call == "wgrad" else w.get("out", "bf16")
    return [k[:2] for k in lq.linear_kernels(call, m, n, k, dtype, out, fmt, also=call == "quantize")]


def needed(w: dict) -> tuple:
    """Bytes that the call has to read and to write, and its operations."""
    m, n, k = w["m"], w["n"], w.get("k", 0)
    size = {"f32": 4, "bf16": 2, "f16": 2}
    e, o = size[w.get("dtype", "bf16")], size[w.get("out", "bf16")]
    kept = 33 / 32
    return {"forward": lambda: (m * k * e + n * k * 17 / 32, m * n * o, 2 * m * n * k),
            "quantize": lambda: (m * k * e, m * k * (17 / 32 + kept), 0),
            "dgrad": lambda: (m * n * 2 + n * k * 17 / 32, m * k * o, 2 * m * n * k),
            "wgrad": lambda: (m * n * 2 + m * k * kept, n * k * 4, 2 * m * n * k),
            "gated": lambda: (2 * m * n * e, m * n * (e + 2 * kept), 0),
            "gated_back": lambda: (m * n * (e + 2 * kept), 2 * m * n * e, 0)}[w["call"]]()


# ------------------------------------------------------------------ on the GPU
def prepare(w: dict):
    """The workload's call, its inputs made."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda rows, cols, dtype="bf16", scale=1.0: (
        torch.randn(rows, cols, generator=gen, device="cuda") * scale).to(lq._torch_dtype(dtype))
    m, n, k, dtype, fmt = w["m"], w["n"], w.get("k", 0), w.get("dtype", "bf16"), w.get("fmt", "int8")
    if w["call"].startswith("gated"):
        act = lq.SwigluCkpt8(m, n, dtype, fmt)
        gate, up = rand(m, n, dtype, 1.5), rand(m, n, dtype)
        act.forward(gate, up)
        return (lambda: act.forward(gate, up)) if w["call"] == "gated" else (lambda: act.backward(up))
    if w["call"] == "quantize":
        x, kept = rand(m, k), lq.Ckpt8(m, k, fmt)
        codes, scales = (torch.empty(f(m, k), dtype=torch.uint8, device="cuda")
                         for f in (lq.load().lq_mx4_codes_bytes, lq.load().lq_mx4_scales_bytes))
        import ctypes

        d = lq.LinearDesc(1, 0, lq.FORMAT[fmt], 0, m, 0, k, k, 0)
        return lambda: lq._check("lq_mx4_quantize", lq.load().lq_mx4_quantize(
            ctypes.byref(d), x.data_ptr(), codes.data_ptr(), scales.data_ptr(), kept.codes.data_ptr(), kept.scales.data_ptr(),
            lq._stream(None)))
    layer = lq.Mx4Linear(rand(n, k, scale=0.02), rows=m, dtype=dtype, out=w.get("out", "bf16"))
    if w["call"] == "forward":
        x = rand(m, k, dtype)
        return lambda: layer.forward(x)
    dy = rand(m, n, scale=0.01)
    if w["call"] == "dgrad":
        return lambda: layer.dgrad(dy)
    kept = lq.Ckpt8(m, k, fmt)
    kept.save(rand(m, k))
    return lambda: layer.wgrad(dy, kept)


def run(passes: int) -> None:
    import torch

    calls = [prepare(w) for w in WORK]
    for _ in range(passes):
        for call in calls:
            call()
    torch.cuda.synchronize()
    print(f"{passes} passes over {len(calls)} calls", flush=True)


def _between_events(fn, calls: int) -> float:
    """Microseconds a call."""
    import torch

    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    a.record()
    fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / calls


def times(out_md: str) -> None:
    import torch

    lines = ["# Times of the low-bit linear layer and the gated unit", "",
             "Command: `python3 -m bit_quantization_block_amd.linear_workloads times`", "",
             "Calls one after another, each on the same inputs, between two events: the least and the largest of five rounds of "
             "about 20 ms, in us; TB/s and TFLOP/s by what the call has to move and compute.", "",
             "| work | least us | largest us | TB/s | TFLOP/s |", "|---|---|---|---|---|"]
    for w in WORK:
        call = prepare(w)
        for _ in range(5):
            call()
        again = max(5, int(2e4 / _between_events(lambda: [call() for _ in range(5)], 5)))
        t = [_between_events(lambda: [call() for _ in range(again)], again) for _ in range(5)]
        read, written, flops = needed(w)
        lines.append(f"| {label(w)} | {min(t):.1f} | {max(t):.1f} | {(read + written) / min(t) / 1e6:.2f} | {flops / min(t) / 1e6:.0f} |")
        print(lines[-1], flush=True)
        del call
    lines += ["", "Weights in memory: one call of each of as many layers as make 700 MB of weights, in a graph, bfloat16 in and out; "
              "us a call, the least and the largest of five replays.", "", "| rows x n x k | least us | largest us | TB/s |", "|---|---|---|---|"]
    for m, n, k in COLD:
        layers = min(200, max(2, int(700e6 / (n * k * 17 / 32)) + 1))
        w = torch.randn(n, k, device="cuda") * 0.02
        x = torch.randn(m, k, device="cuda").bfloat16()
        stack = [lq.Mx4Linear(w, rows=m) for _ in range(layers)]
        for layer in stack:
            layer.forward(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for layer in stack:
                layer.forward(x)
        graph.replay()
        t = [_between_events(graph.replay, layers) for _ in range(5)]
        lines.append(f"| {m}x{n}x{k} | {min(t):.2f} | {max(t):.2f} | {(n * k * 17 / 32 + 2 * m * (n + k)) / min(t) / 1e6:.2f} |")
        print(lines[-1], flush=True)
        del stack, graph
    lines += ["", f"Kernel source digest: {kernel_source_digest('linear')}"]
    with open(out_md, "w") as f:
        f.write("\n".join(lines) + "\n")


# ------------------------------------------------------------------ rocprofv3's records
def short(name: str) -> str:
    """A kernel's name with its template arguments, without namespaces and parameters."""
    return re.sub(r"\(anonymous namespace\)::|lql::|void ", "", name).split("(")[0]


def _attribute(dispatches: list) -> list:
    """[(workload, kernel, workgroups, its records)] from the records of a `run`, in order, each beginning with (kernel,
    workgroups): whole passes over the workloads, counted from the end (what made the inputs comes before them)."""
    order = [(w, *k) for w in WORK for k in kernels(w)]
    found = [[] for _ in order]
    end = len(dispatches)
    while end >= len(order) and [d[:2] for d in dispatches[end - len(order):end]] == [o[1:] for o in order]:
        for into, d in zip(found, dispatches[end - len(order):end]):
            into.append(d)
        end -= len(order)
    if end == len(dispatches):
        raise SystemExit("the last kernels are not a pass over the workloads")
    return [(*o, f) for o, f in zip(order, found)]


def summarize_kernels(trace_csv: str, out_md: str, command: str) -> None:
    seen = []
    for r in sorted(csv.DictReader(open(trace_csv)), key=lambda r: int(r["Dispatch_Id"])):
        if "lql::" in r["Kernel_Name"]:
            groups = int(r["Grid_Size_X"]) // int(r["Workgroup_Size_X"]) * int(r["Grid_Size_Y"])
            seen.append((short(r["Kernel_Name"]), groups, (int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3))
    lines = ["# rocprofv3 kernel summary: the low-bit linear layer and the gated unit", "", f"Command: `{command}`", "",
             "One call of each workload in turn. Times by the profiler, with data that the other calls have driven out of the caches: "
             "longer than those of calls one after another (times_linear.md).", "",
             "| work | kernel | workgroups | dispatches | avg us | min us | max us |", "|---|---|---|---|---|---|---|"]
    for w, name, groups, records in _attribute(seen):
        t = [r[2] for r in records]
        lines.append(f"| {label(w)} | `{name}` | {groups} | {len(t)} | {sum(t) / len(t):.1f} | {min(t):.1f} | {max(t):.1f} |")
    lines += ["", f"Kernel source digest: {kernel_source_digest('linear')}"]
    with open(out_md, "w") as f:
        f.write("\n".join(lines) + "\n")


def summarize_counters(out_md: str, commands: str, *counter_csvs: str) -> None:
    total = [defaultdict(list) for w in WORK for _ in kernels(w)]
    for path in counter_csvs:
        one = {}
        for r in csv.DictReader(open(path)):
            if "lql::" in r["Kernel_Name"]:
                key = (short(r["Kernel_Name"]), int(r["Grid_Size"]) // int(r["Workgroup_Size"]))
                d = one.setdefault(int(r["Dispatch_Id"]), (*key, {"VGPR": float(r["VGPR_Count"])}))
                d[2][r["Counter_Name"]] = float(r["Counter_Value"])
        for into, (_, _, _, records) in zip(total, _attribute([one[i] for i in sorted(one)])):
            for d in records:
                for counter, value in d[2].items():
                    into[counter].append(value)
    lines = ["# rocprofv3 counter summary: the low-bit linear layer and the gated unit", "", f"Commands: {commands}", "",
             "Averages per dispatch. Cycles = GRBM_GUI_ACTIVE / 8 XCDs. MFMA busy = SQ_VALU_MFMA_BUSY_CYCLES / 1024 SIMDs / cycles. "
             "LDS busy = SQ_LDS_IDX_ACTIVE / 256 CUs / cycles, conflicts as a share of that. VALU issue = (SQ_INSTS_VALU - "
             "SQ_INSTS_MFMA) x 4 / 1024 / cycles. Read and written in 10^6 bytes: WRITE_SIZE, and twice FETCH_SIZE, which counts a "
             "request of 128 bytes as 64 here (the streaming kernels show half of what they read, exactly).", "",
             "| work | kernel | VGPR | cycles | MFMA busy | VALU issue | LDS busy | of it conflicts | read MB | written MB | the call needs MB |",
             "|---|---|---|---|---|---|---|---|---|---|---|"]
    for (w, name), values in zip(((w, k[0]) for w in WORK for k in kernels(w)), total):
        c = {k: sum(v) / len(v) for k, v in values.items()}
        cycles = c["GRBM_GUI_ACTIVE"] / 8
        lds = c["SQ_LDS_IDX_ACTIVE"] / 256 / cycles
        read, written, _ = needed(w)
        lines.append(
            f"| {label(w)} | `{name}` | {c['VGPR']:.0f} | {cycles:.0f} | {c['SQ_VALU_MFMA_BUSY_CYCLES'] / SIMDS / cycles:.0%} | "
            f"{(c['SQ_INSTS_VALU'] - c['SQ_INSTS_MFMA']) * CYCLES_PER_VALU / SIMDS / cycles:.0%} | {lds:.0%} | "
            f"{c['SQ_LDS_BANK_CONFLICT'] / max(1.0, c['SQ_LDS_IDX_ACTIVE']):.0%} | {c['FETCH_SIZE'] * 2.048e-3:.0f} | "
            f"{c['WRITE_SIZE'] * 1.024e-3:.0f} | {read / 1e6:.0f} + {written / 1e6:.0f} |")
    lines += ["", f"Kernel source digest: {kernel_source_digest('linear')}"]
    with open(out_md, "w") as f:
        f.write("\n".join(lines) + "\n")


if __name__ == "__main__":
    cmd, args = (sys.argv[1], sys.argv[2:]) if len(sys.argv) > 1 else ("", [])
    if cmd == "run":
        run(int(args[0]))
    elif cmd == "times":
        times(args[0])
    elif cmd == "kernels":
        summarize_kernels(*args)
    elif cmd == "counters":
        summarize_counters(*args)
    else:
        raise SystemExit(__doc__)
