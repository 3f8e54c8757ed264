"""Calls of expert routing, 8-bit products and the gather of expert rows for a profiler, and the table of what it saw.

    python3 profiles/moe_operators_calls.py run TIMES            each call TIMES times, on two sets of inputs in turn
    python3 profiles/moe_operators_calls.py time                 us a call among others, with its floor
    python3 profiles/moe_operators_calls.py read DIR TIMES CTIMES    the table of a trace and three counter runs in DIR:
        t_kernel_trace.csv of `run TIMES`, {f,w,s}_counter_collection.csv of `run CTIMES` with FETCH_SIZE, WRITE_SIZE and the
        SQ counters

The cases are perf/more_operators.py's, through the library, and the forms below that it does not list.
"""
import collections
import csv
import os
import statistics
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from perf import more_operators as operators  # noqa: E402

COPY, PRODUCT = 5.24e12, 1982e12  # bytes/s of a copy of 1 GiB and operations/s of a large 8-bit product of the vendor's library here
READ = 1024 * 1.999912            # bytes of FETCH_SIZE: a 512 MiB copy reads as half of it


def route(name, tokens, experts, **more):
    return dict(dict(name=name, op="route", tokens=tokens, experts=experts, top_k=8, score="softmax", bias=False, groups=1, top_groups=1,
                     best=1, renorm=True, scale=1.0, f16=False, pad=0), **more)


MORE = [
    route("route_biased_groups", 16384, 256, score="sigmoid", bias=True, groups=8, top_groups=4, best=2, scale=2.5),
    route("route_long", 262144, 128),
    dict(name="product_cube", op="product", m=8192, n=8192, k=8192, x16=True, y16=True),
    dict(name="product_middling", op="product", m=512, n=8192, k=2048, x16=True, y16=True),
    dict(name="product_down", op="product", m=2048, n=2048, k=8192, x16=True, y16=True),
    dict(name="experts_down_fp16", op="experts", glu=False, tokens=4096, experts=128, top_k=8, n=2048, k=768, x16=True, y16=True),
    dict(name="experts_decode_down", op="experts", glu=False, tokens=16, experts=128, top_k=8, n=2048, k=768, x16=True, y16=False),
    dict(name="experts_few", op="experts", glu=True, tokens=4096, experts=8, top_k=2, n=4096, k=2048, x16=True, y16=True),
    dict(name="experts_512", op="experts", glu=True, tokens=512, experts=128, top_k=8, n=768, k=2048, x16=True, y16=True),
    dict(name="gather_fp32", op="gather", tokens=4096, top_k=8, n=2048, f16=False, residual=True, pad=0),
]


def cases():
    return operators.listed() + MORE


def floor(case):
    w = operators.work(case)
    return max(w["bytes"] / COPY, w["flops"] / PRODUCT if case["op"] in ("product", "experts") else 0) * 1e6


def run(times):
    import torch
    operators.own = True
    for case in cases():
        states = [operators.prepare(case, 100 + i) for i in range(2)]
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        for i in range(times):
            operators.run(states[i % 2])
        torch.cuda.synchronize()


def time():
    import torch
    operators.own = True
    for case in cases():
        states = [operators.prepare(case, 100 + i) for i in range(2)]
        got = []
        for _ in range(9):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for i in range(60):
                operators.run(states[i % 2])
            b.record()
            b.synchronize()
            got.append(a.elapsed_time(b) * 1000 / 60)
        w = operators.work(case)
        t = statistics.median(got[2:])
        print("%-22s floor %7.1f us  call %7.1f us  %6.2f TB/s %6.0f TOP/s" % (
            case["name"], floor(case), t, w["bytes"] / t / 1e6, w["flops"] / t / 1e6), flush=True)


def groups(path, times):
    """Of each counter (None: the trace) a list for every case: its kernels in the order of a call, each with what `times` calls saw.
    A case's calls stand between those that make inputs, which are no kernels of the library."""
    by = collections.defaultdict(list)
    for r in csv.DictReader(open(path)):
        by[r.get("Counter_Name")].append(r)
    out = {}
    for name, rows in by.items():
        rows.sort(key=lambda r: int(r["Dispatch_Id"]))
        found, inside = [], False
        for r in rows:
            ours = "qmm" in r["Kernel_Name"]
            if ours and not inside:
                found.append([])
            if ours:
                found[-1].append(r)
            inside = ours
        assert len(found) == len(cases()) and all(len(f) % times == 0 for f in found), (path, name, [len(f) for f in found])
        out[name] = [[f[i::len(f) // times] for i in range(len(f) // times)] for f in found]
    return out


def read(where, times, ctimes):
    trace = groups(os.path.join(where, "t_kernel_trace.csv"), times)[None]
    counted = {}
    for f in "fws":
        for name, g in groups(os.path.join(where, f + "_counter_collection.csv"), ctimes).items():
            counted[name] = [[statistics.median(float(r["Counter_Value"]) for r in k) for k in case] for case in g]
    print("| call | kernel | us (least) | read + written MB | matrix cores | vector units | LDS conflicts |")
    print("|---|---|---:|---:|---:|---:|---:|")
    for i, case in enumerate(cases()):
        for j, rows in enumerate(trace[i]):
            us = [(int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3 for r in rows]
            busy = counted["SQ_BUSY_CU_CYCLES"][i][j]
            kernel = rows[0]["Kernel_Name"]
            kernel = next(k for k in ("route_place", "route_running", "route_sums", "route", "quantize_rows", "quantize", "rows_i8", "tile_i8", "gather") if k in kernel)
            print("| %s | %s | %.1f (%.1f) | %.1f + %.1f | %.0f %% | %.0f %% | %.2f |" % (
                case["name"] if j == 0 else "", kernel, statistics.median(us), min(us), counted["FETCH_SIZE"][i][j] * READ / 1e6,
                counted["WRITE_SIZE"][i][j] * 1024 / 1e6, 100 * counted["SQ_VALU_MFMA_BUSY_CYCLES"][i][j] / (4 * busy),
                100 * counted["SQ_ACTIVE_INST_VALU"][i][j] / busy,
                counted["SQ_LDS_BANK_CONFLICT"][i][j] / max(1, counted["SQ_LDS_IDX_ACTIVE"][i][j])))


if __name__ == "__main__":
    what = sys.argv[1] if len(sys.argv) > 1 else ""
    if what == "run":
        run(int(sys.argv[2]))
    elif what == "time":
        time()
    elif what == "read":
        read(sys.argv[2], int(sys.argv[3]), int(sys.argv[4]))
    else:
        sys.exit(__doc__)
