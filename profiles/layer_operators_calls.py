"""Calls of the norm, cache append and attention operators for a profiler, and the table of what it saw.

    python3 profiles/layer_operators_calls.py run TIMES            each call TIMES times, on three sets of inputs in turn
    python3 profiles/layer_operators_calls.py time                 us a call among others, with its floor
    python3 profiles/layer_operators_calls.py read DIR TIMES CTIMES    the table of a trace and three counter runs in DIR:
        t_kernel_trace.csv of `run TIMES`, {f,w,s}_counter_collection.csv of `run CTIMES` with FETCH_SIZE, WRITE_SIZE and the
        SQ counters

The cases are perf/operators.py's, through the library, and the forms below that it does not list.
"""
import collections
import csv
import os
import statistics
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from perf import operators  # noqa: E402

COPY, PRODUCT = 5.3e12, 1175e12  # bytes/s of a large copy and operations/s of a large fp16 product here
READ = 1024 * 1.999912           # bytes of FETCH_SIZE: a 512 MiB copy reads as half of it

MORE = [
    dict(name="norm_odd", op="norm", rows=4096, n=4095, y16=True, y=True, post=True, gate="rows"),
    dict(name="append_8bit", op="append", tokens=4096, seqs=3, hq=32, hkv=8, d=64, bits=8, group=32, page=16, in16=True, fused=True,
         qknorm=False, rot=64, inter=False, far=0, pad=5),
    dict(name="append_8bit_128", op="append", tokens=4096, seqs=3, hq=16, hkv=8, d=128, bits=8, group=64, page=64, in16=True,
         fused=True, qknorm=True, rot=128, inter=False, far=0, pad=0),
    dict(name="append_4bit_128", op="append", tokens=4096, seqs=3, hq=16, hkv=8, d=128, bits=4, group=64, page=64, in16=True,
         fused=True, qknorm=True, rot=128, inter=False, far=0, pad=0),
] + [dict(name="cache_%s_%s" % (kind, "fp16" if bits == 16 else "8bit"), op="cache", seqs=seqs, lo=lo, hi=hi, q_len=1, hq=32, hkv=hkv,
          d=d, bits=bits, group=32 if d == 64 else 64, page=16 if d == 64 else 64)
     for bits in (8, 16) for kind, seqs, lo, hi, hkv, d in (("long", 64, 2000, 8192, 4, 128), ("ragged", 17, 0, 5000, 8, 64))
] + [dict(name="cache_new_%d" % n, op="cache", seqs=2, lo=8192, hi=8192, q_len=n, hq=32, hkv=4, d=128, bits=4, group=64, page=64)
     for n in (16, 64, 256)
] + [dict(name="prompt_long_64", op="prompt", seqs=1, lo=8192, hi=8192, hq=32, hkv=8, d=64, tail=0),
     dict(name="prompt_short_64", op="prompt", seqs=16, lo=128, hi=128, hq=32, hkv=8, d=64, tail=0),
     dict(name="prompt_short_128", op="prompt", seqs=16, lo=128, hi=128, hq=32, hkv=4, d=128, tail=0)]


def cases():
    return operators.listed() + MORE


def floor(case):
    w = operators.work(case)
    return max(w["bytes"] / COPY, w["flops"] / PRODUCT) * 1e6


def run(times):
    import torch
    operators.own = True
    for case in cases():
        states = [operators.prepare(case, 100 + i) for i in range(3)]
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        for i in range(times):
            operators.run(states[i % 3])
        torch.cuda.synchronize()


def time():
    import torch
    operators.own = True
    for case in cases():
        states = [operators.prepare(case, 100 + i) for i in range(3)]
        got = []
        for _ in range(9):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for i in range(60):
                operators.run(states[i % 3])
            b.record()
            b.synchronize()
            got.append(a.elapsed_time(b) * 1000 / 60)
        w = operators.work(case)
        t = statistics.median(got[2:])
        print("%-26s floor %7.1f us  call %7.1f us  %6.2f TB/s %6.0f TFLOP/s" % (
            case["name"], floor(case), t, w["bytes"] / t / 1e6, w["flops"] / t / 1e6), flush=True)


def groups(path, times):
    """The library's dispatches in the order of the calls, `times` to a case; of counters one such list each."""
    by = collections.defaultdict(list)
    for r in csv.DictReader(open(path)):
        if "qmm::" in r["Kernel_Name"]:
            by[r.get("Counter_Name")].append(r)
    out = {}
    for name, rows in by.items():
        rows.sort(key=lambda r: int(r["Dispatch_Id"]))
        assert len(rows) == times * len(cases()), (path, name, len(rows))
        out[name] = [rows[i:i + times] for i in range(0, len(rows), times)]
    return out


def read(where, times, ctimes):
    trace = groups(os.path.join(where, "t_kernel_trace.csv"), times)[None]
    counted = {}
    for f in "fws":
        for name, g in groups(os.path.join(where, f + "_counter_collection.csv"), ctimes).items():
            counted[name] = [statistics.median(float(r["Counter_Value"]) for r in x) for x in g]
    print("| call | kernel us (least) | read + written MB | algorithmic MB | matrix cores | vector units | LDS conflicts |")
    print("|---|---:|---:|---:|---:|---:|---:|")
    for i, case in enumerate(cases()):
        us = [(int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3 for r in trace[i]]
        busy = counted["SQ_BUSY_CU_CYCLES"][i]
        print("| %s | %.1f (%.1f) | %.1f + %.1f | %.1f | %.0f %% | %.0f %% | %.2f |" % (
            case["name"], statistics.median(us), min(us), counted["FETCH_SIZE"][i] * READ / 1e6, counted["WRITE_SIZE"][i] * 1024 / 1e6,
            operators.work(case)["bytes"] / 1e6, 100 * counted["SQ_VALU_MFMA_BUSY_CYCLES"][i] / (4 * busy),
            100 * counted["SQ_ACTIVE_INST_VALU"][i] / busy, counted["SQ_LDS_BANK_CONFLICT"][i] / max(1, counted["SQ_LDS_IDX_ACTIVE"][i])))


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
