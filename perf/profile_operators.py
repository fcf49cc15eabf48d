"""Times and profiles of the training operators over the cases of operators.py,
or, with --block, of the operators inside a block over those of more_operators.py.

  python3 perf/profile_operators.py [--block] --time [--only NAME,NAME]
        microseconds of a pass among others, and captured in a graph where the
        pass can be; inputs change from pass to pass
  python3 perf/profile_operators.py [--block] --profile DIR
        the rocprofv3 passes, each a child with a time limit of its own
  python3 perf/profile_operators.py [--block] --summarize DIR
        profiles/train_operators_*.md (block_operators_*.md) from what --profile
        left in DIR
"""
import argparse
import csv
import importlib
import os
import re
import statistics
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROFILES = os.path.join(ROOT, "profiles")
sys.path.insert(0, ROOT)

TRACED, COUNTED = 30, 6  # passes of a case in the trace, in a counter run
SEEDS = 3
COUNTERS = {"fetch": ["FETCH_SIZE"], "write": ["WRITE_SIZE"], "sq": ["SQ_INSTS_VALU"]}
BLOCK = False  # the operators inside a block
MATRIX, ACTIVE = "SQ_VALU_MFMA_BUSY_CYCLES", "GRBM_GUI_ACTIVE"
SIMDS, XCDS = 1024, 8
CYCLES_FROM = 100.0  # microseconds: of shorter kernels the counter's cycles are largely launch and drain
REGISTER_UNIT = 2  # the tool halves what is allocated (a kernel of 184 registers reads 92)
FETCH_UNIT = 2.0  # a large copy reads this many bytes for each that the counter names
CUS = 256


def module():
    return importlib.import_module("perf.more_operators" if BLOCK else "perf.operators")


def counters():
    return {**COUNTERS, "sq": [*COUNTERS["sq"], MATRIX, ACTIVE]} if BLOCK else COUNTERS


def cases(only=None):
    operators = module()
    operators.own = True
    return [c for c in operators.listed() if not only or c["name"] in only]


def large():
    """The cases whose traffic counts: 10 MB and more."""
    operators = module()
    return [c["name"] for c in cases() if operators.work(c)["bytes"] >= 10e6]


def states(case):
    operators = module()
    return [operators.prepare(case, seed) for seed in range(SEEDS)]


def run_cases(names, passes):
    """The profiled program."""
    import torch

    operators = module()

    for case in cases(names):
        made = states(case)
        torch.cuda.synchronize()
        for k in range(passes):
            operators.run(made[k % SEEDS])
        torch.cuda.synchronize()
        print(case["name"], flush=True)


# ------------------------------------------------------------------------------------------------ times
def best_of(call, passes, rounds=5):
    import torch

    for k in range(10):
        call(k)
    torch.cuda.synchronize()
    best = float("inf")
    for _ in range(rounds):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for k in range(passes):
            call(k)
        end.record()
        torch.cuda.synchronize()
        best = min(best, begin.elapsed_time(end) / passes * 1e3)
    return best


def captured(made):
    """A graph of five passes for each state."""
    import torch

    operators = module()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in made:
            operators.run(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for s in made:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = [operators.run(s) for _ in range(5)]
        graphs.append((graph, kept))
    return graphs


def time_cases(names):
    operators = module()
    for case in cases(names):
        made = states(case)
        eager = best_of(lambda k: operators.run(made[k % SEEDS]), 60)
        made = states(case)  # (no graph of the first ones' leaves may live)
        graphs = captured(made)
        graph = best_of(lambda k: graphs[k % SEEDS][0].replay(), 30) / 5
        print("%-20s %8.2f us  captured %8.2f us" % (case["name"], eager, graph), flush=True)


# ------------------------------------------------------------------------------------------------ profiles
def profile(outdir):
    os.makedirs(outdir, exist_ok=True)
    me = os.path.abspath(__file__)

    def run(name, limit, options, names, passes):
        command = ["timeout", "-s", "KILL", str(limit), "rocprofv3", *options, "--output-format", "csv", "-d",
                   os.path.join(outdir, name), "-o", "t", "--", "python3", me, *(["--block"] if BLOCK else []), "--run", ",".join(names), str(passes)]
        print(name, flush=True)
        subprocess.run(command, check=True)

    run("trace", 100, ["--kernel-trace", "--stats"], [c["name"] for c in cases()], TRACED)
    for name, some in counters().items():
        run(name, 60, ["--pmc", *some], large(), COUNTED)


def kernel_of(row):
    if BLOCK:
        name = row["Kernel_Name"]
        found = re.search(r"attention_(?:forward|join|norms|delta|grads|grad_kv|grad_q)|gated_(?:product|both|finish|slopes|tops|few_rows|copy)|"
                          r"rotary_kernel", name)
        if not found or found[0] != "gated_product":
            return found and found[0]
        # (the tool writes the second product's name with its type and number garbled)
        which = re.search(r"gated_product(?:I(?:DF16b|DF16_|f)Li|<float, )(\d)", name)
        return "gated_product, " + ("forward", "gradient of x", "gradients of weights")[int(which[1]) if which else
                                                                                       2 if "EL, int" in name else 1]
    found = re.search(r"ssim_(?:grad_norm|norm_only|clip|adamw|block_norm)\w*?_kernel", row["Kernel_Name"])
    return found and found[0]


def by_case(rows, names):
    """{case: [(kernel, row)]} of rows in the order of their dispatch: a case's
    launches follow each other, the making of the next one's inputs between."""
    runs, inside = [], False
    for row in rows:
        kernel = kernel_of(row)
        if kernel:
            if not inside:
                runs.append([])
            runs[-1].append((kernel, row))
        inside = bool(kernel)
    if len(runs) != len(names):
        raise RuntimeError(f"{len(runs)} runs of launches for {len(names)} cases")
    return dict(zip(names, runs))


def read(outdir, name, file, order):
    with open(os.path.join(outdir, name, file)) as f:
        return sorted(csv.DictReader(f), key=lambda row: int(row[order]))


def summarize(outdir):
    operators = module()
    times, lines = {}, []
    trace = read(outdir, "trace", "t_kernel_trace.csv", "Start_Timestamp")
    for case, launches in by_case(trace, [c["name"] for c in cases()]).items():
        found = {}
        for kernel, row in launches:
            found.setdefault(kernel, []).append(row)
        for kernel, rows in found.items():
            us = [(int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3 for r in rows]
            times[case, kernel] = statistics.median(us)
            r = rows[-1]
            threads = int(r["Workgroup_Size_X"])
            lines.append("| %s | %s | %d | %.2f | %.2f | %d x %s, %d | %s | %s |" % (
                case, kernel, len(us), times[case, kernel], min(us), int(r["Grid_Size_X"]) // threads,
                r["Grid_Size_Y"], threads, REGISTER_UNIT * int(r["VGPR_Count"]), r["Scratch_Size"]))
    what, file = ("operators inside a block", "block") if BLOCK else ("training operators", "train")
    with open(os.path.join(PROFILES, file + "_operators_kernel_trace.md"), "w") as f:
        f.write(f"""# Kernel times of the {what} (rocprofv3 --kernel-trace), MI355X

By `perf/profile_operators.py`: one process, each case of `perf/{module().__name__[5:]}.py` {TRACED} times over {SEEDS} sets
of inputs in turn. Times in microseconds. Profiled kernels of a few microseconds read 0.3 to 1 us
longer than unprofiled ones. Registers are those allocated to a thread, vector and accumulation registers
together ({REGISTER_UNIT} times the tool's number), of 512 that the waves of a SIMD share.

| case | kernel | calls | median us | least us | workgroups, threads | registers | scratch B |
|---|---|---|---|---|---|---|---|
""" + "\n".join(lines) + "\n")

    counts = {}
    for name in counters():
        for case, launches in by_case(read(outdir, name, "t_counter_collection.csv", "Dispatch_Id"), large()).items():
            found = {}
            for kernel, row in launches:
                found.setdefault((kernel, row["Counter_Name"]), []).append(float(row["Counter_Value"]))
            for key, values in found.items():
                counts[(case, *key)] = statistics.median(values)
    need = {c["name"]: operators.work(c)["bytes"] / 1e6 for c in cases()}
    lines = []
    for case in large():
        total = 0.0
        for (of, kernel), us in times.items():
            if of != case:
                continue
            fetched = FETCH_UNIT * counts[case, kernel, "FETCH_SIZE"] * 1024 / 1e6
            written = counts[case, kernel, "WRITE_SIZE"] * 1024 / 1e6
            total += fetched + written
            lines.append("| %s | %s | %.1f | %.1f | %.0f | %.2f |" % (
                case, kernel, fetched, written, (fetched + written) / us * 1e3,
                counts[case, kernel, "SQ_INSTS_VALU"] / CUS / (us * 1e3)))
            if BLOCK:
                busy, active = (counts[case, kernel, c] for c in (MATRIX, ACTIVE))
                lines[-1] += " %.0f%% | %.2f |" % (100 * busy / SIMDS / (active / XCDS), active / XCDS / us / 1e3) \
                    if us >= CYCLES_FROM else " | |"
        lines.append("| %s | all; the case needs %.1f | %.1f | | | |" % (case, need[case], total) + " | |" * BLOCK)
    matrix = f""" The share of the kernel's
cycles in which a matrix instruction runs, over all SIMDs, and the cycles in GHz of its time in the trace (the
counter run's own is a little longer); left out below {CYCLES_FROM:.0f} us, where launch and drain, which the
cycles include, are a large part of them.""" if BLOCK else ""
    more = (" matrix | GHz |", "---|---|") if BLOCK else ("", "")
    with open(os.path.join(PROFILES, file + "_operators_counters.md"), "w") as f:
        f.write(f"""# Traffic and vector instructions of the {what} (rocprofv3 --pmc), MI355X

By `perf/profile_operators.py`. FETCH_SIZE (times {FETCH_UNIT:g}, as a copy calibrates it) and WRITE_SIZE in MB
per call of a kernel (between the L2s and the memory side, whose 256 MB cache answers some of it), their
sum over the kernel's median time in `{file}_operators_kernel_trace.md` in GB/s, and vector wave
instructions per compute unit and nanosecond (streams of them reach 3.2 to 4.1). Each counter in a run of
its own, over {SEEDS} sets of inputs in turn, {COUNTED} times a case.{matrix}

| case | kernel | read MB | written MB | GB/s | VALU per CU per ns |{more[0]}
|---|---|---|---|---|---|{more[1]}
""" + "\n".join(lines) + "\n")


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--block", action="store_true", help="the operators inside a block")
    ap.add_argument("--time", action="store_true")
    ap.add_argument("--only", default="", help="cases of --time, by name (default: all)")
    ap.add_argument("--profile", metavar="DIR")
    ap.add_argument("--summarize", metavar="DIR")
    ap.add_argument("--run", nargs=2, metavar=("CASES", "PASSES"), help=argparse.SUPPRESS)
    a = ap.parse_args()
    BLOCK = a.block
    if a.run:
        run_cases(a.run[0].split(","), int(a.run[1]))
    elif a.time:
        time_cases(a.only.split(",") if a.only else None)
    elif a.profile:
        profile(a.profile)
    elif a.summarize:
        summarize(a.summarize)
    else:
        ap.error("one of --time, --profile and --summarize")
