"""bench.py --traffic-summarize on the counter files of a run: the step's kernels are known by
their names as the profiler prints them, with the template arguments that the product's plain form
leaves at their defaults."""
import csv
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

IN = "fp8lin::(anonymous namespace)::"
PLAIN = f"{IN}NoEpilogue"


def dispatches():
    """Kernel names in the order of bench.traffic_run."""
    names = ["void at::native::vectorized_elementwise_kernel<8, at::native::neg_kernel_cuda>(int)"] * 3
    plan = bench.c5_plan()
    for mode in ("delayed", "block"):
        for lab, kind, _ in plan:
            if not lab.startswith(mode) or kind == "gemm":
                continue
            names.append(f"void {IN}" + ("k_history_update<1>(float*)" if kind == "state" else
                                         "k_cast_transpose<0, true>(void*)" if mode == "delayed" else
                                         f"k_cast_block<0, {2 if ' W ' in lab else 1}>(void*)"))
        for lab, kind, _ in plan:
            if lab.startswith(mode) and kind == "gemm":
                k = bench.C5_KERNEL[lab.rsplit(" ", 1)[0]]
                last = f", {PLAIN}, 8>" if "w4" in k else f", {PLAIN}>"
                names += [f"void {IN}{k[:-1]}{last}(fp8lin::GemmParams, int, int, {PLAIN})"] * 2
    return names + [f"void {IN}{k}<1>(void*)" for k in ("k_rw_rows", "k_rw_colmax", "k_rw_transpose", "k_rw_finalize")] * 2


def test_summary_knows_the_steps_kernels(tmp_path, capsys):
    kib = bench.COPY_BYTES / 1024
    for sub, counter in (("fetch", "FETCH_SIZE"), ("write", "WRITE_SIZE")):
        os.makedirs(tmp_path / sub)
        with open(tmp_path / sub / "p_counter_collection.csv", "w", newline="") as f:
            w = csv.writer(f)
            w.writerow(["Dispatch_Id", "Kernel_Name", "Counter_Name", "Counter_Value"])
            for i, name in enumerate(dispatches()):
                w.writerow([i, name, counter, kib if "neg_kernel" in name else 1000 + i])
    out = tmp_path / "out.json"
    bench.traffic_summarize(str(tmp_path), str(out))
    capsys.readouterr()
    got = json.load(open(out))
    assert set(got["kernels"]) == set(bench.C5_KERNEL)
    assert all(e["launches"] == 5 for e in got["kernels"].values())
    assert got["sources_sha256"] == bench.traffic_sources_sha256()
