"""The library's choice between the two kernels of the experts' products, run on the
host from its own header, against the times that both were measured to take.  No GPU."""
import os
import subprocess

from conftest import GOLDEN, ROOT
from q8_quantized_gemv_gb300 import build


def test_the_kernel_chosen_is_about_the_faster(tmp_path):
    exe = str(tmp_path / "moe_rule_check")
    src = os.path.join(ROOT, "tests", "csrc", "moe_rule_check.cu")
    subprocess.run([build.nvcc(), *build.ARCH, "-O1", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", exe, src],
                   check=True, capture_output=True, text=True)
    with open(os.path.join(GOLDEN, "moe_kernel_times.txt")) as f:
        lines = [x for x in f if not x.startswith("#")]
    r = subprocess.run([exe], input="".join(lines), capture_output=True, text=True, timeout=60, check=True)
    chosen = [int(x) for x in r.stdout.split()]
    assert len(chosen) == len(lines) >= 300
    lost = {}
    for line, rows in zip(lines, chosen):
        *_, mode, op, t1, t2 = line.split()
        t = (float(t1), float(t2))
        lost.setdefault((mode, op), []).append(t[rows] / min(t) - 1)
    for of, v in lost.items():
        assert max(v) <= 0.2 and sum(v) / len(v) <= 0.01, (of, max(v), sum(v) / len(v))
