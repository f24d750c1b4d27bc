"""The attention step's deal of key units to blocks, run on the host from the
library's own header: no product of it may pass 32 bits for a number of units
that the calls accept.  No GPU."""
import os
import subprocess

from conftest import ROOT
from q8_quantized_gemv_gb300 import build


def test_every_number_of_units_is_dealt_whole(tmp_path):
    exe = str(tmp_path / "deal_check")
    src = os.path.join(ROOT, "tests", "csrc", "deal_check.cu")
    subprocess.run([build.nvcc(), *build.ARCH, "-O1", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", exe, src],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
