"""The build says so if the compiler gives a kernel that splits its registers at
run time another number than the split is made for (the library then refuses to
launch it).  No GPU."""
import os

import pytest

from q8_quantized_gemv_gb300 import build

LOG = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_ZN6lkattn16attn_tile_kernelILi0ELi128EEEvNS_8AttnArgsE' for 'sm_103a'
ptxas info    : Function properties for _ZN6lkattn16attn_tile_kernelILi0ELi128EEEvNS_8AttnArgsE
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN6lkattn5otherEv' for 'sm_103a'
ptxas info    : Used 32 registers, used 0 barriers
"""


def test_other_register_counts_stop_the_build():
    with open(os.path.join(build.CSRC, "lk_tile.cu")) as f:
        src = f.read()
    build.check_registers("lk_tile.cu", src, LOG % 168)
    for n in (160, 167, 255):
        with pytest.raises(RuntimeError, match=f"{n} registers"):
            build.check_registers("lk_tile.cu", src, LOG % n)
    with pytest.raises(RuntimeError, match="no register counts"):
        build.check_registers("lk_tile.cu", src, LOG.replace("tile", "tail") % 168)


def test_the_kernels_are_there():
    build.build()  # checked where it compiles
    for name, (kernel, const) in build.SPLIT_KERNELS.items():
        with open(os.path.join(build.CSRC, name)) as f:
            s = f.read()
        assert kernel + "(" in s and const + " = " in s
