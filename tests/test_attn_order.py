"""What the attention step's kernels must not do under dependent launches, read
from their source: a kernel that may start while its predecessors run
(programmatic dependent launch) sees their writes only behind its own
griddepcontrol.wait.  A stale read shows in no result as long as the timing is
kind, so the order in the source is the test.  No GPU."""
import glob
import os
import re

import pytest

from q8_quantized_gemv_gb300 import build

# where each kernel first reads what a caller's earlier launch may have written, or
# takes what such a launch may still be waiting for (tensor memory)
KERNELS = [("lk_attn.cu", "attn_body(", "make_deal"), ("lk_attn.cu", "attn_body(", "a.lens"),
           ("lk_attn.cu", "attn_body(", "a.q"), ("lk_attn.cu", "attn_join_kernel(", "z.ml"),
           ("lk_attn.cu", "attn_join_kernel(", "z.o"), ("lk_tile.cu", "attn_tile_kernel(", "make_deal"),
           ("lk_tile.cu", "attn_tile_kernel(", "a.q"), ("lk_tile.cu", "attn_tile_kernel(", "tm_alloc"), ("lk_kv.cu", "kv_append_kernel(", "__ldcg"),
           ("lk_kv.cu", "kv_append_kernel(", "a.lens")]


def source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernel_body(file, kernel):
    s = source(file)
    at = s.index(kernel)
    return s[at:s.index("\n}\n", at)]


@pytest.mark.parametrize("file,kernel,read", KERNELS)
def test_waits_before_it_reads(file, kernel, read):
    body = kernel_body(file, kernel)
    wait = body.index("griddepcontrol.wait")
    assert wait < re.search(re.escape(read) + r"(?![a-z0-9_])", body).start()
    line = body[body.rindex("\n", 0, wait):wait]
    assert "if" not in line, "the wait is not conditional: " + line


def test_tensor_memory_is_taken_before_dependents_start():
    """One that wants some too and got it first would wait for this launch, and this
    launch for it."""
    body = kernel_body("lk_tile.cu", "attn_tile_kernel(")
    assert body.count("griddepcontrol.launch_dependents") == 1
    taken = body.index("tm_alloc")
    assert taken < body.index("__syncthreads();", taken) < body.index("griddepcontrol.launch_dependents")


def test_join_reads_the_lengths_again():
    """The join works its deal out ahead of the wait; what it does behind it
    follows from lengths that it read there."""
    body = kernel_body("lk_attn.cu", "attn_join_kernel(")
    after = body[body.index("griddepcontrol.wait"):]
    again = re.search(r"const int2 now = lens_pair\(a\);.*?if \(__syncthreads_or\(other\)\) \{\s*lens = now;\s*deals\(\);", after, re.S)
    assert again and again.end() < after.index("ld_cg")


@pytest.mark.parametrize("file", ["lk_kv.cu", "lk_attn.cu", "lk_tile.cu", "lk_attn.cuh", "lk_tc.cuh"])
def test_no_loads_by_the_read_only_path(file):
    """That path promises that nobody writes for the kernel's whole life, which
    begins while its predecessors run."""
    s = source(file)
    assert "__ldg(" not in s and ".nc" not in s and "__restrict__" not in s


def test_error_bits_tell_the_waits_apart():
    """Every wait of the library that can run out has a bit of its own in the
    device error word."""
    bits = {}
    for f in glob.glob(os.path.join(build.CSRC, "*.cu*")):
        for name, v in re.findall(r"\b(ERR_[A-Z_]+) = (\d+)", source(os.path.basename(f))):
            bits[f"{os.path.basename(f)} {name}"] = int(v)
    assert len(bits) >= 8 and all(v & (v - 1) == 0 for v in bits.values())
    assert len(set(bits.values())) == len(bits), bits
    with open(os.path.join(build.INCLUDE, "lk_attn.h")) as f:
        doc = f.read()
    for name in ("ERR_ATTN_WAIT", "ERR_TILE_WAIT"):
        assert f"{bits['lk_attn.cuh ' + name]} in the" in doc
