"""A block that gives up a wait leaves only when its copies in flight have landed:
what bounds the waits for these is no shorter than a second, however short the
option wait_us is.  Read from the source.  No GPU."""
import glob
import os
import re

import pytest

from q8_quantized_gemv_gb300 import build


def source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("file,helper", [("lk_ring_kernel.cuh", "drain_wait"), ("lk_tc.cuh", "bar_drain")])
def test_copies_in_flight_have_a_second_at_least(file, helper):
    s = source(file)
    at = s.index(f"{helper}(unsigned bar, unsigned parity, unsigned long long limit_ns")
    body = s[at:s.index("\n}\n", at)]
    floor = re.search(r"limit = limit_ns > (\w+) \? limit_ns : \1;", body)
    assert floor, body
    v = floor.group(1)
    named = re.search(rf"{v} = (\d+)ull", s)
    assert int(named.group(1) if named else v.rstrip("ul")) >= 10 ** 9
    assert "> limit_ns)" not in body and "- t0 > limit)" in body


def test_every_kernel_that_bounds_its_waits_drains():
    """The kernels with copies of their own and a way to give up."""
    for name in (os.path.basename(p) for p in glob.glob(os.path.join(build.CSRC, "lk_*.cu*"))):
        s = source(name)
        if "__global__" in s and re.search(r"\braise_error\(|abort_flag = 1", s):
            assert re.search(r"\b(drain_wait|bar_drain)\(", s), name
