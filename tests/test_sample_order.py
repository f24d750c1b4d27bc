"""What lk_sample's kernel must not do, read from its source.  No GPU.

The blocks of a cluster are on the GPU at the same time, but nothing says that one
has begun when another reaches for its shared memory: that takes a cluster barrier
first.  A missing one shows in no result as long as the timing is kind, so the
order in the source is the test."""
import os
import re

from q8_quantized_gemv_gb300 import build


def body():
    with open(os.path.join(build.CSRC, "lk_sample.cu")) as f:
        s = re.sub(r"//[^\n]*", "", f.read())
    at = s.index("void run(const SampleArgs")
    return s[at:s.index("\n};\n", at)]


def test_blocks_have_begun_before_one_reaches_into_another():
    b = body()
    arrive, wait = b.index("barrier.cluster.arrive"), b.index("barrier.cluster.wait")
    first = min(m.start() for m in re.finditer(r"map_shared_rank|meet\(\);", b))
    assert arrive < wait < first
    assert b.count("barrier.cluster.arrive") == b.count("barrier.cluster.wait") == 1
    # both by all threads of all blocks of a row: ahead of the branch of one warp, and
    # under no condition but that there are several blocks
    assert wait < b.index("if (warp == 0)")
    for at in (arrive, wait):
        line = b[b.rindex("\n", 0, at):at]
        assert re.fullmatch(r"\s*if \(C > 1\) asm volatile\(\"", line), line
    # the arrival comes before anything is waited for: the row's read hides it
    assert arrive < b.index("griddepcontrol.wait") < wait
