"""The gated recurrence's and the grouped norm's sums are launched so that they may start while the kernel before them runs: what that one writes is
read plainly, behind the wait (see test_dependent_reads.py; read from the sources, no GPU needed)."""
import os
import re

from test_dependent_reads import CSRC, definition


def test_what_the_launch_before_writes_is_read_plainly():
    parameters, body = definition("k_gated.cu", "gated_sums_kernel")
    assert re.search(r"\bpartial\b", parameters) and not re.search(r"__restrict__\s+partial\b", parameters)
    assert "grid_dep_wait()" in body and "__ldg" not in body[body.index("grid_dep_wait()"):]
    assert body.index("grid_dep_wait()") < body.index("partial[")


def test_every_dependent_kernel_is_known():
    seen = set()
    for file in ("k_gated.cu", "gated.cuh", "group_norm.cuh", "norm.cuh", "k_rotary.cu"):
        seen |= set(re.findall(r"launch_dependent\((\w+)", open(os.path.join(CSRC, file)).read()))
    assert seen == {"gated_sums_kernel"}, "the grouped norm's sums are the layer norm's kernel"
