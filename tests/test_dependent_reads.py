"""A dependent launch may start while the launch before it runs.  What that one writes is then not constant for the kernel:
it may not be read through the read-only path (__ldg), nor through a pointer whose __restrict__ lets a compiler do so or
move the read in front of the wait.  Read from the sources (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "state_space_sequence_ssd_gb300", "csrc")
# kernel -> its file, the parameters that the launch before it writes, and whether it reads nothing else after its wait
KERNELS = {"state_passing_kernel": ("k_state_passing.cu", ["S", "S16", "dec"], True),
           "conv_reduce_kernel": ("k_conv.cu", ["partial"], True),
           "norm_reduce_kernel": ("k_norm.cu", ["partial"], True),
           "selective_hop_kernel": ("k_selective.cu", ["hops", "dtsum"], True),
           "selective_kernel": ("selective_forward.cuh", ["hops"], False),
           "selective_hops_kernel": ("k_selective_bwd.cu", ["hops", "mus", "nu0", "dtsum"], True),
           "selective_block_kernel": ("selective_backward.cuh", ["start", "end"], False),
           "selective_sums_kernel": ("k_selective_bwd.cu", [], True)}


def definition(file, name):
    """(parameters, body) of a kernel, comments taken out."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    at = text.index("{", text.index(")", text.index(name + "(")))
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
        if depth == 0:
            return text[text.index(name + "("):at], text[at:end]


@pytest.mark.parametrize("name", KERNELS)
def test_what_the_launch_before_writes_is_read_plainly(name):
    file, written, alone = KERNELS[name]
    parameters, body = definition(file, name)
    assert "grid_dep_wait()" in body
    for p in written:
        assert re.search(rf"\b{p}\b", parameters), p
        assert not re.search(rf"__restrict__\s+{p}\b", parameters), f"{p} is written while the kernel may run"
    if alone:
        assert "__ldg" not in body[body.index("grid_dep_wait()"):]


def test_every_dependent_kernel_is_listed():
    seen = set()
    for file in ("k_state_passing.cu", "k_conv.cu", "k_norm.cu", "k_selective.cu", "k_selective_bwd.cu", "selective_backward.cuh", "selective_forward.cuh"):
        seen |= set(re.findall(r"launch_dependent\((\w+)", open(os.path.join(CSRC, file)).read()))
    assert seen - {"kernel"} == set(KERNELS) - {"selective_kernel"}  # that one is launched under a generic name
