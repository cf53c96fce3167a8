"""The kernels' sources and arithmetic, as far as they can be checked without
a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "blockwise_online_softmax_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["paged_kernel.cu", "paged_tc_kernel.cu"])
def test_a_cta_decides_once_whether_it_runs(name):
    """A warp's first wait may raise the abort flag.  A kernel that lets each
    warp read the flag for its early return could lose one warp of a group
    whose others then wait for it at a barrier without a limit.  The flag is
    read between the barriers of find_run, where no warp can wait yet."""
    kernel = source(name)
    assert "run.stop" in kernel
    assert not re.search(r"(if|\|\||&&|while)[^;{]*[^&\w]\*abort_flag", kernel)
    walk = source("paged_walk.cuh")
    body = walk[walk.index("Run find_run("):]
    body = body[:body.index("return run;")]
    first, second = (m.start() for m in re.finditer(r"__syncthreads\(\)", body))
    assert first < body.index("*abort_flag != 0") < second


def test_the_fused_ring_decides_once_whether_it_runs():
    """The same in the fused ring forward, where the barrier in front of the
    roles carries the decision.  (The other kernels read the flag between two
    barriers.)"""
    code = source("umma_kernel.cu")
    ring = code[code.index("umma_ring_kernel(const __grid_constant__"):]
    ring = ring[:ring.index("regs_dec")]
    assert "__syncthreads_or(launch_status)" in ring
    assert not re.search(r"(if|\|\||&&|while)[^;{]*[^&\w]\*abort_flag(?!\s*=[^=])", ring)
