"""The kernels' sources and arithmetic, as far as they can be checked without
a GPU."""
import os
import re

import numpy as np
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
    """The same in the fused ring forward, where the decision has a word of its
    own that no wait writes.  (The other kernels read the flag between two
    barriers.)"""
    code = source("umma_kernel.cu")
    ring = code[code.index("umma_ring_kernel(const __grid_constant__"):]
    ring = ring[:ring.index("regs_dec")]
    assert re.search(r"if \(no_keys \|\| \*stop\)", ring) and ring.count("*stop =") == 1
    assert not re.search(r"(if|\|\||&&|while)[^;{]*[^&\w]\*abort_flag(?!\s*=[^=])", ring)


# ------------------------------------------------------------------ the weights' bar

def rounded(x):
    """fp32 to bf16, to nearest even."""
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7fff + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)).view(np.float32)


def cut(x):
    return (x.astype(np.float32).view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)


@pytest.mark.parametrize("head", [rounded, cut])
def test_the_bar_on_the_weights_sees_a_lost_term(head):
    """The GPU test of the paged decode's weights (three live keys, scores in
    [-1, 1], an output is one weight of their sum) refuses more than 32 u.
    Three bf16 terms hold fp32's 24 bits; two miss the bar, at the fewest
    rows that the test has (24 of three keys)."""
    s = np.random.default_rng(0).uniform(-1, 1, (24, 3))
    p = np.exp(s - s.max(1, keepdims=True)).astype(np.float32)
    total, rest, err = np.zeros_like(p, dtype=np.float64), p, []
    for _ in range(3):
        h = head(rest)
        total += h
        rest = rest - h
        err.append(np.abs(total / p - 1).max() * 2.0 ** 24)
    assert err[0] > 1000 and err[1] > 2 * 32 and err[2] <= 1
