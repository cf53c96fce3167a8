"""Attention with shared prefixes without a GPU: refusals (every check runs
before any CUDA call; the pointers are never dereferenced)."""
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
from test_serve_host import FAKE, lib, refused  # noqa: F401

PREFIX = dict(q=FAKE, kc=FAKE, vc=FAKE, out=FAKE, lse=FAKE, T=8, n_groups=2, cu_req=FAKE,
              ptable=FAKE, pmax=16, plens=FAKE, n_req=4, n_q=2, cu_q=0, table=FAKE, max_pages=8,
              lengths=FAKE, n_pages=10, page_size=16, kps=4096, vps=4096, d=128, heads=4,
              kv_heads=2, dtype=1, out_dtype=0, stream=None)


@pytest.mark.parametrize("change, code, msg", [
    (dict(dtype=0), -2, b"bf16"),
    (dict(out_dtype=2), -1, b"out_dtype"),
    (dict(d=80), -2, b"head dim"),
    (dict(heads=5), -1, b"multiple of kv_heads"),
    (dict(heads=258, kv_heads=2), -2, b"exceeds 128"),
    (dict(T=7), -1, b"n_req * n_q"),
    (dict(n_q=-1), -1, b"n_q"),
    (dict(n_groups=-1), -1, b"n_groups"),
    (dict(pmax=0), -1, b"max_pages"),
    (dict(pmax=1 << 28, n_groups=1), -2, b"max_pages * page_size"),
    (dict(pmax=1 << 20, n_groups=1 << 12), -2, b"n_req * max_pages"),
    (dict(T=1 << 30, n_req=1 << 29, max_pages=1), -2, b"T * heads"),
    (dict(page_size=24), -2, b"page_size"),
    (dict(kps=4095), -1, b"k_page_stride"),
    (dict(cu_q=FAKE + 1), -1, b"cu_q"),
    (dict(cu_req=0), -1, b"NULL"),
    (dict(cu_req=FAKE + 2), -1, b"4-byte"),
    (dict(ptable=0), -1, b"NULL"),
    (dict(plens=FAKE + 2), -1, b"4-byte"),
    (dict(q=FAKE + 8), -1, b"aligned"),
])
def test_prefix_refusals(lib, change, code, msg):  # noqa: F811
    refused(lib, lib.ra_paged_decode_prefix(*{**PREFIX, **change}.values()), code, msg)


def test_empty_calls_are_no_ops(lib):  # noqa: F811
    assert lib.ra_paged_decode_prefix(*{**PREFIX, "T": 0, "n_req": 0, "n_q": 0, "q": 0}.values()) == 0
    assert lib.ra_paged_decode_prefix(*{**PREFIX, "T": 0, "cu_q": FAKE, "cu_req": 0}.values()) == 0


def test_binding_refusals():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="multiple of 3"):
        ra.ra_paged_decode_prefix(q, c, c, i.view(1, 4), i[:1], i[:2], i[:3].view(3, 1), i[:3])
    with pytest.raises(TypeError, match="prefix_lengths"):
        ra.ra_paged_decode_prefix(q, c, c, i.view(1, 4), None, i[:2], i.view(4, 1), i)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_paged_decode_prefix(q, c, c, i.view(1, 4), i[:1], i[:2], i.view(4, 1), i)


@pytest.mark.parametrize("name", ["paged_prefix_kernel.cu", "paged_fp8_kernel.cu"])
def test_a_cta_decides_once_whether_it_runs(name):
    """As test_serve_edges_host.py's test of the other decode kernels: the abort
    flag is read for the early return only inside find_run, between its barriers."""
    import re

    from test_serve_edges_host import source

    kernel = source(name)
    assert "run.stop" in kernel
    assert not re.search(r"(if|\|\||&&|while)[^;{]*[^&\w]\*abort_flag", kernel)


def test_two_rounded_terms_are_below_a_bf16_step():
    """With bf16 output a weight is held in two rounded bf16 terms (8 bits each).
    For w in [1, 2): the first leaves at most half of its step 2^-7, that is 2^-8;
    what is at most 2^-8 has a step of at most 2^-16 (2^-8 itself is exact), of
    which the second leaves half: 2^-17, 2^-9 of what rounding the output may."""
    import numpy as np

    from test_serve_edges_host import rounded

    w = np.random.default_rng(0).uniform(2.0 ** -20, 1, 100000).astype(np.float32)
    hi = rounded(w)
    lo = rounded(w - hi)
    left = np.abs(w.astype(np.float64) - hi - lo)
    assert (left <= 2.0 ** -17 * w).all()
    assert (np.abs(w - hi) > 2.0 ** -9 * w).any()  # one term alone is as coarse as the output
