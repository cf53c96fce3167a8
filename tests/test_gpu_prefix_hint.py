"""Which launches a call over shared prefixes makes goes by the rows that the
caller says to expect, as in the paged decode, and not by padding rows."""
import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
from test_gpu_paged import check_decode, i32
from test_gpu_prefix import DEV, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q, launches", [(1, [0, 1, 1]), (0, [1, 1, 1]), (64, [1, 1, 1])])
def test_padding_rows_are_nobodys(n_q, launches):
    """A step of 256 rows, one each for 8 requests of one group and the others
    padding: with n_q = 1 32 rows of a KV head, which go with the own keys in one
    launch; with no such word 1024."""
    rows = [1] * 8
    args, k, v = make([(1001, [300, 1, 20, 77, 64, 65, 2, 150])], rows, 32, 8, 128, 16, extra=248)
    out = torch.full(args[0].shape, 9.0, device=DEV)
    lse = torch.full(args[0].shape[:2], 9.0, device=DEV)
    cu = i32(np.arange(9))
    ra.ra_trace_enable()
    ra.ra_trace_reset()
    try:
        ra.ra_paged_decode_prefix(*args, cu_q=cu, n_q=n_q, out=out, lse=lse)
        torch.cuda.synchronize()
        assert [ra.ra_trace_query(x)[0] for x in ("paged_decode", "paged_prefix", "paged_combine")] == launches
    finally:
        ra.ra_trace_enable(False)
    ra.ra_device_status()
    check_decode(out, lse, args[0], k, v, rows)
    assert (out[8:] == 9.0).all() and (lse[8:] == 9.0).all()
