"""Rows in 8 bits at the largest numbers of the type: what is held and read back
is a number up to 248 * 2^120 = 1.9375 * 2^127, and an infinity from there on."""
import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
from test_gpu_fp8 import DEV, bytes_of, make_pages

pytestmark = pytest.mark.gpu


def test_the_largest_bf16_numbers():
    """All 128 bf16 numbers of [2^127, 2^128), of either sign: steps of 2^120, codes
    128 to 240 in steps of 16 and then 256, halves to even; byte 247 (e = 120)."""
    d, ps = 128, 16
    x = torch.from_numpy(np.ldexp(np.arange(128.0, 256.0), 120)).bfloat16()
    assert float(x[-1]) == torch.finfo(torch.bfloat16).max
    rows = torch.stack((x, -x)).view(2, 1, d).to(DEV)
    pages = make_pages(1, ps, 1, d)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    ra.ra_paged_append_fp8(rows, rows, rows, None, *pages, torch.arange(2, device=DEV), pos)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    n = torch.full((1,), 2, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    read = ra.ra_paged_read_fp8(*pages, table, n, cu, tokens=2)
    ra.ra_device_status()
    c = np.arange(128.0, 256.0)
    code = np.rint(c / 16) * 16  # (rint: halves to even, as the codes' last bit is)
    for held, scale, out in zip(pages[:2], pages[2:], read):
        got = held.double().cpu().numpy()[0, :2, 0]
        np.testing.assert_array_equal(got, np.stack((code, -code)))
        assert (bytes_of(scale)[0, 0, :2] == 247).all()
        want = np.where(c < 248, code * 2.0 ** 120, np.inf)
        np.testing.assert_array_equal(out.double().cpu().numpy()[:, 0], np.stack((want, -want)))
    assert (np.abs(code - c) <= 2.0 ** -4 * c).all()


def test_a_decode_below_the_infinities():
    """Values up to 240 * 2^120 are attended as numbers, beside an entry that is held
    as an infinity."""
    d, ps, n = 64, 16, 5
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device=DEV)
    v = torch.full((n, 1, d), 2.0 ** 120, dtype=torch.bfloat16, device=DEV)
    v[2] = 247.0 * 2.0 ** 120
    v[4, 0, 7] = torch.finfo(torch.bfloat16).max
    pages = make_pages(1, ps, 1, d)
    zero = torch.zeros_like(v)
    pos = torch.zeros(n, dtype=torch.int32, device=DEV)
    ra.ra_paged_append_fp8(zero, zero, v, None, *pages, torch.arange(n, device=DEV), pos)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    lens = torch.full((1,), n, dtype=torch.int32, device=DEV)
    out, _ = ra.ra_paged_decode_fp8(q, *pages, table, lens)
    ra.ra_device_status()
    got = out.double().cpu().numpy()[0, 0]
    # Five equal weights; row 4's other entries are codes 1 of scale 2^120.
    want = (240.0 + 1.0 * 3 + 1.0) / 5 * 2.0 ** 120
    keep = np.arange(d) != 7
    assert (np.abs(got[keep] - want) <= 2.0 ** -20 * want).all()
