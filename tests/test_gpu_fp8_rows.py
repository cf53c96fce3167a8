"""Attention over pages in 8 bits where rows of one KV head weigh values of far
apart scales: every row is as near to the fp64 form of its own keys as if it
stood alone.

Tolerance, by column, relative to the row's own sum S of |p v|: scores off by 4 d u
A (A the largest |q| |k| / sqrt d), weights by less than 2^-16, sums by 2 n u, as in
test_gpu_fp8_decode.py.  Beside it, for columns in which a row's largest weights
meet small codes: a weight times its scale is held to 2^-39 of the largest, w, that
the row has among 32 keys, and a code is at most 448; the value at w has an entry
above 224 scales.  So 32 keys are off by at most 32 * 2 * 2^-39 of p max |v| there,
and all of them by 64 * 2^-39 of the sum of p max |v|.
"""
import math

import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import fp8_ref
from test_gpu_fp8_decode import DEV, U, hold, make8, widen
from test_gpu_rope import np64

pytestmark = pytest.mark.gpu

SHAPES = [
    # new tokens, heads, kv_heads, d, pairs of KV heads an item
    (2, 8, 2, 128, False),    # one group of 8 rows
    (4, 16, 4, 128, False),   # two
    (7, 8, 2, 128, False),    # 28 rows: two row tiles
    (2, 8, 2, 64, False),
    (2, 8, 2, 64, True),
    (4, 16, 4, 64, False),
]
IDS = [f"q{s[0]}-h{s[1]}/{s[2]}-d{s[3]}{'-pairs' if s[4] else ''}" for s in SHAPES]


def scale_token(pages, vs, table, i, at, k):
    """Value `at` of request i times 2^k."""
    ps = pages[0].shape[1]
    pages[3].view(torch.uint8)[int(table[i, at // ps]), :, at % ps] += k
    vs[i][at] = torch.ldexp(vs[i][at].float(), torch.tensor(k, device=DEV)).bfloat16()


def check_rows(out, q, ks, vs, n_q, window=0):
    for i, (k, v) in enumerate(zip(ks, vs)):
        n, (H, d) = k.shape[0], q.shape[1:]
        rows = slice(i * n_q, (i + 1) * n_q)
        qd, kd, vd = np64(q[rows]), np64(k), np64(v)
        ro, _, size = fp8_ref.attention(qd, kd, vd, window=window)
        A = np.linalg.norm(qd, axis=-1).max() * np.linalg.norm(kd, axis=-1).max() / math.sqrt(d)
        top = np.zeros((n_q, H, 1))  # sum of p max |v|
        for j in range(n_q):
            for h in range(H):
                hi = n - n_q + j + 1
                lo = max(0, hi - window) if window else 0
                s = kd[lo:hi, h // (H // k.shape[1])] @ qd[j, h] / math.sqrt(d)
                p = np.exp(s - s.max())
                top[j, h] = (p * np.abs(vd[lo:hi, h // (H // k.shape[1])]).max(-1)).sum() / p.sum()
        bar = (4 * d * U * A + 2.0 ** -16 + 2 * n * U) * size + 64 * 2.0 ** -39 * top
        err = np.abs(np64(out[rows]) - ro)
        assert (err <= bar).all(), f"request {i}: {(err / bar).max():.2e} of the bar"


@pytest.mark.parametrize("k", [30, 41, 110])
@pytest.mark.parametrize("n_q, H, Hkv, d, pairs", SHAPES, ids=IDS)
def test_a_later_token_of_large_values(n_q, H, Hkv, d, pairs, k):
    """The newest token's values are 2^k above all others', and the rows before it
    must not see them."""
    lengths = [200, 77, 1000]
    q, pages, table, lens, ks, vs = make8(lengths, [n_q] * 3, H, Hkv, d, 16, seed=k)
    for i, n in enumerate(lengths):
        scale_token(pages, vs, table, i, n - 1, k)
    out, lse = ra.ra_paged_decode_fp8(q, *pages, widen(table, Hkv) if pairs else table, lens)
    ra.ra_device_status()
    check_rows(out, q, ks, vs, n_q)


@pytest.mark.parametrize("n_q, H, Hkv, d, pairs", SHAPES, ids=IDS)
def test_a_token_of_large_values_behind_some_rows_windows(n_q, H, Hkv, d, pairs):
    """The oldest key that the first row's window holds: later rows do not see it."""
    lengths, window = [200, 77, 1000], 50
    q, pages, table, lens, ks, vs = make8(lengths, [n_q] * 3, H, Hkv, d, 32, seed=5)
    for i, n in enumerate(lengths):
        scale_token(pages, vs, table, i, n - n_q + 1 - window, 60)
    out, lse = ra.ra_paged_decode_fp8(q, *pages, widen(table, Hkv) if pairs else table, lens, window=window)
    ra.ra_device_status()
    check_rows(out, q, ks, vs, n_q, window)


@pytest.mark.parametrize("n_q, H, Hkv, d, pairs", SHAPES, ids=IDS)
def test_a_token_of_large_values_that_some_heads_ignore(n_q, H, Hkv, d, pairs):
    """A value 2^41 above the others' whose key has a score of 0 for even heads and
    one near -44 (a weight of 2^-63) for odd ones."""
    lengths, at = [200, 77, 1000], 70
    q, pages, table, lens, ks, vs = make8(lengths, [n_q] * 3, H, Hkv, d, 16, seed=6)
    q[:, ::2, 0] = 0.0
    q[:, 1::2, 0] = -22.0
    for i in range(3):
        key = torch.zeros(1, Hkv, d, device=DEV)
        key[:, :, 0] = 2.0 * math.sqrt(d)
        code, byte, val = hold(key)
        page, row = int(table[i, at // 16]), at % 16
        pages[0].view(torch.uint8)[page, row] = code[0].view(torch.uint8)
        pages[2].view(torch.uint8)[page, :, row] = byte[0]
        ks[i][at] = val[0]
        scale_token(pages, vs, table, i, at, 41)
    out, lse = ra.ra_paged_decode_fp8(q, *pages, widen(table, Hkv) if pairs else table, lens)
    ra.ra_device_status()
    check_rows(out, q, ks, vs, n_q)
