"""Plain 64-bit forms of rows held in 8 bits and of attention over pages, for
the tests (numpy)."""
import numpy as np


def code_values():
    """The values of the 256 e4m3 codes: sign, four bits of exponent, three of
    mantissa, 0x7f and 0xff NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def quantise(x):
    """Rows of x [..., d] as (code values, scale exponents): the least e in
    [-117, 120] with max |x| <= 448 2^e, codes to nearest, halves to even."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x)
    top = np.where(fine, np.abs(x), 0).max(-1)
    e = np.full(top.shape, -117)
    for _ in range(240):
        e = np.where((top > 448.0 * 2.0 ** e.astype(np.float64)) & (e < 120), e + 1, e)
    y = np.where(fine, x, 0) / (2.0 ** e.astype(np.float64))[..., None]
    p = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -60)))
    p = np.where(np.abs(y) < 2.0 ** p, p - 1, p)
    step = 2.0 ** (np.maximum(p, -6) - 3)
    return np.where(fine, np.rint(y / step) * step, np.nan), e


def paged_rows(pages, table, length, page_size):
    """The first `length` rows [length, kv_heads, d] of a request's pages."""
    ids = np.asarray(table)[:-(-length // page_size)]
    return pages[ids].reshape(-1, *pages.shape[2:])[:length]


def attention(q, k, v, n_shared=0, window=0):
    """Rows q [n, heads, d] at the last n positions after k's, v's rows [t,
    kv_heads, d]; all rows see the first n_shared of them.  (out, lse, and the
    sums of absolute terms of out.)"""
    n, H, d = q.shape
    t, hkv = k.shape[0], k.shape[1]
    g = H // hkv
    out, size, lse = np.zeros((n, H, d)), np.zeros((n, H, d)), np.full((n, H), -np.inf)
    for j in range(n):
        hi = max(t - n + j + 1, n_shared)
        lo = max(0, hi - window) if window else 0
        if hi <= lo:
            continue
        for h in range(H):
            s = k[lo:hi, h // g] @ q[j, h] / np.sqrt(d)
            m = s.max()
            p = np.exp(s - m)
            lse[j, h] = m + np.log(p.sum())
            out[j, h] = p @ v[lo:hi, h // g] / p.sum()
            size[j, h] = p @ np.abs(v[lo:hi, h // g]) / p.sum()
    return out, lse, size
