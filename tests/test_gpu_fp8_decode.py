"""Attention over pages in 8 bits on the GPU, against the fp64 oracle over the
values that the codes and scales stand for (exact in bf16).

Tolerances are those of the paged decode (test_gpu_paged.py: scores off by d u A,
weights by less than 2^-16, sums by n u), and for single weights a bound of
their own below.
"""
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import oracle
from test_gpu_paged import check_decode, i32, pool
from test_gpu_rope import np64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
CODE, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu
U = 2.0 ** -24


def hold(x):
    """Rows of x (fp32) as codes and scale bytes, and their values in bf16."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = (e - 9 + (m > 0.875)).clamp(-117, 120)
    code = torch.ldexp(x, -e).to(CODE)
    return code, (e[..., 0] + 127).to(torch.uint8), torch.ldexp(code.float(), e).bfloat16()


def make8(lengths, rows, H, Hkv, d, ps, *, seed=0, scale=1.5, together=False, extra=0, spread=0):
    """Random pages with NaN codes and NaN scales behind every request's last
    token and in the pages of nobody; scales differ by up to 2^spread."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    width = max(1, max(-(-n // ps) for n in lengths)) + 1
    n_pages = sum(-(-n // ps) for n in lengths) + 3
    table, _, _ = pool(lengths, ps, width, n_pages, seed)
    c = torch.full((n_pages, 2, ps, Hkv, d), 0xff, dtype=torch.uint8, device=DEV)
    s = torch.full((n_pages, 2, Hkv, ps), 0xff, dtype=torch.uint8, device=DEV)
    vals = [[], []]
    for i, n in enumerate(lengths):
        for side in range(2):
            x = torch.randn(n, Hkv, d, generator=g, device=DEV)
            if spread:
                x = torch.ldexp(x, torch.randint(-spread, 1, (n, Hkv, 1), generator=g, device=DEV))
            if n == 0:
                vals[side].append(x.bfloat16())
                continue
            code, byte, val = hold(x)
            vals[side].append(val)
            for p in range(-(-n // ps)):
                part = slice(p * ps, min(n, p * ps + ps))
                c[table[i, p], side, :part.stop - part.start] = code[part].view(torch.uint8)
                s[table[i, p], side, :, :part.stop - part.start] = byte[part].t()
    table[table < 0] = 2**30  # never read
    q = (torch.randn(sum(rows) + extra, H, d, generator=g, device=DEV) * scale).bfloat16()
    pages = [c[:, 0].view(CODE), c[:, 1].view(CODE), s[:, 0].view(SCALE), s[:, 1].view(SCALE)]
    if not together:
        pages = [x.contiguous() for x in pages]
    return q, pages, i32(table), i32(lengths), vals[0], vals[1]


CASES = [
    # lengths, rows per request, heads, kv_heads, d, page size, window
    ([1], 1, 1, 1, 64, 16, 0),
    ([1, 0, 2], 1, 8, 2, 128, 16, 0),
    ([127, 128, 129, 0, 5], 1, 32, 8, 128, 16, 0),
    ([1000], 1, 32, 8, 128, 64, 0),
    ([5000, 3, 70], 1, 4, 4, 128, 256, 0),
    ([700, 255, 256, 257], 1, 12, 4, 64, 128, 0),
    ([4097, 600], 1, 8, 1, 64, 32, 100),
    ([333, 64, 2000], 2, 64, 8, 128, 16, 0),      # 16 rows per KV head
    ([333, 64, 2000], 3, 12, 4, 128, 32, 37),
    ([50, 4, 900], 4, 32, 8, 64, 16, 0),
    ([17, 2500], 5, 32, 8, 128, 64, 0),           # 20 rows
    ([300, 129], 16, 8, 8, 128, 32, 0),
    ([900, 128, 140], 16, 64, 8, 64, 16, 1),      # 128 rows, window of one key
    ([600, 90], 3, 128, 1, 128, 16, 0),           # 128 heads on one KV head
    ([3, 1000, 2], 3, 16, 16, 64, 128, 0),        # rows before the first key
    ([1000, 20], 70, 8, 2, 128, 16, 300),         # more rows than keys
    ([40000, 9, 12345], 1, 32, 8, 128, 64, 0),
    ([12345], 1, 8, 8, 64, 16, 5000),
    ([int(x) for x in np.random.default_rng(1).integers(0, 300, 300)], 1, 8, 2, 64, 16, 0),
]


@pytest.mark.parametrize("together, spread", [(False, 0), (True, 12)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0][:4])}-q{c[1]}-h{c[2]}/{c[3]}"
                         f"-d{c[4]}-p{c[5]}-w{c[6]}")
def test_decode_fp8(case, together, spread):
    lengths, n_q, H, Hkv, d, ps, window = case
    rows = [n_q] * len(lengths)
    q, pages, table, lens, ks, vs = make8(lengths, rows, H, Hkv, d, ps, together=together, spread=spread)
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens, window=window)
    ra.ra_device_status()
    check_decode(out, lse, q, ks, vs, rows, window)
    again = ra.ra_paged_decode_fp8(q, *pages, table, lens, window=window)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def widen(table, heads):
    """The same table with room for so many pages that pairs of KV heads of 64
    columns make an item (pages behind a request's last are never read)."""
    width = (1 << 19) // (table.shape[0] * 16 * heads) + table.shape[1]
    wide = torch.full((table.shape[0], width), 2**30, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    return wide


PAIRS = [
    # lengths, rows per request, heads, kv_heads, page size, window
    ([1, 0, 2], 1, 8, 2, 16, 0),
    ([700, 255, 256, 257], 1, 12, 4, 128, 0),
    ([4097, 600], 1, 16, 8, 32, 100),
    ([333, 64, 2000], 2, 16, 4, 16, 37),
    ([50, 4, 900], 4, 8, 4, 64, 0),
    ([3, 1000, 2], 3, 16, 16, 256, 0),            # rows before the first key
    ([40000, 9, 12345], 1, 32, 8, 64, 0),
    ([int(x) for x in np.random.default_rng(1).integers(0, 300, 300)], 1, 8, 2, 16, 0),
]


@pytest.mark.parametrize("together, spread", [(False, 0), (True, 12)])
@pytest.mark.parametrize("case", PAIRS, ids=lambda c: f"{str(c[0][:4])}-q{c[1]}-h{c[2]}/{c[3]}-p{c[4]}-w{c[5]}")
def test_pairs_of_heads(case, together, spread):
    lengths, n_q, H, Hkv, ps, window = case
    rows = [n_q] * len(lengths)
    q, pages, table, lens, ks, vs = make8(lengths, rows, H, Hkv, 64, ps, together=together, spread=spread, seed=7)
    wide = widen(table, Hkv)
    out, lse = ra.ra_paged_decode_fp8(q, *pages, wide, lens, window=window)
    ra.ra_device_status()
    check_decode(out, lse, q, ks, vs, rows, window)
    again = ra.ra_paged_decode_fp8(q, *pages, wide, lens, window=window)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    bf = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    _, lse2 = ra.ra_paged_decode_fp8(q, *pages, wide, lens, window=window, out=bf)
    assert torch.equal(bf, out.bfloat16()) and torch.equal(lse2, lse)


def test_pairs_of_heads_with_ragged_rows():
    for rows in ([1, 0, 3, 1], [0, 0, 2, 0], [40, 1, 0, 7]):
        q, pages, table, lens, ks, vs = make8([500, 77, 300, 1025], rows, 8, 2, 64, 16, extra=5)
        out = torch.full(q.shape, 9.0, device=DEV)
        lse = torch.full(q.shape[:2], 9.0, device=DEV)
        cu = i32(np.concatenate([[0], np.cumsum(rows)]))
        ra.ra_paged_decode_fp8(q, *pages, widen(table, 2), lens, cu_q=cu, n_q=1, out=out, lse=lse)
        ra.ra_device_status()
        check_decode(out, lse, q, ks, vs, rows)
        assert (out[-5:] == 9.0).all() and (lse[-5:] == 9.0).all()


@pytest.mark.parametrize("rows", [[1, 0, 3, 1], [0, 0, 2, 0], [40, 1, 0, 7]])
def test_ragged_rows(rows):
    """cu_q: idle requests, several rows, and rows behind the last request
    left as they were."""
    q, pages, table, lens, ks, vs = make8([500, 77, 300, 1025], rows, 8, 2, 128, 16, extra=5)
    out = torch.full(q.shape, 9.0, device=DEV)
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    cu = i32(np.concatenate([[0], np.cumsum(rows)]))
    ra.ra_paged_decode_fp8(q, *pages, table, lens, cu_q=cu, out=out, lse=lse)
    check_decode(out, lse, q, ks, vs, rows)
    assert (out[-5:] == 9.0).all() and (lse[-5:] == 9.0).all()
    for n_q in (1, 8):  # what is expected does not decide the result
        o2, l2 = ra.ra_paged_decode_fp8(q, *pages, table, lens, cu_q=cu, n_q=n_q)
        check_decode(o2, l2, q, ks, vs, rows)


def test_bf16_output_is_the_fp32_one_rounded():
    for n_q, H, Hkv, d in [(1, 8, 2, 64), (1, 32, 8, 128), (4, 16, 4, 128), (9, 8, 4, 64)]:
        q, pages, table, lens, _, _ = make8([700, 45, 3000], [n_q] * 3, H, Hkv, d, 32)
        want = ra.ra_paged_decode_fp8(q, *pages, table, lens)
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
        _, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens, out=out)
        assert torch.equal(out, want[0].bfloat16()) and torch.equal(lse, want[1])


@pytest.mark.parametrize("n_q, H, Hkv, d, window", [(1, 32, 8, 128, 0), (3, 12, 4, 64, 700), (2, 8, 8, 128, 0)])
def test_near_the_decode_over_the_same_values_in_bf16(n_q, H, Hkv, d, window):
    """Both are within (2 d u A + 2^-16 + n u) max|V| of the oracle."""
    lengths = [2100, 333]
    q, pages, table, lens, ks, vs = make8(lengths, [n_q] * 2, H, Hkv, d, 16)
    n_pages = pages[0].shape[0]
    kc = torch.zeros(n_pages, 16, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    tab = table.cpu()
    for i, n in enumerate(lengths):
        for p in range(-(-n // 16)):
            part = slice(p * 16, min(n, p * 16 + 16))
            kc[tab[i, p], :part.stop - part.start] = ks[i][part]
            vc[tab[i, p], :part.stop - part.start] = vs[i][part]
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens, window=window)
    ref, rlse = ra.ra_paged_decode(q, kc, vc, table, lens, window=window)
    A = float(q.float().norm(dim=-1).max()) * max(float(k.float().norm(dim=-1).max()) for k in ks) / math.sqrt(d)
    bar = 2 * (4 * d * U * A + 2.0 ** -16 + 2 * max(lengths) * U) * max(float(v.abs().max()) for v in vs)
    assert float((out - ref).abs().max()) <= bar
    assert float((lse - rlse).abs().max()) <= 2 * (2 * d * U * A + 2 * max(lengths) * U + 8 * U * 12)


# ------------------------------------------------------------------ numbers

@pytest.mark.parametrize("qmag", [-90, -40, 0, 40])
def test_query_magnitudes(qmag):
    """Rows of q of any size, entries 2^20 apart among them: scores of order 1
    by keys of the inverse size."""
    H, Hkv, d, ps, n = 8, 2, 128, 16, 300
    q, pages, table, lens, ks, vs = make8([n], [1], H, Hkv, d, ps, seed=3)
    q = torch.ldexp(q.float(), torch.full_like(q, qmag, dtype=torch.int32))
    q[:, :, ::3] = torch.ldexp(q[:, :, ::3], torch.tensor(-20, device=DEV))
    q = q.bfloat16()
    pages[2].view(torch.uint8)[:] = torch.where(
        pages[2].view(torch.uint8) == 0xff, 0xff,
        pages[2].view(torch.uint8).int() - qmag).to(torch.uint8)
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens)
    ra.ra_device_status()
    # The powers of two cancel: the reference and its bar are those of order 1.
    check_decode(out, lse, torch.ldexp(q.float(), torch.tensor(-qmag, device=DEV)).bfloat16(), ks, vs, [1])


@pytest.mark.parametrize("vmag", [-109, -60, 60, 110])
def test_value_magnitudes(vmag):
    """Values at the ends of the scales' range (fp32's normal range on the way)."""
    q, pages, table, lens, ks, vs = make8([700, 20], [2, 2], 8, 2, 64, 32, seed=4)
    b = pages[3].view(torch.uint8)
    b[:] = torch.where(b == 0xff, 0xff, (b.int() + vmag).clamp(10, 247)).to(torch.uint8)
    vs = [torch.ldexp(v.float(), torch.full_like(v, vmag, dtype=torch.int32)) for v in vs]
    ok = all(float(v.abs().max()) < 3e38 for v in vs)
    assert ok
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens)
    ra.ra_device_status()
    # (as doubles, scaled to order 1: the bar is relative to max |V|)
    up = 2.0 ** -vmag
    check_decode(torch.from_numpy(np64(out) * up), lse, q, ks,
                 [torch.from_numpy(np64(v) * up).bfloat16() for v in vs], [2, 2])


def test_a_token_of_large_values_beside_small_ones():
    """A value of a scale 2^40 above the others', with next to no weight: the
    others keep theirs (their sum is what an fp32 sum keeps of it)."""
    H, Hkv, d, ps, n = 4, 2, 128, 16, 200
    q, pages, table, lens, ks, vs = make8([n], [1], H, Hkv, d, ps, seed=9)
    tab = table.cpu()
    at = 77
    pages[3].view(torch.uint8)[tab[0, at // ps], :, at % ps] += 40
    vs[0][at] = torch.ldexp(vs[0][at].float(), torch.tensor(40, device=DEV)).bfloat16()
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens)
    ro, _ = oracle.attention(q.cpu(), ks[0].cpu(), vs[0].cpu(), causal=True, q_pos=np.array([n - 1]),
                             k_pos=np.arange(n))
    A = float(q.float().norm(dim=-1).max() * ks[0].float().norm(dim=-1).max()) / math.sqrt(d)
    _, _, size = attention_size(q, ks[0], vs[0])
    assert (np.abs(np64(out) - ro) <= (4 * d * U * A + 2.0 ** -16 + 2 * n * U) * size).all()


def attention_size(q, k, v):
    import fp8_ref

    return fp8_ref.attention(np64(q), np64(k), np64(v))


def test_codes_of_every_kind():
    """All 254 finite codes in k and v."""
    H = Hkv = 2
    d, ps, n = 64, 16, 320
    g = torch.Generator(device=DEV).manual_seed(8)
    c = torch.randint(0, 256, (20, 2, ps, Hkv, d), generator=g, device=DEV, dtype=torch.uint8)
    c[(c & 127) == 127] = 0
    e = torch.randint(118, 122, (20, 2, Hkv, ps), generator=g, device=DEV, dtype=torch.uint8)
    pages = [c[:, 0].view(CODE), c[:, 1].view(CODE), e[:, 0].view(SCALE), e[:, 1].view(SCALE)]
    val = c.view(CODE).float() * e.view(SCALE).float().transpose(2, 3)[..., None]
    ks, vs = (val[:, x].reshape(n, Hkv, d).bfloat16() for x in range(2))
    q = (torch.randn(3, H, d, generator=g, device=DEV) * 0.3).bfloat16()
    out, lse = ra.ra_paged_decode_fp8(q, *pages, torch.arange(20, device=DEV, dtype=torch.int32).view(1, 20), i32([n]))
    check_decode(out, lse, q, [ks], [vs], [3])


@pytest.mark.parametrize("where", ["whole", "cut"])
@pytest.mark.parametrize("n_q, H, Hkv, d", [(1, 8, 2, 64), (1, 8, 2, 128), (3, 8, 2, 64), (3, 8, 2, 128),
                                            (5, 32, 8, 128), (16, 8, 1, 64)])
def test_weights_have_22_bits_and_more(n_q, H, Hkv, d, where):
    """An output is one weight p_i / l (a query row picks a column of K; three
    live keys with scores in [-1, 1]; column c of V is 1 at live key c % 3, its
    scale 2^-7 of a code 128 or 2^-8 of 256, so that terms of different scales
    meet).  As in the paged decode a weight is off by 6.4 u (the score's one
    rounding of at most 2 u of |y| <= 3, the factor on it, ex2), here 1 u more
    for the factor from q's power of two; its two fp16 terms leave at most 2 u
    of it (a half step of the second term, 2^-12 2^-11); their products meet in a
    sum that truncates twice (2 u each) and one rounding; l adds two; 1 / l and
    the product one each: 2 * 7.4 + 2 + 4 + 1 + 2 + 2 = 26 u, 32 u is used.
    Where tiles, warps and parts meet: 26 + 2 * 6 * 6.4 = 103 u, 112 u is used.
    One term, off by up to 2^-12 = 4096 u, misses either."""
    lengths = [n_q + 2, n_q + 5, n_q + 9] if where == "whole" else [3000 + n_q, 70000, 500]
    q, pages, table, lens, ks, vs = make8(lengths, [n_q] * 3, H, Hkv, d, 16, seed=d + n_q)
    r = np.random.default_rng(d + n_q)
    g = H // Hkv
    q.zero_()
    for i in range(3):
        for j in range(n_q):
            for h in range(H):
                q[i * n_q + j, h, (j * g + h % g) % d] = 1.0
    tab = table.cpu().numpy()
    for i, n in enumerate(lengths):
        live = np.sort(r.choice(n - n_q + 1, 3, replace=False)) if where == "cut" else np.arange(3)
        at = torch.from_numpy(live).to(DEV)
        k = torch.full((n, Hkv, d), -200.0 * math.sqrt(d), device=DEV)
        k[at] = torch.from_numpy(r.uniform(-1, 1, (3, Hkv, d)) * math.sqrt(d)).to(DEV).float()
        v = torch.randn(n, Hkv, d, device=DEV)
        v[at] = 0.0
        for c in range(3):
            v[at[c], :, c::3] = 1.0
        kcode, kbyte, kval = hold(k)
        vcode, vbyte, vval = hold(v)
        vcode[at[1]] = (vcode[at[1]].float() / 2).to(CODE)
        vbyte[at[1]] += 1
        ks[i], vs[i] = kval, vval
        for p in range(-(-n // 16)):
            part = slice(p * 16, min(n, p * 16 + 16))
            m = part.stop - part.start
            pages[0].view(torch.uint8)[tab[i, p], :m] = kcode[part].view(torch.uint8)
            pages[1].view(torch.uint8)[tab[i, p], :m] = vcode[part].view(torch.uint8)
            pages[2].view(torch.uint8)[tab[i, p], :, :m] = kbyte[part].t()
            pages[3].view(torch.uint8)[tab[i, p], :, :m] = vbyte[part].t()
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens)
    ra.ra_device_status()
    bar = 32 if where == "whole" else 112
    for i, n in enumerate(lengths):
        rows = slice(i * n_q, (i + 1) * n_q)
        ro, rl = oracle.attention(q[rows].cpu(), ks[i].cpu(), vs[i].cpu(), causal=True,
                                  q_pos=n - n_q + np.arange(n_q), k_pos=np.arange(n))
        err = np.abs(np64(out[rows]) - ro)
        assert (err <= bar * U * ro).all(), f"max error {(err / (U * ro)).max():.1f} u"
        assert (np.abs(np64(lse[rows]) - rl) <= (bar + 4) * U).all()


@pytest.mark.parametrize("what", ["key", "value"])
def test_nan_codes_stay_with_those_who_see_them(what):
    """A NaN key gives NaN in the rows that see it and nowhere else; a NaN value
    in every row of its request and KV head, and in no other request."""
    q, pages, table, lens, ks, vs = make8([300, 200], [2, 2], 8, 2, 128, 16)
    tab = table.cpu()
    at = 299  # the last token of request 0, seen by its second row alone
    c = pages[0 if what == "key" else 1].view(torch.uint8)
    c[tab[0, at // 16], at % 16, 1, 5] = 0x7f
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens)
    ra.ra_device_status()
    assert torch.isnan(out[1, 4:]).any(-1).all()
    if what == "key":
        assert torch.isnan(lse[1, 4:]).all()
        assert not torch.isnan(out[0]).any()
    assert not torch.isnan(out[0, :4]).any() and not torch.isnan(out[1, :4]).any()
    check_decode(out[2:], lse[2:], q[2:], ks[1:], vs[1:], [2])


# ------------------------------------------------------------------ edges

def test_empty_cache_and_lengths_past_the_row():
    q = torch.randn(3, 8, 128, device=DEV).bfloat16()
    c = torch.empty(0, 16, 2, 128, dtype=torch.uint8, device=DEV).view(CODE)
    s = torch.empty(0, 2, 16, dtype=torch.uint8, device=DEV).view(SCALE)
    out, lse = ra.ra_paged_decode_fp8(q, c, c, s, s, torch.zeros(3, 2, dtype=torch.int32, device=DEV), i32([0, 0, 0]))
    ra.ra_device_status()
    assert (out == 0).all() and torch.isneginf(lse).all()
    q, pages, table, lens, ks, vs = make8([64, 32], [1, 1], 4, 2, 64, 16)
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table[:, :2].contiguous(), i32([64, 10**9]))
    check_decode(out, lse, q, [ks[0][:32], ks[1]], [vs[0][:32], vs[1]], [1, 1])


def test_pages_out_of_range_stay_with_their_request():
    q, pages, table, lens, ks, vs = make8([300, 700, 64], [2] * 3, 8, 2, 128, 16)
    table[1, ::2] = torch.tensor([-1, 2**30, -2**31, pages[0].shape[0]], dtype=torch.int32,
                                 device=DEV).repeat(table.shape[1])[:table[1, ::2].numel()]
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens)
    ra.ra_device_status()
    check_decode(out[:2], lse[:2], q[:2], ks[:1], vs[:1], [2])
    check_decode(out[4:], lse[4:], q[4:], ks[2:], vs[2:], [2])


@pytest.mark.parametrize("H, d", [(4, 64), (4, 128)])
def test_the_longest_history(H, d):
    """2^31 - 256 keys, one page over and over; with q = 0 the output is the mean
    of the values 0 and 1 (their sums inside a CTA are exact below 2^24; up to 304
    partials and a warp's states join in fp32, a rounding each)."""
    ps, max_pages = 256, (1 << 23) - 1
    g = torch.Generator(device=DEV).manual_seed(1)
    kc = torch.zeros(1, ps, 1, d, dtype=torch.uint8, device=DEV)
    one = torch.randint(0, 2, (1, ps, 1, d), generator=g, device=DEV)
    vc = (one * 0x38).to(torch.uint8)  # 1.0
    s = torch.full((1, 1, ps), 127, dtype=torch.uint8, device=DEV).view(SCALE)
    q = torch.zeros(1, H, d, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(1, max_pages, dtype=torch.int32, device=DEV)
    out, lse = ra.ra_paged_decode_fp8(q, kc.view(CODE), vc.view(CODE), s, s, table, i32([max_pages * ps]))
    ra.ra_device_status()
    want = one[0].double().mean(0).repeat_interleave(H, 0)
    assert ((out.double() - want).abs() <= 320 * U).all()
    assert (lse.double() - math.log(max_pages * ps)).abs().max().item() <= 320 * U + 2 * U * 22


@pytest.mark.slow
def test_pages_past_32_bit_offsets():
    """A cache of more than 2^32 bytes: its last pages."""
    ps, Hkv, d = 256, 8, 128
    n_pages = (1 << 32) // (ps * Hkv * d) + 40
    c = torch.zeros(n_pages, ps, Hkv, d, dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(c)
    s = torch.full((n_pages, Hkv, ps), 127, dtype=torch.uint8, device=DEV)
    q, pages, table, lens, ks, vs = make8([5000], [1], 32, Hkv, d, ps)
    n = pages[0].shape[0]
    c[-n:], v[-n:] = pages[0].view(torch.uint8), pages[1].view(torch.uint8)
    ss = [s.clone(), s.clone()]
    ss[0][-n:], ss[1][-n:] = pages[2].view(torch.uint8), pages[3].view(torch.uint8)
    table = torch.where(table < n, table + n_pages - n, table)
    big = (c.view(CODE), v.view(CODE), ss[0].view(SCALE), ss[1].view(SCALE))
    out, lse = ra.ra_paged_decode_fp8(q, *big, table, lens)
    ra.ra_device_status()
    check_decode(out, lse, q, ks, vs, [1])
    k, vv = ra.ra_paged_read_fp8(*big, table, lens, i32([0, 5000]), tokens=5000)
    assert torch.equal(k, ks[0]) and torch.equal(vv, vs[0])
    # And the append there.
    at = torch.arange((n_pages - 1) * ps, n_pages * ps, device=DEV)
    x = torch.randn(ps, Hkv, d, device=DEV).bfloat16()
    ra.ra_paged_append_fp8(x, x, x, None, *big, at, torch.zeros(ps, dtype=torch.int32, device=DEV))
    code, byte, _ = hold(x.float())
    for cc, sc in ((c, ss[0]), (v, ss[1])):
        assert torch.equal(cc[-1].view(CODE).float(), code.float()) and torch.equal(sc[-1], byte.t())


# ------------------------------------------------------------------ streams, graphs, threads

def test_captured_and_replayed_with_longer_histories():
    lengths = [700, 64, 1, 3000]
    q, pages, table, lens, ks, vs = make8(lengths, [1] * 4, 32, 8, 128, 16)
    ra.ra_paged_decode_fp8(q, *pages, table, lens)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ra.ra_paged_decode_fp8(q, *pages, table, lens))
        graphs.append(g)
    for part in ([1, 1, 1, 1], [300, 64, 0, 129], lengths):
        lens.copy_(i32(part))
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for _ in range(3):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for out, lse in outs:
            check_decode(out, lse, q, [k[:n] for k, n in zip(ks, part)],
                         [v[:n] for v, n in zip(vs, part)], [1] * 4)
    ra.ra_device_status()


def test_two_threads_on_streams_of_their_own():
    cases = [make8([3000, 40, 900], [1] * 3, 32, 8, 128, 16, seed=1), make8([2000, 700], [6] * 2, 8, 2, 128, 16, seed=2)]
    run = lambda c: ra.ra_paged_decode_fp8(c[0], *c[1], c[2], c[3])  # noqa: E731
    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(30):
                    out, lse = run(cases[i])
                    st.synchronize()
                    if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    ra.ra_device_status()
    assert not bad


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import blockwise_online_softmax_gb300 as ra
from test_gpu_fp8_decode import check_decode, make8
q, pages, table, lens, ks, vs = make8([700, 64, 3000], [1] * 3, 32, 8, 128, 16)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out, lse = ra.ra_paged_decode_fp8(q, *pages, table, lens)
for _ in range(3):
    g.replay()
torch.cuda.synchronize()
check_decode(out, lse, q, ks, vs, [1] * 3)
ra.ra_device_status()
print("captured first")
"""


def test_first_call_of_a_process_may_be_captured():
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("name", ["append", "read", "decode"])
def test_outputs_left_out_on_another_stream(name):
    """Outputs are made on the stream of the call, whatever is current."""
    q, pages, table, lens, ks, vs = make8([900, 50], [1, 1], 8, 2, 128, 16)
    cu = i32([0, 900, 950])
    x = torch.randn(950, 2, 128, device=DEV).bfloat16()
    slots = torch.arange(950, device=DEV)
    spare = [p.clone() if p.dtype == CODE else p.view(torch.uint8).clone().view(SCALE) for p in pages]

    def run(stream):
        if name == "append":
            return (ra.ra_paged_append_fp8(x, x, x, None, *spare, slots, torch.zeros_like(slots, dtype=torch.int32),
                                           stream=stream),)
        if name == "read":
            return ra.ra_paged_read_fp8(*pages, table, lens, cu, tokens=950, stream=stream)
        return ra.ra_paged_decode_fp8(q, *pages, table, lens, stream=stream)

    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream):
        got = run(st)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_wrong_tensors_are_refused():
    q, pages, table, lens, _, _ = make8([60, 30], [1, 1], 4, 2, 64, 16)
    run = lambda p=pages, **kw: ra.ra_paged_decode_fp8(q, *p, table, lens, **kw)  # noqa: E731
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        run([pages[0].view(torch.uint8), *pages[1:]])
    with pytest.raises(TypeError, match="float8_e8m0fnu"):
        run([*pages[:3], pages[3].view(torch.uint8)])
    with pytest.raises(ValueError, match="v_scale must be"):
        run([*pages[:3], pages[3].transpose(1, 2)])
    with pytest.raises(ValueError, match="k_scale: a page must be dense"):
        run([*pages[:2], pages[2].view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(SCALE), pages[3]])
    with pytest.raises(ValueError, match="must match in pages"):
        run([pages[0], pages[1][:-1], *pages[2:]])
    with pytest.raises(ra.RaError, match="page_size=8"):
        c = torch.zeros(3, 8, 2, 64, dtype=torch.uint8, device=DEV).view(CODE)
        s = torch.zeros(3, 2, 8, dtype=torch.uint8, device=DEV).view(SCALE)
        run([c, c, s, s])
    with pytest.raises(ra.RaError, match="window"):
        run(window=-1)
    with pytest.raises(ValueError, match="cpu|CUDA"):
        run([pages[0].cpu(), *pages[1:]])


# ------------------------------------------------------------------ a run of them

def test_a_prompt_in_chunks_and_tokens_one_by_one():
    """Extend, append, attend, as a server uses them.  A prompt comes in three
    chunks: each is appended, the history read back and the chunk's rows
    attend to it by ra_decode_forward; then tokens one by one over the pages.
    The reference holds k and v in 8 bits as the append does and attends in 64
    bits.  The chunks' attention rounds P to bf16 (bar 1e-2)."""
    H, Hkv, d, ps = 8, 2, 128, 16
    g = torch.Generator(device=DEV).manual_seed(12)
    total, chunks = 700, [(0, 300), (300, 555), (555, 697), (697, 698), (698, 699), (699, 700)]
    q, k, v = (torch.randn(total, h, d, device=DEV, generator=g).bfloat16() for h in (H, Hkv, Hkv))
    ph = ra.rope_phases(ra.rope_freqs(d)[0]).to(DEV)
    n_pages = 60
    kc, vc = (torch.full((n_pages, ps, Hkv, d), 0xff, dtype=torch.uint8, device=DEV).view(CODE) for _ in range(2))
    sk, sv = (torch.full((n_pages, Hkv, ps), 0xff, dtype=torch.uint8, device=DEV).view(SCALE) for _ in range(2))
    pages = (kc, vc, sk, sv)
    table = torch.full((1, 50), -1, dtype=torch.int32, device=DEV)
    free, lens, count = torch.randperm(n_pages).int().to(DEV), i32([0]), i32([n_pages])
    outs, rows = [], []
    for lo, hi in chunks:
        slots, pos, cu, _, _, status = ra.ra_paged_extend(
            lens, i32([hi - lo]), table, free, count, page_size=ps, tokens=hi - lo, lengths_out=lens,
            free_count_out=count)
        assert status.tolist() == [0, 0, 0]
        qr = ra.ra_paged_append_fp8(q[lo:hi], k[lo:hi], v[lo:hi], ph, *pages, slots, pos)
        rows.append(qr)
        if hi - lo > 1:
            kd, vd = ra.ra_paged_read_fp8(*pages, table, lens, i32([0, hi]), tokens=hi)
            outs.append(ra.ra_decode_forward(qr, kd, vd, P=4)[0])
        else:
            outs.append(ra.ra_paged_decode_fp8(qr, *pages, table, lens)[0])
    ra.ra_device_status()
    kd, vd = ra.ra_paged_read_fp8(*pages, table, lens, i32([0, total]), tokens=total)
    assert torch.equal(vd, hold(v.float())[2])
    qr, kr = ra.ra_qk_norm_rope(q, k, ph)
    assert torch.equal(torch.cat(rows), qr)
    # k: within half a code step (2^-4, or 2^-10 scales of at most max|k| / 224) of
    # the bf16 rows (2^-8 more).
    top = kr.float().abs().amax(-1, keepdim=True)
    assert ((kd.float() - kr.float()).abs() <= (2.0 ** -4 + 2.0 ** -7) * kr.float().abs() + 2.0 ** -10 * top / 224 * 1.01).all()
    ref, _ = oracle.attention(qr.cpu(), kd.cpu(), vd.cpu(), causal=True)
    err = np.abs(np64(torch.cat(outs)) - ref)
    assert err[:697].max() <= 1e-2 and err[697:].max() <= 1e-4


@pytest.mark.parametrize("d, Hkv", [(64, 4), (128, 2)])
def test_more_rows_than_expected_and_windows_past_the_history(d, Hkv):
    rows = [1, 30, 2, 0, 1]
    q, pages, table, lens, ks, vs = make8([700, 90, 3, 40, 1], rows, 4 * Hkv, Hkv, d, 16, extra=3)
    cu = i32(np.concatenate([[0], np.cumsum(rows)]))
    for window in (0, 700, 2**31 - 1, 2**31, 2**62):
        out = torch.full(q.shape, 9.0, device=DEV)
        lse = torch.full(q.shape[:2], 9.0, device=DEV)
        ra.ra_paged_decode_fp8(q, *pages, table, lens, cu_q=cu, n_q=1, window=window, out=out, lse=lse)
        ra.ra_device_status()
        check_decode(out, lse, q, ks, vs, rows)
        assert (out[-3:] == 9.0).all() and (lse[-3:] == 9.0).all()
