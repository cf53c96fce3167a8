"""Page bookkeeping, the append and the paged decode on the GPU.

Bookkeeping is exact.  Decode is compared with the fp64 oracle over each
request's own keys.  Tolerance, with u = 2^-23 (a truncating fp32 step) and
A = max |q| |k| / sqrt(d), which bounds a score's absolute terms: a score is
off by d u A, so every weight by that relative amount; a weight's value for
the product with V by 2^-16 at most; the sums over n keys by n u.  The
output is a weighted mean of V: |dO| <= (2 d u A + 2^-16 + n u) max|V|, a
bf16 output half a step (2^-8) more.  The LSE: d u A + n u + 4 u |LSE|.
"""
import math

import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import oracle
import serve_ref
from blockwise_online_softmax_gb300 import binding
from test_gpu_rope import check_rope

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    from blockwise_online_softmax_gb300 import build

    build.build()
    binding.lib()
    yield
    torch.cuda.empty_cache()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def pool(lengths, page_size, width, n_pages, seed=0):
    """A random deal of pages: table (-1 behind each row's pages), stack, count."""
    ids = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    table = np.full((len(lengths), width), -1, dtype=np.int32)
    used = 0
    for i, n in enumerate(lengths):
        c = -(-n // page_size)
        table[i, :c] = ids[used:used + c]
        used += c
    free = np.full(n_pages, -7, dtype=np.int32)
    free[:n_pages - used] = ids[used:]
    return table, free, n_pages - used


# ------------------------------------------------------------------ bookkeeping

def run_extend(ln, nw, table, free, count, ps, tokens, in_place=False):
    a = dict(lengths=i32(ln), new_tokens=i32(nw), block_table=i32(table).view(table.shape),
             free_pages=i32(free), free_count=i32([count]))
    kw = dict(lengths_out=a["lengths"], free_count_out=a["free_count"]) if in_place else {}
    slots, pos, cu, ln2, count2, status = ra.ra_paged_extend(
        *a.values(), page_size=ps, tokens=tokens, **kw)
    assert torch.equal(a["free_pages"].cpu(), torch.from_numpy(free))
    return [x.cpu().numpy() for x in (slots, pos, cu, ln2, count2, status, a["block_table"])]


def check_extend(ln, nw, width, ps, tokens, n_pages, in_place=False, seed=0):
    table, free, count = pool(np.maximum(ln, 0), ps, width, n_pages, seed)
    got = run_extend(ln, nw, table, free, count, ps, tokens, in_place)
    want = serve_ref.extend(ln, nw, table, free, count, ps, tokens)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.reshape(-1), np.asarray(w).reshape(-1))
    return got


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n, ps, top, new, pad", [
    (1, 8, 0, 1, 0), (1, 16, 5, 40, 3), (3, 16, 33, 1, 5), (256, 16, 500, 1, 8),
    (1023, 32, 100, 3, 0), (1024, 8, 60, 2, 1), (1025, 8, 60, 2, 1), (5000, 64, 90, 2, 100),
    (40, 64, 200, 700, 50), (9, 256, 1000, 5000, 7), (2, 128, 20000, 30000, 0),
])
def test_extend(n, ps, top, new, pad, in_place):
    r = np.random.default_rng(n + ps)
    ln, nw = r.integers(0, top + 1, n), r.integers(0, new + 1, n)
    ln[::3] = ln[::3] // ps * ps  # full last pages
    width = -(-(top + new) // ps)
    pages = int((-(-(ln + nw) // ps)).sum())
    got = check_extend(ln, nw, width, ps, int(nw.sum()) + pad, pages + 2, in_place, seed=n)
    assert got[5].tolist() == [0, 0, 0]


def test_extend_takes_the_last_page_and_no_more():
    assert check_extend([16, 3], [1, 13], 4, 16, 14, 3)[5].tolist() == [0, 0, 0]
    assert check_extend([16, 3], [1, 14], 4, 16, 15, 3)[5].tolist() == [1, 0, 0]


def test_extend_refuses_a_step_as_a_whole():
    assert check_extend([10, 60], [5, 10], 4, 16, 20, 9)[5].tolist() == [0, 1, 0]
    assert check_extend([10, 20], [5, 10], 4, 16, 14, 9)[5].tolist() == [0, 0, 1]
    assert check_extend([0, 0], [2**31 - 1, 2**31 - 1], 2, 16, 8, 9)[5].tolist() == \
        [2**28 - 9, 2, 2**31 - 1]


def test_extend_counts_negative_values_as_zero():
    check_extend([-4, 7, 0], [3, -2, 0], 4, 8, 6, 9)


def test_extend_without_requests_or_tokens():
    got = run_extend([], [], np.zeros((0, 4), np.int32), np.zeros(3, np.int32), 3, 16, 4)
    assert got[0].tolist() == [-1] * 4 and got[2].tolist() == [0] and got[4].tolist() == [3]
    check_extend([5, 6], [0, 0], 4, 16, 0, 4)


@pytest.mark.parametrize("n, ps, top, share", [(1, 16, 100, 1.0), (64, 16, 500, 0.3),
                                               (1025, 8, 60, 0.5), (2048, 32, 3000, 0.5),
                                               (7, 256, 0, 1.0)])
def test_release(n, ps, top, share):
    r = np.random.default_rng(n)
    ln, fin = r.integers(0, top + 1, n), (r.random(n) < share).astype(np.int32) * 3
    table, free, count = pool(ln, ps, max(1, -(-top // ps)), int((-(-ln // ps)).sum()) + 3, n)
    want = serve_ref.release(ln, fin, table, free, count, ps)
    lens, cnt, stack = i32(ln), i32([count]), i32(free)
    out = ra.ra_paged_release(lens, i32(fin), i32(table), stack, cnt, page_size=ps)
    for g, w in zip((stack, *out), want):
        np.testing.assert_array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    stack = i32(free)  # the arrays themselves
    ra.ra_paged_release(lens, i32(fin), i32(table), stack, cnt, page_size=ps, lengths_out=lens,
                        free_count_out=cnt)
    assert torch.equal(lens, out[0]) and torch.equal(cnt, out[1])


def test_release_stays_inside_the_stack():
    """Lengths that claim more pages than the stack or the row can hold."""
    stack = torch.full((8,), -7, dtype=torch.int32, device=DEV)
    lens, cnt = ra.ra_paged_release(i32([10**9, 40]), i32([1, 1]), i32([[1, 2, 3], [4, 5, 6]]),
                                    stack[:4], i32([1]), page_size=16)
    assert stack.tolist() == [-7, 1, 2, 3, -7, -7, -7, -7]
    assert lens.tolist() == [0, 0] and cnt.tolist() == [4]


def test_extend_then_release_returns_every_page():
    r = np.random.default_rng(2)
    n, ps, n_pages = 50, 16, 400
    table = torch.full((n, 20), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(n_pages).int().to(DEV)
    lens, count = i32(np.zeros(n)), i32([n_pages])
    state = dict(page_size=ps, lengths_out=lens, free_count_out=count)
    for step in range(30):
        nw = i32(r.integers(0, 12, n))
        _, _, _, _, _, status = ra.ra_paged_extend(lens, nw, table, free, count,
                                                   tokens=600, **state)
        held = [table[i, :-(-int(x) // ps)].tolist() for i, x in enumerate(lens)]
        live = sum(held, []) + free[:int(count)].tolist()
        assert sorted(live) == list(range(n_pages))  # each page once
        ra.ra_paged_release(lens, i32(r.random(n) < 0.2), table, free, count, **state)
    ra.ra_paged_release(lens, i32(np.ones(n)), table, free, count, **state)
    assert sorted(free.tolist()) == list(range(n_pages)) and int(count) == n_pages


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("T, H, Hkv, d, ps, rot, inter, norm", [
    (1, 1, 1, 64, 8, 64, False, True), (5, 32, 8, 128, 16, 128, False, True),
    (300, 12, 4, 64, 64, 32, True, False), (77, 8, 1, 128, 256, 96, True, True),
    (40, 3, 3, 128, 32, 0, False, True), (2700, 32, 8, 128, 16, 128, False, True),
])
@pytest.mark.parametrize("together", [False, True])
def test_append(T, H, Hkv, d, ps, rot, inter, norm, together):
    g = torch.Generator().manual_seed(T)
    n_pages = -(-2 * T // ps) + 1
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g).bfloat16().to(DEV)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    if together:  # K and V of a page side by side: strided pages
        kv = torch.full((n_pages, 2, ps, Hkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
        kc, vc = kv[:, 0], kv[:, 1]
    else:
        kc, vc = (torch.full((n_pages, ps, Hkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
                  for _ in range(2))
    slots = torch.randperm(n_pages * ps, generator=g)[:T]
    slots[T // 2::5] = -1
    if T > 6:
        slots[3] = n_pages * ps  # past the pages: padding too
    pos = torch.randint(0, 200000, (T,), generator=g).int()
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) if norm else None for _ in range(2)]
    f = ra.rope_freqs(rot)[0].numpy() if rot else np.zeros(0)
    ph = ra.rope_phases(torch.from_numpy(f)).to(DEV) if rot else None
    qo = torch.full((T, H, d), 5.0, dtype=torch.bfloat16, device=DEV)
    ra.ra_paged_append(q, k, v, ph, kc, vc, slots.to(DEV), pos.to(DEV), q_weight=w[0],
                       k_weight=w[1], interleaved=inter, q_out=qo)
    real = ((slots >= 0) & (slots < n_pages * ps)).numpy()
    sl = slots.numpy()[real]
    rows = torch.from_numpy(np.flatnonzero(real)).to(DEV)
    k_all, v_all = kc.reshape(-1, Hkv, d), vc.reshape(-1, Hkv, d)
    at = torch.from_numpy(sl).to(DEV)
    assert torch.equal(v_all[at], v[rows])
    p = pos.numpy()[real]
    check_rope(k_all[at], k[rows], w[1], p, f, interleaved=inter)
    check_rope(qo[rows], q[rows], w[0], p, f, interleaved=inter)
    rest = torch.ones(n_pages * ps, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert (k_all[rest] == 3.0).all() and (v_all[rest] == 3.0).all()
    pad = torch.ones(T, dtype=torch.bool, device=DEV)
    pad[rows] = False
    assert (qo[pad] == 5.0).all()


# ------------------------------------------------------------------ decode

def make_decode(lengths, rows, H, Hkv, d, ps, *, seed=0, scale=1.5, together=False, extra=0):
    """Random pages with NaN behind every request's last token and in the
    pages of nobody; q rows packed, `extra` rows behind the last."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    width = max(1, max(-(-n // ps) for n in lengths)) + 1
    n_pages = sum(-(-n // ps) for n in lengths) + 3
    table, _, _ = pool(lengths, ps, width, n_pages, seed)
    kv = torch.full((n_pages, 2, ps, Hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    kc, vc = (kv[:, 0], kv[:, 1]) if together else (kv[:, 0].contiguous(), kv[:, 1].contiguous())
    ks, vs = [], []
    for i, n in enumerate(lengths):
        k, v = (torch.randn(n, Hkv, d, generator=g, device=DEV).bfloat16() for _ in range(2))
        ks.append(k)
        vs.append(v)
        for c in range(-(-n // ps)):
            part = slice(c * ps, min(n, c * ps + ps))
            kc[table[i, c], :part.stop - part.start] = k[part]
            vc[table[i, c], :part.stop - part.start] = v[part]
    table[table < 0] = 2**30  # never read
    q = (torch.randn(sum(rows) + extra, H, d, generator=g, device=DEV) * scale).bfloat16()
    return q, kc, vc, i32(table), i32(lengths), ks, vs


def check_decode(out, lse, q, ks, vs, rows, window=0):
    r0 = 0
    for k, v, n in zip(ks, vs, rows):
        if n == 0:
            continue
        L, (_, Hkv, d) = k.shape[0], k.shape
        o, l = (np.asarray(x[r0:r0 + n].cpu().double()) for x in (out, lse))
        qi = q[r0:r0 + n]
        r0 += n
        if L == 0:
            assert (o == 0).all() and np.isneginf(l).all()
            continue
        ro, rl = oracle.attention(qi.cpu(), k.cpu(), v.cpu(), causal=True, window=window,
                                  q_pos=L - n + np.arange(n), k_pos=np.arange(L))
        A = float(qi.float().norm(dim=-1).max() * k.float().norm(dim=-1).max()) / math.sqrt(d)
        vmax = float(v.abs().max())
        bar = (2 * d * U * A + 2.0 ** -16 + L * U) * vmax
        step = 2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0
        assert (np.abs(o - ro) <= bar + step * np.abs(ro)).all(), \
            f"max |dO| = {np.abs(o - ro).max():.2e}, bar {bar:.2e}"
        fin = np.isfinite(rl)
        assert (np.isneginf(l) == ~fin).all()
        assert (np.abs(l[fin] - rl[fin]) <= d * U * A + L * U + 4 * U * np.abs(rl[fin])).all()


DECODE = [
    # lengths, rows per request, heads, kv_heads, d, page size, window
    ([1], 1, 1, 1, 64, 8, 0),
    ([1, 0, 2], 1, 8, 2, 128, 16, 0),
    ([127, 128, 129, 0, 5], 1, 32, 8, 128, 16, 0),
    ([1000], 1, 32, 8, 128, 64, 0),
    ([5000, 3, 70], 1, 4, 4, 128, 256, 0),
    ([700, 255, 256, 257], 1, 12, 4, 64, 128, 0),
    ([4097, 600], 1, 8, 1, 64, 32, 100),
    ([333, 64, 2000], 2, 64, 8, 128, 16, 0),      # 16 rows per KV head
    ([333, 64, 2000], 3, 12, 4, 128, 8, 37),
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


@pytest.mark.parametrize("together", [False, True])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{str(c[0][:4])}-q{c[1]}-h{c[2]}/{c[3]}"
                         f"-d{c[4]}-p{c[5]}-w{c[6]}")
def test_decode(case, together):
    lengths, n_q, H, Hkv, d, ps, window = case
    rows = [n_q] * len(lengths)
    q, kc, vc, table, lens, ks, vs = make_decode(lengths, rows, H, Hkv, d, ps, together=together)
    out, lse = ra.ra_paged_decode(q, kc, vc, table, lens, window=window)
    ra.ra_device_status()
    check_decode(out, lse, q, ks, vs, rows, window)
    again = ra.ra_paged_decode(q, kc, vc, table, lens, window=window)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_decode_bf16_output():
    rows = [2, 2]
    q, kc, vc, table, lens, ks, vs = make_decode([300, 20], rows, 16, 4, 128, 16)
    out = torch.empty(4, 16, 128, dtype=torch.bfloat16, device=DEV)
    _, lse = ra.ra_paged_decode(q, kc, vc, table, lens, out=out)
    check_decode(out, lse, q, ks, vs, rows)


@pytest.mark.parametrize("rows", [[1, 0, 3, 1], [0, 0, 2, 0], [40, 1, 0, 7], [300, 2, 1, 1]])
def test_decode_ragged_rows(rows):
    """cu_q: idle requests, several rows, and rows behind the last request
    left as they were."""
    lengths = [500, 77, 300, 1025]
    q, kc, vc, table, lens, ks, vs = make_decode(lengths, rows, 8, 2, 128, 16, extra=5)
    out = torch.full(q.shape, 9.0, device=DEV)
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    cu = i32(np.concatenate([[0], np.cumsum(rows)]))
    ra.ra_paged_decode(q, kc, vc, table, lens, cu_q=cu, out=out, lse=lse)
    check_decode(out, lse, q, ks, vs, rows)
    assert (out[-5:] == 9.0).all() and (lse[-5:] == 9.0).all()


def test_decode_large_scores_and_equal_scores():
    q, kc, vc, table, lens, ks, vs = make_decode([2000, 60], [1, 1], 8, 2, 128, 16, scale=40.0)
    check_decode(*ra.ra_paged_decode(q, kc, vc, table, lens), q, ks, vs, [1, 1])
    q.zero_()
    check_decode(*ra.ra_paged_decode(q, kc, vc, table, lens), q, ks, vs, [1, 1])


def test_decode_lengths_past_the_row_count_as_the_row():
    q, kc, vc, table, lens, ks, vs = make_decode([64, 32], [1, 1], 4, 2, 64, 16)
    table = table[:, :2].contiguous()
    out, lse = ra.ra_paged_decode(q, kc, vc, table, i32([64, 10**9]))
    check_decode(out, lse, q, [ks[0][:32], ks[1]], [vs[0][:32], vs[1]], [1, 1])


def test_decode_captured_and_replayed_with_longer_histories():
    """Two graphs captured once, replayed on two streams as lengths grow: no
    host value is baked in, and they share no workspace."""
    lengths = [700, 64, 1, 3000]
    q, kc, vc, table, lens, ks, vs = make_decode(lengths, [1] * 4, 32, 8, 128, 16)
    ra.ra_paged_decode(q, kc, vc, table, lens)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ra.ra_paged_decode(q, kc, vc, table, lens))
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 200])
def test_decode_many_rows_over_items_of_every_length(d, window):
    """More rows than a 16-row tile holds, items of 0 to 5 key tiles whole and
    cut between CTAs, idle requests among them: the two softmax groups meet in
    every order."""
    rng = np.random.default_rng(d + window)
    lengths = [int(x) for x in rng.choice([0, 1, 60, 128, 129, 250, 256, 300, 520, 640], 170)]
    rows = [int(x) for x in rng.choice([0, 9, 12, 40], 170, p=[0.1, 0.4, 0.4, 0.1])]
    q, kc, vc, table, lens, ks, vs = make_decode(lengths, rows, 8, 2, d, 32, extra=3)
    cu = i32(np.concatenate([[0], np.cumsum(rows)]))
    out, lse = torch.full(q.shape, 9.0, device=DEV), torch.full(q.shape[:2], 9.0, device=DEV)
    ra.ra_paged_decode(q, kc, vc, table, lens, cu_q=cu, window=window, out=out, lse=lse)
    ra.ra_device_status()
    check_decode(out, lse, q, ks, vs, rows, window)
    assert (out[-3:] == 9.0).all() and (lse[-3:] == 9.0).all()
    for _ in range(5):
        o2, l2 = ra.ra_paged_decode(q, kc, vc, table, lens, cu_q=cu, window=window)
        assert torch.equal(o2[:-3], out[:-3]) and torch.equal(l2[:-3], lse[:-3])


def test_decode_of_an_empty_cache():
    q = torch.randn(3, 8, 128, device=DEV).bfloat16()
    kc = torch.empty(0, 16, 2, 128, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    out, lse = ra.ra_paged_decode(q, kc, torch.empty_like(kc), table, i32([0, 0, 0]))
    ra.ra_device_status()
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_decode_two_eager_calls_at_once():
    """Two streams, calls in turn, no synchronisation between them."""
    cases = [make_decode([3000, 40, 900], [1] * 3, 32, 8, 128, 16, seed=1),
             make_decode([2000, 700], [16] * 2, 8, 2, 128, 16, seed=2)]
    want = [ra.ra_paged_decode(*c[:5]) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(20):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(ra.ra_paged_decode(*c[:5]))
    torch.cuda.synchronize()
    ra.ra_device_status()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_decode_equals_the_contiguous_decode():
    """One request's pages against ra_decode_forward on the same history."""
    q, kc, vc, table, lens, ks, vs = make_decode([5000], [3], 32, 8, 128, 64)
    out, lse = ra.ra_paged_decode(q, kc, vc, table, lens)
    ref, ref_lse = ra.ra_decode_forward(q, ks[0], vs[0], P=4)
    ra.ra_device_status()
    assert (out - ref).abs().max().item() <= 1e-2 and (lse - ref_lse).abs().max().item() <= 1e-2


@pytest.mark.slow
def test_decode_pages_past_32_bit_offsets():
    """A cache whose elements and bytes pass 2^32: the last pages of it."""
    ps, Hkv, d = 256, 8, 128
    n_pages = (1 << 32) // (ps * Hkv * d) + 40
    kc = torch.empty(n_pages, ps, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    g = torch.Generator(device=DEV).manual_seed(1)
    ids = torch.arange(n_pages - 5, n_pages).flip(0)
    k, v = (torch.randn(1100, Hkv, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    for c, p in enumerate(ids.tolist()):
        n = min(1100, c * ps + ps) - c * ps
        kc[p, :n], vc[p, :n] = k[c * ps:c * ps + n], v[c * ps:c * ps + n]
    q = torch.randn(1, 32, d, generator=g, device=DEV).bfloat16()
    out, lse = ra.ra_paged_decode(q, kc, vc, i32(ids.view(1, 5)), i32([1100]))
    ra.ra_device_status()
    check_decode(out, lse, q, [k], [v], [1])


# ------------------------------------------------------------------ a serving loop

@pytest.mark.parametrize("norm", [True, False])
def test_serving_steps_equal_the_ring_over_the_whole_sequences(norm):
    """Requests arrive, grow by uneven steps and finish, all bookkeeping on
    the device; every token's output equals the causal attention of its whole
    sequence, as the ring computes it on the rotated q, k, v."""
    H, Hkv, d, ps, n_req, n_pages = 8, 2, 128, 16, 5, 64
    g = torch.Generator().manual_seed(4)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) if norm else None for _ in range(2)]
    f, ms = ra.rope_freqs(128, scaling="yarn", factor=4.0)
    ph = ra.rope_phases(f).to(DEV)
    how = dict(q_weight=w[0], k_weight=w[1], mscale=ms)
    total = [130, 40, 77, 201, 16]
    qkv = [torch.randn(n, H + 2 * Hkv, d, generator=g).bfloat16().to(DEV) for n in total]
    refs = []
    for x in qkv:
        q, k = ra.ra_qk_norm_rope(x[:, :H], x[:, H:H + Hkv], ph, **how)
        refs.append(ra.ra_ring_forward(q, k, x[:, H + Hkv:].contiguous(), P=1, causal=True))
    cache = torch.full((n_pages, 2, ps, Hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((n_req, 16), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(n_pages, generator=g).int().to(DEV)
    lens, count = i32([0] * n_req), i32([n_pages])
    state = dict(page_size=ps, lengths_out=lens, free_count_out=count)
    done = [0] * n_req
    r = np.random.default_rng(0)
    while any(a < b for a, b in zip(done, total)):
        first = all(x == 0 for x in done)
        nw = [min(t - a, int(r.integers(20, 60)) if first else int(r.integers(0, 4)))
              for a, t in zip(done, total)]
        rows = 256
        slots, pos, cu, _, _, status = ra.ra_paged_extend(lens, i32(nw), table, free, count,
                                                          tokens=rows, **state)
        step = torch.zeros(rows, H + 2 * Hkv, d, dtype=torch.bfloat16, device=DEV)
        if sum(nw):
            step[:sum(nw)] = torch.cat([x[a:a + n] for x, a, n in zip(qkv, done, nw)])
        q = ra.ra_paged_append(step[:, :H], step[:, H:H + Hkv], step[:, H + Hkv:], ph,
                               cache[:, 0], cache[:, 1], slots, pos, **how)
        out, lse = ra.ra_paged_decode(q, cache[:, 0], cache[:, 1], table, lens, cu_q=cu)
        assert status.tolist() == [0, 0, 0]
        at = 0
        for i, n in enumerate(nw):
            ro, rl = (x[done[i]:done[i] + n] for x in refs[i])
            # the ring rounds P to bf16: the stated 1e-2 and 1e-3 bars
            assert n == 0 or (out[at:at + n] - ro).abs().max().item() <= 1e-2
            assert n == 0 or ((lse[at:at + n] - rl).abs()
                              / rl.abs().clamp(min=1.0)).max().item() <= 1e-3
            at, done[i] = at + n, done[i] + n
        fin = [int(a == t) for a, t in zip(done, total)]
        if any(fin):
            keep = lens.clone()
            before = int(count)
            ra.ra_paged_release(lens, i32(fin), table, free, count, **state)
            assert int(count) == before + sum(-(-int(x) // ps) for x, y in zip(keep, fin) if y)
    ra.ra_device_status()
    assert sorted(free.tolist()) == list(range(n_pages))


def test_refusals_reach_python_with_the_library_s_message():
    """A status of the C ABI raises RaError with the message of the same
    thread; shapes, types and placement raise before the call."""
    q, kc, vc, table, lens, _, _ = make_decode([64, 32], [1, 1], 4, 2, 64, 16)
    with pytest.raises(binding.RaError, match="page_size=12"):
        ra.ra_paged_extend(lens, lens, table, lens, lens[:1], page_size=12, tokens=4)
    with pytest.raises(binding.RaError, match="window"):
        ra.ra_paged_decode(q, kc, vc, table, lens, window=-1)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_paged_decode(q, kc, vc, table, lens.cpu())
    with pytest.raises(TypeError, match="int32"):
        ra.ra_paged_decode(q, kc, vc, table, lens.long())
    with pytest.raises(TypeError, match="bfloat16"):
        ra.ra_paged_decode(q.float(), kc, vc, table, lens)
    with pytest.raises(ValueError, match="dense"):
        ra.ra_paged_decode(q, kc.transpose(1, 2).contiguous().transpose(1, 2), vc, table, lens)
    with pytest.raises(ValueError, match="match in pages"):
        ra.ra_paged_decode(q, kc, vc[:1], table, lens)
    with pytest.raises(ValueError, match="block_table"):
        ra.ra_paged_decode(q, kc, vc, table[:1], lens)
    with pytest.raises(TypeError, match="tensor"):
        ra.ra_paged_decode(q, kc, vc, table, [64, 32])
    out = ra.ra_paged_decode(q, kc, vc, table, lens, stream=torch.cuda.current_stream())
    assert torch.equal(out[0], ra.ra_paged_decode(q, kc, vc, table, lens)[0])
