"""Attention with shared prefixes on the GPU, against the fp64 oracle over each
request's prefix and own keys together.  Tolerances: test_gpu_paged.py, with n
the prefix's and the own keys, and for the join of two partial sums of a row 16 u
more (a factor ex2 good to 6.4 u on either side, two roundings)."""
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
from test_gpu_paged import check_decode, i32, make_decode
from test_gpu_rope import np64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24


def make(groups, rows, H, Hkv, d, ps, *, seed=0, scale=1.5, together=False, extra=0, room=False):
    """groups: (prefix length, own lengths of its requests) each; rows: new
    tokens of every request.  Pages of prefixes and requests are dealt from one
    cache, with NaN where nobody's tokens are.  room: a prefix table for 2^18 keys
    and more, with which groups of more than 16 rows get a launch of their own."""
    plens = [p for p, _ in groups]
    own = [n for _, ls in groups for n in ls]
    q, kc, vc, table, _, ks, vs = make_decode(plens + own, rows, H, Hkv, d, ps, seed=seed, scale=scale,
                                              together=together, extra=extra)
    G = len(groups)
    cu_req = i32(np.concatenate([[0], np.cumsum([len(ls) for _, ls in groups])]))
    ptab = torch.nn.functional.pad(table[:G], (0, 2**18 // ps + 1 if room else 0), value=2**30).contiguous()
    args = (q, kc, vc, ptab, i32(plens), cu_req, table[G:].contiguous(), i32(own))
    of = [g for g, (_, ls) in enumerate(groups) for _ in ls]
    k = [torch.cat((ks[g], x)) for g, x in zip(of, ks[G:])]
    v = [torch.cat((vs[g], x)) for g, x in zip(of, vs[G:])]
    return args, k, v


CASES = [
    # groups, new tokens each, heads, kv_heads, d, page size
    ([(1, [1])], 1, 1, 1, 64, 8),
    ([(17, [1, 5])], 1, 4, 2, 128, 16),
    ([(100, [3, 30, 1])], 1, 8, 2, 64, 16),
    ([(1001, [300, 1, 20, 77, 64, 65, 2, 150])], 1, 32, 8, 128, 16),
    ([(128, [128]), (129, [127, 129])], 1, 32, 8, 128, 64),
    ([(0, [40, 2]), (500, [9]), (0, [1])], 1, 12, 4, 64, 32),
    ([(5000, [1] * 40)], 1, 8, 2, 128, 128),            # 160 rows of a KV head: two tiles of 128
    ([(3000, [10] * 100), (2, [700] * 3)], 1, 8, 1, 64, 256),
    ([(777, [33] * 9), (64, [4, 5])], 4, 32, 8, 128, 16),
    ([(777, [40] * 9), (64, [40, 50])], 9, 32, 8, 64, 16),   # own rows on the 128-row tiles too
    ([(20000, [300, 3])], 2, 16, 16, 128, 64),           # few rows, a long prefix: many CTAs an item
    ([(9, [2] * 300)], 1, 64, 8, 128, 16),
    ([(300, [6] * 3), (1, []), (40, [8])], 3, 128, 1, 128, 16),
    ([(int(p), [int(x) for x in np.random.default_rng(p).integers(1, 200, p % 7 + 1)])
      for p in range(0, 400, 13)], 1, 8, 2, 64, 16),     # 31 groups
    ([(int(p), [int(p) % 50 + 1]) for p in range(1, 100)], 1, 4, 4, 128, 16),
]


@pytest.mark.parametrize("together, room", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{[(p, len(x)) for p, x in c[0][:3]]}-q{c[1]}-h{c[2]}/{c[3]}-d{c[4]}-p{c[5]}")
def test_prefix(case, together, room):
    groups, n_q, H, Hkv, d, ps = case
    rows = [n_q] * sum(len(x) for _, x in groups)
    args, k, v = make(groups, rows, H, Hkv, d, ps, together=together, room=room)
    out, lse = ra.ra_paged_decode_prefix(*args)
    ra.ra_device_status()
    check_decode(out, lse, args[0], k, v, rows)
    again = ra.ra_paged_decode_prefix(*args)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    bf = torch.empty(args[0].shape, dtype=torch.bfloat16, device=DEV)
    _, lse2 = ra.ra_paged_decode_prefix(*args, out=bf)
    check_decode(bf, lse2, args[0], k, v, rows)


def attend(q, k, v, n_own, n_new):
    """Oracle: rows at the last n_new positions; all see what is before the own."""
    L = k.shape[0]
    return oracle.attention(q.cpu(), k.cpu(), v.cpu(), causal=True, q_pos=L - n_new + np.arange(n_new),
                            k_pos=np.arange(L))


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("rows", [[1, 0, 3, 1, 2], [0, 0, 2, 0, 0], [40, 1, 0, 7, 1]])
def test_ragged_rows(rows, room):
    """cu_q: idle requests, several rows, and rows behind the last left as they were."""
    groups = [(300, [50, 20]), (129, [77, 10, 41])]
    args, k, v = make(groups, rows, 8, 2, 128, 16, extra=5, room=room)
    out = torch.full(args[0].shape, 9.0, device=DEV)
    lse = torch.full(args[0].shape[:2], 9.0, device=DEV)
    cu = i32(np.concatenate([[0], np.cumsum(rows)]))
    for n_q in (0, 1, 9):
        out.fill_(9.0)
        lse.fill_(9.0)
        ra.ra_paged_decode_prefix(*args, cu_q=cu, n_q=n_q, out=out, lse=lse)
        ra.ra_device_status()
        check_decode(out, lse, args[0], k, v, rows)
        assert (out[-5:] == 9.0).all() and (lse[-5:] == 9.0).all()


def test_requests_of_no_group_see_their_own_keys():
    groups = [(300, [50, 20]), (129, [77, 10, 41])]
    rows = [2] * 5
    args, k, v = make(groups, rows, 8, 2, 128, 16)
    own = ra.ra_paged_decode(args[0], args[1], args[2], args[6], args[7])
    for cu in ([1, 2, 4], [0, 0, 3], [2, 2, 2], [5, 5, 5]):
        a = list(args)
        a[5] = i32(cu)
        out, lse = ra.ra_paged_decode_prefix(*a)
        ra.ra_device_status()
        for i in range(5):
            g = next((j for j in range(2) if cu[j] <= i < cu[j + 1]), None)
            r = slice(2 * i, 2 * i + 2)
            if g is None:
                check_decode(out[r], lse[r], args[0][r], [k[i][-int(args[7][i]):]], [v[i][-int(args[7][i]):]], [2])
            else:
                first = k[0 if g == 0 else 2][:groups[g][0]], v[0 if g == 0 else 2][:groups[g][0]]
                n = int(args[7][i])
                check_decode(out[r], lse[r], args[0][r], [torch.cat((first[0], k[i][-n:]))],
                             [torch.cat((first[1], v[i][-n:]))], [2])
    # No groups at all.
    none = torch.empty(0, 4, dtype=torch.int32, device=DEV)
    out, lse = ra.ra_paged_decode_prefix(*args[:3], none, i32([]), i32([0]), *args[6:])
    ra.ra_device_status()
    assert float((out - own[0]).abs().max()) <= 1e-5 and float((lse - own[1]).abs().max()) <= 1e-5


def test_rows_before_the_own_keys_and_nothing_at_all():
    """Fewer own keys than rows: the earlier rows see the prefix alone; without
    prefix and own keys a row is 0 with an LSE of -inf."""
    args, k, v = make([(50, [2, 0]), (0, [1, 0])], [3] * 4, 8, 2, 64, 16)
    out, lse = ra.ra_paged_decode_prefix(*args)
    ra.ra_device_status()
    pre = k[0][:50], v[0][:50]

    def check(row, kk, vv):
        check_decode(out[row:row + 1], lse[row:row + 1], args[0][row:row + 1], [kk], [vv], [1])

    check(0, *pre)                      # rows at own positions -1, 0, 1
    check(1, k[0][:51], v[0][:51])
    check(2, k[0], v[0])
    for j in range(3, 6):
        check(j, *pre)
    for j in (6, 7, 9, 10, 11):
        assert (out[j] == 0).all() and torch.isneginf(lse[j]).all()
    check(8, k[2], v[2])


def test_equals_the_paged_decode_over_whole_tables():
    """The same pages in every request's row: within the two calls' bars."""
    ps, P, own = 16, 320, [40, 7, 90]  # full prefix pages
    args, k, v = make([(P, own)], [2] * 3, 32, 8, 128, ps)
    q, kc, vc, ptab, plens, cu, tab, lens = args
    whole = torch.cat((ptab[:, :P // ps].expand(3, -1), tab), 1).contiguous()
    ref, rlse = ra.ra_paged_decode(q, kc, vc, whole, lens + P)
    out, lse = ra.ra_paged_decode_prefix(*args)
    ra.ra_device_status()
    A = float(q.float().norm(dim=-1).max()) * max(float(x.float().norm(dim=-1).max()) for x in k) / math.sqrt(128)
    bar = 4 * 128 * U * A + 2.0 ** -16 + 500 * 2 * U
    assert float((out - ref).abs().max()) <= 2 * bar * max(float(x.abs().max()) for x in v)
    assert float((lse - rlse).abs().max()) <= 2 * (2 * 128 * U * A + 500 * 2 * U + 8 * U * 12)


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("scale", [0.0, 40.0])
def test_equal_and_large_scores(scale, room):
    args, k, v = make([(700, [50, 3] * 20)], [1] * 40, 8, 2, 128, 16, scale=scale, room=room)
    out, lse = ra.ra_paged_decode_prefix(*args)
    ra.ra_device_status()
    check_decode(out, lse, args[0], k, v, [1] * 40)


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("n_q, per, H, Hkv, d", [(1, 2, 8, 2, 64), (1, 3, 8, 2, 128), (1, 40, 8, 2, 128), (2, 40, 8, 1, 64)])
def test_weights_have_24_bits(n_q, per, H, Hkv, d, room):
    """As the paged decode's test of that name: an output is one weight of three
    live keys, here two in the prefix and one among the own, all others weightless:
    99 u there where parts meet, the join of the two launches two factors of 6.4 u
    and three roundings more: 115 u, 128 u is used."""
    P, n = 700, 40
    groups = [(P, [n] * per)]
    args, ks, vs = make(groups, [n_q] * per, H, Hkv, d, 16, seed=d + per, room=room)
    q, kc, vc, ptab, _, _, tab, _ = args
    r = np.random.default_rng(per)
    g = H // Hkv
    q.zero_()
    for t in range(per * n_q):
        for h in range(H):
            q[t, h, (t * g + h % g) % d] = 1.0
    live = [100, 650]

    def fill(pages, rows_k, rows_v, length):
        for p in range(-(-length // 16)):
            m = min(16, length - 16 * p)
            kc[pages[p], :m] = rows_k[16 * p:16 * p + m]
            vc[pages[p], :m] = rows_v[16 * p:16 * p + m]

    def rows(length, at, first):
        k = torch.full((length, Hkv, d), -200.0 * math.sqrt(d), device=DEV).bfloat16()
        v = torch.randn(length, Hkv, d, device=DEV).bfloat16()
        for j, a in enumerate(at):
            k[a] = torch.from_numpy(r.uniform(-1, 1, (Hkv, d)) * math.sqrt(d)).to(DEV).bfloat16()
            v[a] = 0.0
            v[a, :, first + j::3] = 1.0
        return k, v

    pk, pv = rows(P, live, 0)
    fill(ptab[0].tolist(), pk, pv, P)
    own = []
    for i in range(per):
        own.append(rows(n, [5], 2))
        fill(tab[i].tolist(), *own[i], n)
    out, lse = ra.ra_paged_decode_prefix(*args)
    ra.ra_device_status()
    for i in range(per):
        rr = slice(i * n_q, (i + 1) * n_q)
        k, v = torch.cat((pk, own[i][0])), torch.cat((pv, own[i][1]))
        ro, rl = attend(q[rr], k, v, n, n_q)
        err = np.abs(np64(out[rr]) - ro)
        assert (err <= 128 * U * ro).all(), f"max error {(err / (U * ro)).max():.1f} u"
        assert (np.abs(np64(lse[rr]) - rl) <= 132 * U).all()


@pytest.mark.parametrize("n_q, room", [(2, False), (8, True)])
def test_arrays_in_disorder_stay_inside(n_q, room):
    """Offsets that are no prefix sums, lengths and pages out of range: results
    are undefined, nothing outside out and lse is written, nothing hangs."""
    args, k, v = make([(300, [50, 20]), (129, [77, 10, 41])], [n_q] * 5, 8, 2, 128, 16, room=room)
    T = 5 * n_q
    whole = torch.full((T + 4, 8, 128), 3.0, device=DEV)
    wl = torch.full((T + 4, 8), 3.0, device=DEV)
    for cu_req in ([0, 5, 2], [-7, 3, 99], [4, 1, 0], [2**31 - 1, -2**31, 5]):
        for plens in ([300, 129], [-5, 10**9], [2**31 - 1, -2**31]):
            for cu_q in (None, [0, 9, 3, 99, -4, T], [5, 4, 3, 2, 1, 0], [-9, 2, 4, 6, 8, 2**31 - 1]):
                a = list(args)
                a[5], a[4] = i32(cu_req), i32(plens)
                ra.ra_paged_decode_prefix(*a, cu_q=None if cu_q is None else i32(cu_q), out=whole[2:T + 2], lse=wl[2:T + 2])
    ra.ra_device_status()
    assert (whole[:2] == 3).all() and (whole[T + 2:] == 3).all() and (wl[:2] == 3).all() and (wl[T + 2:] == 3).all()
    bad = args[3].clone()
    bad[0, ::2] = 2**30
    bad[1, 1::2] = -1
    a = list(args)
    a[3] = bad
    ra.ra_paged_decode_prefix(*a)
    ra.ra_device_status()


@pytest.mark.parametrize("n_q, room", [(1, False), (6, True)])
def test_captured_and_replayed_as_lengths_grow(n_q, room):
    """Two graphs of one call on two streams share no workspace and bake no host value in."""
    groups = [(500, [60, 3, 20]), (1300, [90])]
    args, k, v = make(groups, [n_q] * 4, 32, 8, 128, 16, room=room)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ra.ra_paged_decode_prefix(*args))
        graphs.append(g)
    of = [0, 0, 0, 1]
    for plens, own in (([500, 1300], [60, 3, 20, 90]), ([1, 700], [1, 1, 1, 50]), ([0, 129], [60, 3, 7, 90])):
        args[4].copy_(i32(plens))
        args[7].copy_(i32(own))
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for _ in range(3):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()

        def part(x, i, j):  # what row j of request i sees: the prefix, however few its own keys are
            P = groups[of[i]][0]
            return torch.cat((x[i][:plens[of[i]]], x[i][P:P + max(0, own[i] - n_q + j + 1)]))

        each = [(i, j) for i in range(4) for j in range(n_q)]
        for out, lse in outs:
            check_decode(out, lse, args[0], [part(k, *e) for e in each], [part(v, *e) for e in each], [1] * 4 * n_q)
    ra.ra_device_status()


def test_two_eager_calls_at_once_and_other_kernels_between():
    """Calls on two streams, in turn, with the plain decode among them: the second
    launch of a call starts before the first has ended, and touches nothing that
    a call before it still uses."""
    cases = [make([(900, [40, 2, 64])], [1] * 3, 32, 8, 128, 16, seed=1)[0],
             make([(2000, [700] * 5), (3, [9])], [16] * 6, 8, 2, 128, 16, seed=2, room=True)[0]]
    want = [ra.ra_paged_decode_prefix(*c) for c in cases]
    plain = [ra.ra_paged_decode(c[0], c[1], c[2], c[6], c[7]) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(20):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append((ra.ra_paged_decode_prefix(*c), ra.ra_paged_decode(c[0], c[1], c[2], c[6], c[7])))
    torch.cuda.synchronize()
    ra.ra_device_status()
    for i, (a, b) in enumerate(got):
        assert torch.equal(a[0], want[i % 2][0]) and torch.equal(a[1], want[i % 2][1])
        assert torch.equal(b[0], plain[i % 2][0]) and torch.equal(b[1], plain[i % 2][1])


@pytest.mark.parametrize("room", [False, True])
def test_a_chain_in_one_stream_uses_what_the_call_before_wrote(room):
    """Every step's keys are written by the kernel just before the call."""
    groups = [(300, [33] * 12)]
    args, k, v = make(groups, [1] * 12, 8, 2, 128, 16, seed=5, room=room)
    q, kc, vc, ptab, plens, cu, tab, lens = args
    k0, v0 = kc.clone(), vc.clone()
    want = ra.ra_paged_decode_prefix(*args)
    for _ in range(30):
        kc.zero_()
        vc.zero_()
        kc.copy_(k0)
        vc.copy_(v0)
        got = ra.ra_paged_decode_prefix(*args)
        kc.fill_(1.0)  # what follows must not reach the call either
        vc.fill_(1.0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("per, room, launches", [(2, True, [0, 1, 1]), (100, False, [0, 1, 1]), (100, True, [1, 1, 1])])
def test_tracing_counts_the_launches(per, room, launches):
    """Few rows or a short prefix: the own keys and the prefix in one launch."""
    args, k, v = make([(300, [50, 20] * (per // 2))], [1] * per, 8, 2, 128, 16, room=room)
    ra.ra_trace_enable()
    ra.ra_trace_reset()
    try:
        out, lse = ra.ra_paged_decode_prefix(*args)
        check_decode(out, lse, args[0], k, v, [1] * per)
        assert [ra.ra_trace_query(x)[0] for x in ("paged_decode", "paged_prefix", "paged_combine")] == launches
    finally:
        ra.ra_trace_enable(False)


def test_a_serving_loop_on_a_shared_prompt():
    """A prompt is cached once, as a request of its own; three requests go on from
    it, token by token, at positions behind it: extend, append, attend, captured
    as a step would be.  Against the oracle over each whole sequence."""
    H, Hkv, d, ps, P, steps, n = 8, 2, 128, 16, 203, 6, 3
    g = torch.Generator(device=DEV).manual_seed(4)
    ph = ra.rope_phases(ra.rope_freqs(d)[0]).to(DEV)
    n_pages = 40
    kc = torch.full((n_pages, ps, Hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    free, count = torch.randperm(n_pages).int().to(DEV), i32([n_pages])
    ptab, plen = torch.full((1, 20), -1, dtype=torch.int32, device=DEV), i32([0])
    kp, vp = (torch.randn(P, Hkv, d, device=DEV, generator=g).bfloat16() for _ in range(2))
    qp = torch.randn(P, H, d, device=DEV, generator=g).bfloat16()
    slots, pos, *_ = ra.ra_paged_extend(plen, i32([P]), ptab, free, count, page_size=ps, tokens=P,
                                        lengths_out=plen, free_count_out=count)
    ra.ra_paged_append(qp, kp, vp, ph, kc, vc, slots, pos)
    tab, lens = torch.full((n, 4), -1, dtype=torch.int32, device=DEV), i32([0] * n)
    q, k, v = (torch.randn(steps, n, h, d, device=DEV, generator=g).bfloat16() for h in (H, Hkv, Hkv))
    outs = []
    for s in range(steps):
        slots, pos, cu, _, _, status = ra.ra_paged_extend(
            lens, i32([1] * n), tab, free, count, page_size=ps, tokens=n, lengths_out=lens, free_count_out=count)
        qr = ra.ra_paged_append(q[s], k[s], v[s], ph, kc, vc, slots, pos + plen)
        outs.append(ra.ra_paged_decode_prefix(qr, kc, vc, ptab, plen, i32([0, n]), tab, lens)[0])
    ra.ra_device_status()
    for i in range(n):
        kk, vv = torch.cat((kp, k[:, i])), torch.cat((vp, v[:, i]))
        qq = torch.cat((qp, q[:, i]))
        qr, kr = ra.ra_qk_norm_rope(qq, kk, ph)
        ref, _ = oracle.attention(qr[-steps:].cpu(), kr.cpu(), vv.cpu(), causal=True,
                                  q_pos=P + np.arange(steps), k_pos=np.arange(P + steps))
        got = np.stack([np64(o[i]) for o in outs])
        assert np.abs(got - ref).max() <= 1e-4
    # Own pages go back, the prefix's stay out.
    ra.ra_paged_release(lens, i32([1] * n), tab, free, count, page_size=ps, lengths_out=lens, free_count_out=count)
    assert int(count) == n_pages - -(-P // ps)


def test_wrong_tensors_are_refused():
    args, _, _ = make([(60, [30, 20])], [1] * 2, 4, 2, 64, 16)
    run = lambda **kw: ra.ra_paged_decode_prefix(*[kw.get(n, x) for n, x in zip(  # noqa: E731
        ("q", "kc", "vc", "ptab", "plens", "cu_req", "tab", "lens"), args)])
    with pytest.raises(ValueError, match="prefix_table must be"):
        run(ptab=args[3][0])
    with pytest.raises(TypeError, match="prefix_lengths must be torch.int32"):
        run(plens=args[4].long())
    with pytest.raises(ValueError, match="cu_req must have shape"):
        run(cu_req=args[5][:1])
    with pytest.raises(TypeError, match="k_cache must be torch.bfloat16"):
        run(kc=args[1].half())
    with pytest.raises(ValueError, match="must match in pages"):
        run(vc=args[2][:-1])


@pytest.mark.parametrize("d, bf16", [(128, True), (128, False), (64, True), (64, False)])
def test_warps_that_are_tiles_apart(d, bf16):
    """Few rows and many short runs of tiles, keys from HBM and from L2 in turn: the
    warps that form a tile's weights drift apart by as much as the kernel lets
    them.  A weight handed over for another tile's shows as a wait that runs out,
    or as another result.  Every call's result is the first one's."""
    groups = [(16000, [int(x) for x in np.random.default_rng(d).integers(1, 300, 16)])]
    sets = [make(groups, [1] * 16, 32, 8, d, 16, seed=s) for s in range(3)]
    outs = [torch.empty(16, 32, d, dtype=torch.bfloat16 if bf16 else torch.float32, device=DEV) for _ in sets]
    want = []
    for (args, k, v), out in zip(sets, outs):
        _, lse = ra.ra_paged_decode_prefix(*args, out=out)
        ra.ra_device_status()
        check_decode(out, lse, args[0], k, v, [1] * 16)
        want.append((out.clone(), lse))
    for rep in range(12):
        cold = torch.empty(1 << 28, dtype=torch.uint8, device=DEV).fill_(rep)  # L2 holds something else
        got = []
        for i in range(3 if rep < 8 else 60):
            got.append((i % 3, ra.ra_paged_decode_prefix(*sets[i % 3][0], out=torch.empty_like(outs[0]))))
        ra.ra_device_status()
        for i, (out, lse) in got:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
        del cold


def test_more_groups_than_threads():
    """Every CTA looks through all of them; many are of no request or no key."""
    r = np.random.default_rng(7)
    groups = [(int(r.integers(0, 24)), [int(x) for x in r.integers(1, 12, int(r.integers(0, 3)))]) for _ in range(1200)]
    rows = [1] * sum(len(x) for _, x in groups)
    args, k, v = make(groups, rows, 2, 1, 64, 8)
    out, lse = ra.ra_paged_decode_prefix(*args)
    ra.ra_device_status()
    check_decode(out, lse, args[0], k, v, rows)


def test_cache_without_pages():
    q = torch.randn(4, 8, 128, device=DEV).bfloat16()
    none = torch.empty(0, 16, 2, 128, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    cu, zero = i32([0, 1, 2]), i32([0, 0])
    out, lse = ra.ra_paged_decode_prefix(q, none, none, table, zero, cu, table, zero)
    assert (out == 0).all() and torch.isneginf(lse).all()
    ra.ra_paged_decode_prefix(q, none, none, table, i32([40, 3]), cu, table, i32([2, 48]))  # pages that are not there
    ra.ra_device_status()


@pytest.mark.parametrize("per, room", [(2, False), (40, False), (40, True)])
@pytest.mark.parametrize("what", ["key", "value"])
def test_nan_in_a_prefix_stays_with_its_group(per, room, what):
    groups = [(300, [20] * per), (300, [20] * per)]
    args, k, v = make(groups, [1] * 2 * per, 8, 2, 128, 16, room=room)
    want = ra.ra_paged_decode_prefix(*args)
    page = int(args[3][0, 200 // 16])
    (args[1] if what == "key" else args[2])[page, 200 % 16, 1, 5] = float("nan")
    out, lse = ra.ra_paged_decode_prefix(*args)
    ra.ra_device_status()
    assert torch.equal(out[per:], want[0][per:]) and torch.equal(lse[per:], want[1][per:])
    assert torch.equal(out[:per, :4], want[0][:per, :4])  # the other KV head's rows
    if what == "key":
        assert out[:per, 4:].isnan().all() and lse[:per, 4:].isnan().all()
    else:
        assert out[:per, 4:, 5].isnan().all() and torch.equal(lse[:per], want[1][:per])


def test_outputs_left_out_on_another_stream():
    args, k, v = make([(900, [40, 2, 64])], [1] * 3, 32, 8, 128, 16)
    want = ra.ra_paged_decode_prefix(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream):
        got = ra.ra_paged_decode_prefix(*args, stream=st)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads_on_streams_of_their_own():
    cases = [make([(900, [40, 2, 64])], [1] * 3, 32, 8, 128, 16, seed=1)[0],
             make([(2000, [70] * 25), (3, [9])], [2] * 26, 8, 2, 128, 16, seed=2, room=True)[0]]
    want = [ra.ra_paged_decode_prefix(*c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(30):
                    out, lse = ra.ra_paged_decode_prefix(*cases[i])
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
from test_gpu_prefix import check_decode, make
args, k, v = make([(700, [64, 3] * 10), (50, [4])], [1] * 21, 8, 2, 128, 16, room=True)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out, lse = ra.ra_paged_decode_prefix(*args)
for _ in range(3):
    g.replay()
torch.cuda.synchronize()
check_decode(out, lse, args[0], k, v, [1] * 21)
ra.ra_device_status()
print("captured first")
"""


def test_first_call_of_a_process_may_be_captured():
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


@pytest.mark.slow
def test_rows_past_32_bit_offsets():
    """Outputs and states of more than 2^31 elements: the first and the last rows."""
    n_req, H, ps, P = 66000, 256, 8, 100
    assert n_req * H * 128 > 2**31
    g = torch.Generator(device=DEV).manual_seed(1)
    kv = torch.randn(2, n_req + 13, ps, 2, 128, generator=g, device=DEV).bfloat16()
    q = torch.empty(n_req, H, 128, dtype=torch.bfloat16, device=DEV)
    for part in q.split(6000):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV))
    table = torch.arange(n_req, dtype=torch.int32, device=DEV)[:, None].contiguous()
    ptab = torch.arange(n_req, n_req + 13, dtype=torch.int32, device=DEV)[None].contiguous()
    lens = torch.arange(n_req, dtype=torch.int32, device=DEV) % 8 + 1
    out = torch.empty_like(q)
    _, lse = ra.ra_paged_decode_prefix(q, kv[0], kv[1], ptab, i32([P]), i32([0, n_req]), table, lens, out=out)
    ra.ra_device_status()
    for i in (0, 1, n_req // 2, n_req - 2, n_req - 1):
        k, v = (torch.cat((x[n_req:].reshape(-1, 2, 128)[:P], x[i, :int(lens[i])])) for x in kv)
        check_decode(out[i:i + 1], lse[i:i + 1], q[i:i + 1], [k], [v], [1])


@pytest.mark.parametrize("order", ["rising", "falling", "steps", "one"])
@pytest.mark.parametrize("d, bf16", [(64, False), (64, True), (128, False), (128, True)])
def test_scores_far_above_those_before(order, d, bf16):
    """A row's first keys say nothing of the others: scores that climb by hundreds
    inside a tile and from tile to tile, fall, or stand out once in every 32 keys."""
    n, P = 24, 1500
    args, k, v = make([(P, [5] * n)], [1] * n, 8, 2, d, 16, seed=3, room=True)
    q, kc, ptab = args[0], args[1], args[3]
    u = torch.randn(2, d, device=DEV)
    u /= u.norm(dim=-1, keepdim=True)
    q[:] = (u.repeat_interleave(4, 0)[None] * torch.linspace(0.5, 3, n, device=DEV)[:, None, None]).bfloat16()
    at = torch.arange(P, device=DEV, dtype=torch.float32)
    size = {"rising": at * 0.4, "falling": (P - at) * 0.4, "steps": torch.floor(at / 90) * 30,
            "one": torch.where(at % 37 == 36, at * 0.3, -at * 0.1)}[order]
    rows = (u[None] * size[:, None, None] + 0.2 * torch.randn(P, 2, d, device=DEV)).bfloat16()
    for p in range(-(-P // 16)):
        part = rows[16 * p:16 * p + 16]
        kc[ptab[0, p], :len(part)] = part
    for x in k:
        x[:P] = rows
    out = torch.empty(q.shape, dtype=torch.bfloat16 if bf16 else torch.float32, device=DEV)
    _, lse = ra.ra_paged_decode_prefix(*args, out=out)
    ra.ra_device_status()
    check_decode(out, lse, q, k, v, [1] * n)
