"""The serving and rotary calls at their edges: streams other than the current
one, values that are not finite, launches counted, long sequences and offsets
past 32 bits, and tolerances tight enough to see a lost term of the softmax
weights or a lost partial sum.

u = 2^-24 throughout (half a step of fp32, relative).
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
import serve_ref
from blockwise_online_softmax_gb300 import binding
from test_gpu_paged import check_decode, i32, make_decode
from test_gpu_rope import check_rope, np64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from blockwise_online_softmax_gb300 import build

    build.build()
    binding.lib()
    yield
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ the gradient's weights

@pytest.mark.parametrize("d, H, Hkv", [(128, 3, 1), (64, 5, 1), (64, 2, 2), (128, 2, 2)])
def test_weight_gradient_without_eps(d, H, Hkv):
    """eps = 0 is allowed.  With heads that do not fill a warp's rows, the
    rows of nobody must not add (0 / 0) to the sums.  The bar is the one of
    the other gradients: 64 u for a term, n u for their sum."""
    T, g = 9, torch.Generator().manual_seed(d + H)
    q, k, dqo, dko = (torch.randn(T, h, d, generator=g).to(DEV) for h in (H, Hkv, H, Hkv))
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
    f = ra.rope_freqs(64)[0]
    got = ra.ra_qk_norm_rope_backward(q, k, ra.rope_phases(f).to(DEV), dqo, dko, q_weight=w,
                                      k_weight=w, eps=0.0)
    for x, dy, dx, dw in ((q, dqo, got[0], got[2]), (k, dko, got[1], got[3])):
        rx, rw, size, wsize = serve_ref.rope_grad(np64(x), np64(w), np.arange(T), f.numpy(),
                                                  np64(dy), eps=0.0)
        assert (np.abs(np64(dx) - rx) <= 128 * U * size + 1e-30).all()
        assert (np.abs(np64(dw) - rw) <= (64 + T * x.shape[1]) * U * wsize).all()


# ------------------------------------------------------------------ streams

def side_calls():
    """Each call as f(stream) -> its outputs (what it updates in place it
    updates to the same every time), and the bytes of its first allocation."""
    g = torch.Generator(device=DEV).manual_seed(3)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEV).to(dtype)

    T, H, Hkv, d, ps = 8192, 8, 2, 128, 16
    q, k, v = randn(T, H, d), randn(T, Hkv, d), randn(T, Hkv, d)
    ph = ra.rope_phases(ra.rope_freqs(d)[0]).to(DEV)
    dqo, dko = randn(T, H, d, dtype=torch.float32), randn(T, Hkv, d, dtype=torch.float32)
    n = 1 << 20
    lens, news = i32(np.arange(n) % 7), i32(np.arange(n) % 3)
    tokens = int(news.sum())
    table = i32(np.arange(n)).view(n, 1)
    free, count = i32(np.arange(n)), i32([n // 2])
    kc, vc = randn(T // ps, ps, Hkv, d), randn(T // ps, ps, Hkv, d)
    slots, pos = torch.arange(T, device=DEV), i32(np.arange(T))
    ptab, plen = i32(np.arange(T // ps)).view(16, -1), i32(np.full(16, T // 16))

    out, lse = torch.zeros_like(dqo), torch.full((T, H), 5.0, device=DEV)

    def up(*sizes):
        return sum(-(-x // 512) * 512 for x in sizes)

    return {
        "rope": (lambda s: ra.ra_qk_norm_rope(q, k, ph, stream=s), up(q.numel() * 2)),
        "rope backward": (lambda s: ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, stream=s)[:2],
                          up(q.numel() * 2)),
        "extend": (lambda s: ra.ra_paged_extend(lens, news, table, free, count, page_size=16,
                                                tokens=tokens, stream=s),
                   up(tokens * 8, tokens * 4, n * 4 + 4, n * 4, 4, 12)),
        "release": (lambda s: ra.ra_paged_release(lens, news, table, free, count,
                                                  page_size=16, stream=s), up(n * 4, 4)),
        "append": (lambda s: (ra.ra_paged_append(q, k, v, ph, kc, vc, slots, pos, stream=s),),
                   up(q.numel() * 2)),
        "decode": (lambda s: ra.ra_paged_decode(q, kc, vc, ptab, plen, stream=s),
                   up(q.numel() * 4, T * H * 4)),
        "ring": (lambda s: ra.ra_ring_forward(q, k, v, P=4, causal=True, stream=s), up(q.numel() * 4)),
        "ring backward": (lambda s: ra.ra_ring_backward(q, k, v, out, lse, q, P=4, causal=True,
                                                        stream=s), up(q.numel() * 4)),
        "contiguous decode": (lambda s: ra.ra_decode_forward(q[:4096], k, v, P=4, stream=s),
                              up(4096 * H * d * 4)),
    }


CALLS = ["rope", "rope backward", "extend", "release", "append", "decode", "ring", "ring backward",
         "contiguous decode"]
BUSY = 200_000_000  # cycles of a sleeping kernel: about 0.1 s


def same(a, b):
    return len(a) == len(b) and all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("form", ["object", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_outputs_left_out_belong_to_the_stream_of_the_call(name, form):
    """stream= other than the current one, outputs left out.  They must not
    take memory that work on the current stream still uses; a result that is
    dropped must not be written after its memory went to the current stream;
    and one that the current stream still reads must not go back early."""
    f, size = side_calls()[name]
    side = torch.cuda.Stream()
    s = side if form == "object" else side.cuda_stream
    torch.cuda.synchronize()
    want = [x if x is None else x.clone() for x in f(None)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        f(None)  # the scratch pool has memory for the side stream
    torch.cuda.synchronize()
    torch.cuda.empty_cache()

    # 1. Memory that the current stream has yet to write.
    block = torch.empty(size, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    block.fill_(171)
    del block
    got = f(s)
    torch.cuda.synchronize()
    assert same(got, want)

    # 2. A dropped result's memory, taken by the current stream.
    del got
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = f(s)
    del got
    block = torch.empty(size, dtype=torch.uint8, device=DEV).fill_(171)
    torch.cuda.synchronize()
    assert bool((block == 171).all())
    del block

    # 3. A dropped result that the current stream has yet to read.
    torch.cuda.empty_cache()
    got = f(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    keep = [x if x is None else x.clone() for x in got]
    del got
    with torch.cuda.stream(side):
        block = torch.empty(size, dtype=torch.uint8, device=DEV).fill_(171)
    torch.cuda.synchronize()
    assert same(keep, want)
    ra.ra_device_status()


@pytest.mark.parametrize("name", ["decode", "ring"])
@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_stream_by_its_handles(handle, name):
    """NULL and cudaStreamLegacy, with another stream current."""
    f, _ = side_calls()[name]
    want = f(None)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = f(handle)
    torch.cuda.synchronize()
    assert same(got, want)


# ------------------------------------------------------------------ launches counted

def test_trace_counts_every_launch_of_the_bookkeeping():
    """A large step is two launches, a small one is one."""
    def count(kind, run):
        ra.ra_trace_reset()
        ra.ra_trace_enable(True)
        try:
            run()
            return ra.ra_trace_query(kind)[0]
        finally:
            ra.ra_trace_enable(False)
            ra.ra_trace_reset()

    for n, launches in ((16, 1), (6000, 2)):
        lens, ones = i32(np.zeros(n)), i32(np.ones(n))
        table, free = i32(np.zeros(4 * n)).view(n, 4), i32(np.arange(n))
        got = count("paged_extend", lambda: ra.ra_paged_extend(
            lens, ones, table, free, i32([n]), page_size=16, tokens=n))
        assert got == launches
        got = count("paged_release", lambda: ra.ra_paged_release(
            ones, ones, table, free, i32([0]), page_size=16))
        assert got == launches


# ------------------------------------------------------------------ values that are not finite

@pytest.mark.parametrize("lengths, n_q, H, Hkv, d", [
    ([40, 30], 1, 8, 2, 128), ([60000, 50], 1, 8, 2, 64), ([300, 200], 16, 64, 8, 128),
    ([40000, 100], 16, 8, 1, 64),
])
def test_a_nan_key_gives_nan_and_not_an_empty_row(lengths, n_q, H, Hkv, d):
    """A key that is NaN makes the rows that see it NaN, the LSE too: -inf
    there says that a row sees no key.  Other requests are as without it."""
    q, kc, vc, table, lens, ks, vs = make_decode(lengths, [n_q] * 2, H, Hkv, d, 16)
    kc[table[0, 0].long(), 3] = float("nan")
    out, lse = ra.ra_paged_decode(q, kc, vc, table, lens)
    ra.ra_device_status()
    assert torch.isnan(out[:n_q]).all() and torch.isnan(lse[:n_q]).all()
    check_decode(out[n_q:], lse[n_q:], q[n_q:], ks[1:], vs[1:], [n_q])


# ------------------------------------------------------------------ softmax weights to 24 bits

def one_hot_case(lengths, n_q, H, Hkv, d, ps, spread, seed):
    """A decode whose scores are exact and whose outputs are single weights.
    Each query row picks one column of K (one product, no sum).  Of a
    request's keys three are live, with scores in [-1, 1]; the others are so
    far below that their weight is exactly 0 in fp32.  Column c of V is 1 at
    live key c % 3 and 0 at the two others."""
    q, kc, vc, table, lens, ks, vs = make_decode(lengths, [n_q] * len(lengths), H, Hkv, d, ps, seed=seed)
    r = np.random.default_rng(seed)
    g = H // Hkv
    q.zero_()
    for i in range(len(lengths)):
        for j in range(n_q):
            for h in range(H):
                q[i * n_q + j, h, (j * g + h % g) % d] = 1.0
    tab = table.cpu().numpy()
    for i, n in enumerate(lengths):
        live = np.sort(r.choice(n - n_q + 1, 3, replace=False)) if spread else np.arange(3)
        at = torch.from_numpy(live).to(DEV)
        ks[i].fill_(-200.0 * math.sqrt(d))
        ks[i][at] = torch.from_numpy(r.uniform(-1, 1, (3, Hkv, d)) * math.sqrt(d)).to(DEV).bfloat16()
        vs[i][at] = 0.0
        for c in range(3):
            vs[i][at[c], :, c::3] = 1.0
        for p in range(-(-n // ps)):
            part = slice(p * ps, min(n, p * ps + ps))
            kc[tab[i, p], :part.stop - part.start] = ks[i][part]
            vc[tab[i, p], :part.stop - part.start] = vs[i][part]
    return q, kc, vc, table, lens, ks, vs


WHOLE = [
    # n_q, heads, kv_heads, d: row tiles of 8, 16 and 128
    (1, 8, 2, 64), (1, 8, 2, 128), (3, 8, 2, 64), (3, 8, 2, 128), (5, 32, 4, 64), (16, 8, 1, 64),
    (5, 32, 8, 128), (16, 16, 2, 128),
]


@pytest.mark.parametrize("where", ["whole", "cut"])
@pytest.mark.parametrize("n_q, H, Hkv, d", WHOLE)
def test_weights_have_24_bits(n_q, H, Hkv, d, where):
    """An output is one weight p_i / l.  With scores s exact, y = s sl2 - m in
    one rounding (|y| <= 3: 2 u, times ln 2) with sl2 off by u of |s| log2 e
    (times ln 2: 1 u), and ex2 good to 2^-22 = 4 u: a weight is off by 6.4 u.
    Three terms of it meet V = 1 in a sum that truncates twice (2 u each) and
    one rounding; l adds two; 1 / l and the product one each: in an item of
    one tile 2 * 6.4 + 4 + 1 + 2 + 2 = 22 u, 32 u is used.  Where tiles, warps
    and parts meet, each of up to six levels brings a factor ex2(m - m') good
    to 6.4 u, in numerator and denominator: 22 + 2 * 6 * 6.4 = 99 u, 112 u is used.
    A weight in two bf16 terms is off by up to 2^-17 = 128 u (rounded) or
    2^-15 = 512 u (cut), which the first bar, or both, refuse."""
    lengths = [n_q + 2, n_q + 5, n_q + 9] if where == "whole" else [3000 + n_q, 70000, 500]
    got = one_hot_case(lengths, n_q, H, Hkv, d, 16, where == "cut", seed=d + n_q)
    q, kc, vc, table, lens, ks, vs = got
    out, lse = ra.ra_paged_decode(q, kc, vc, table, lens)
    ra.ra_device_status()
    bar = 32 if where == "whole" else 112
    for i, n in enumerate(lengths):
        rows = slice(i * n_q, (i + 1) * n_q)
        ro, rl = oracle.attention(q[rows].cpu(), ks[i].cpu(), vs[i].cpu(), causal=True,
                                  q_pos=n - n_q + np.arange(n_q), k_pos=np.arange(n))
        err = np.abs(np64(out[rows]) - ro)
        assert (err <= bar * U * ro).all(), f"max error {(err / (U * ro)).max():.1f} u"
        # The LSE: the weights' sum to the same, m ln 2 and the logarithm 2 u of |m ln 2| <= 1 each.
        assert (np.abs(np64(lse[rows]) - rl) <= (bar + 4) * U).all()


def test_bf16_output_of_every_row_tile():
    """bf16 outputs are the fp32 ones rounded once."""
    for n_q, H, Hkv, d in WHOLE:
        q, kc, vc, table, lens, _, _ = make_decode([700, 45, 3000], [n_q] * 3, H, Hkv, d, 32)
        want = ra.ra_paged_decode(q, kc, vc, table, lens)
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
        _, lse = ra.ra_paged_decode(q, kc, vc, table, lens, out=out)
        assert torch.equal(out, want[0].bfloat16()) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ angles and sums

@pytest.mark.parametrize("inter", [False, True])
def test_cos_and_sin_to_their_last_bits(inter):
    """Pairs (1, 0) give cos and sin themselves.  sincospif is good to an ulp
    (u here: the values are at most 1), its argument carries no rounding, the
    correction for the turn's low bits is one rounding (u / 2) with a factor
    below 4e-7: 1.6 u.  An argument rounded to 24 bits of half a turn costs
    pi 2^-25 = 1.6 u more."""
    d, T = 128, 4096
    f = ra.rope_freqs(d)[0]
    ph = ra.rope_phases(f)
    a, b = serve_ref.pairs(d, inter)
    x = torch.zeros(T, 1, d)
    x[..., a] = 1.0
    r = np.random.default_rng(0)
    pos = r.integers(-2 ** 31, 2 ** 31, T)
    pos[:1024] = np.arange(1024)
    x = x.to(DEV)
    out, _ = ra.ra_qk_norm_rope(x, x, ph.to(DEV), positions=i32(pos), interleaved=inter)
    turn = (pos.astype(np.int64)[:, None] * ph.numpy()[None, :])  # wraps, as the kernel's does
    ang = turn.astype(np.float64) * (2 * math.pi / 2.0 ** 64)
    got = np64(out)[:, 0]
    err = max(np.abs(got[:, a] - np.cos(ang)).max(), np.abs(got[:, b] - np.sin(ang)).max())
    assert err <= 1.6 * U, f"{err / U:.2f} u"


LONG = [
    # T, heads, kv_heads, d, rot, interleaved: whole tokens with shares of the rest's rows, and
    # sequences past eight turns of every warp
    (2701, 24, 8, 64, 32, True), (4099, 32, 8, 128, 128, False), (33001, 3, 1, 64, 64, False),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(str(x) for x in c))
def test_weight_gradients_of_long_sequences(case):
    """A term is off by 64 u of its size (see test_gpu_rope.py); up to 64 of
    them and four lanes are added in one word, the rest in two, and one
    rounding: 130 u of the absolute sum, however many there are.  What one CTA contributes is
    thousands of times that."""
    T, H, Hkv, d, rot, inter = case
    g = torch.Generator().manual_seed(T)
    q, k, dqo, dko = (torch.randn(T, h, d, generator=g).to(DEV) for h in (H, Hkv, H, Hkv))
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
    f = ra.rope_freqs(rot)[0]
    ph = ra.rope_phases(f).to(DEV)
    how = dict(q_weight=w, k_weight=w, interleaved=inter)
    qo, ko = ra.ra_qk_norm_rope(q, k, ph, **how)
    pos = np.arange(T)
    check_rope(qo, q, w, pos, f.numpy(), interleaved=inter)
    check_rope(ko, k, w, pos, f.numpy(), interleaved=inter)
    got = ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, **how)
    for x, dy, dx, dw in ((q, dqo, got[0], got[2]), (k, dko, got[1], got[3])):
        rx, rw, size, wsize = serve_ref.rope_grad(np64(x), np64(w), pos, f.numpy(), np64(dy),
                                                  eps=1e-6, interleaved=inter)
        assert (np.abs(np64(dx) - rx) <= 128 * U * size + 1e-30).all()
        assert (np.abs(np64(dw) - rw) <= 130 * U * wsize).all()
        assert np.abs(rw).max() > 1000 * 130 * U * wsize.max() / math.sqrt(T)  # the bar bites


@pytest.mark.parametrize("H, d", [(32, 128), (4, 64)])
def test_weight_gradients_keep_small_terms_beside_a_large_one(H, d):
    """Terms that are exact (rows of +-1 normalise to themselves without eps,
    nothing turns): one of 2^24 among ones.  In one fp32 word every addition
    after it is off by up to half a step, 1; here the 63 of its run are and two
    that join lanes, and the result has its own half step."""
    T = 40000
    g = torch.Generator(device=DEV).manual_seed(1)
    q = (torch.randint(0, 2, (T, H, d), generator=g, device=DEV) * 2 - 1).float()
    dy = q.clone()          # every term is dy x = 1
    dy[5, 1] *= 2.0 ** 24
    w = torch.ones(d, device=DEV)
    dw = ra.ra_qk_norm_rope_backward(q, q[:, :1].contiguous(), None, dy, dy[:, :1].contiguous(),
                                     q_weight=w, k_weight=w, eps=0.0)
    want = T * H - 1 + 2 ** 24
    assert (dw[2].double() - want).abs().max().item() <= 64 + want * U
    assert (dw[3] == T).all()


# ------------------------------------------------------------------ rows to expect

@pytest.mark.parametrize("d", [64, 128])
def test_padding_rows_do_not_pick_the_kernel(d):
    """A fixed-size step with cu_q and the rows to expect gives the bits of the
    call on its real rows, whatever the padding, and leaves that as it was."""
    rows, extra = [1] * 16, 240
    lengths = [int(x) for x in np.linspace(5, 900, 16)]
    q, kc, vc, table, lens, ks, vs = make_decode(lengths, rows, 32, 8, d, 16, extra=extra)
    want = ra.ra_paged_decode(q[:16], kc, vc, table, lens)
    out, lse = torch.full(q.shape, 9.0, device=DEV), torch.full(q.shape[:2], 9.0, device=DEV)
    ra.ra_paged_decode(q, kc, vc, table, lens, cu_q=i32(np.arange(17)), n_q=1, out=out, lse=lse)
    assert torch.equal(out[:16], want[0]) and torch.equal(lse[:16], want[1])
    assert (out[16:] == 9.0).all() and (lse[16:] == 9.0).all()


@pytest.mark.parametrize("n_q", [0, 1, 3, 5, 40, 2**31 - 1])
def test_rows_other_than_the_expected(n_q):
    lengths, rows = [500, 77, 300, 1025, 9], [300, 2, 0, 1, 1]
    q, kc, vc, table, lens, ks, vs = make_decode(lengths, rows, 8, 2, 128, 16)
    cu = i32(np.concatenate([[0], np.cumsum(rows)]))
    out, lse = ra.ra_paged_decode(q, kc, vc, table, lens, cu_q=cu, n_q=n_q)
    ra.ra_device_status()
    check_decode(out, lse, q, ks, vs, rows)


def test_rows_to_expect_without_cu_q_are_the_rows():
    q, kc, vc, table, lens, ks, vs = make_decode([60, 20], [2, 2], 8, 2, 128, 16)
    check_decode(*ra.ra_paged_decode(q, kc, vc, table, lens, n_q=2), q, ks, vs, [2, 2])
    with pytest.raises(ValueError, match="n_q=3"):
        ra.ra_paged_decode(q, kc, vc, table, lens, n_q=3)
    with pytest.raises(binding.RaError, match="n_q=-1"):
        ra.ra_paged_decode(q, kc, vc, table, lens, cu_q=i32([0, 2, 4]), n_q=-1)


# ------------------------------------------------------------------ sizes past the others

def test_decode_more_requests_than_threads_on_the_large_row_tile():
    """The 128-row kernel with several requests to a thread of its sums."""
    r = np.random.default_rng(5)
    lengths = [int(x) for x in r.integers(0, 200, 1300)]
    q, kc, vc, table, lens, ks, vs = make_decode(lengths, [5] * 1300, 8, 1, 128, 16)
    out, lse = ra.ra_paged_decode(q, kc, vc, table, lens)
    ra.ra_device_status()
    check_decode(out, lse, q, ks, vs, [5] * 1300)


def test_append_past_eight_turns_of_the_warps():
    T, H, Hkv, d, ps = 33001, 3, 1, 64, 32
    g = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn(T, h, d, generator=g).bfloat16().to(DEV) for h in (H, Hkv, Hkv))
    n_pages = -(-T // ps)
    kc, vc = (torch.zeros(n_pages, ps, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.randperm(n_pages * ps, generator=g)[:T].to(DEV)
    f = ra.rope_freqs(d)[0]
    qo = ra.ra_paged_append(q, k, v, ra.rope_phases(f).to(DEV), kc, vc, slots, i32(np.arange(T)))
    check_rope(qo, q, None, np.arange(T), f.numpy())
    check_rope(kc.view(-1, Hkv, d)[slots], k, None, np.arange(T), f.numpy())
    assert torch.equal(vc.view(-1, Hkv, d)[slots], v)


def test_rotary_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the first and last tokens, forward
    and backward; then token strides whose product with the index passes 2^32."""
    H, d = 128, 128
    T = (1 << 31) // (H * d) + 3
    g = torch.Generator(device=DEV).manual_seed(2)
    f = ra.rope_freqs(d)[0]
    ph = ra.rope_phases(f).to(DEV)
    w = torch.linspace(0.5, 1.5, d, device=DEV)
    q = torch.empty(T, H, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    k = torch.randn(T, 1, d, generator=g, device=DEV).bfloat16()
    at = [0, 1, T // 2, T - 2, T - 1]
    idx = torch.tensor(at, device=DEV)
    qo, _ = ra.ra_qk_norm_rope(q, k, ph, q_weight=w)
    check_rope(qo[idx], q[idx], w, np.array(at), f.numpy())
    del qo
    dqo = torch.empty(T, H, d, device=DEV).normal_(generator=g)
    dko = torch.randn(T, 1, d, generator=g, device=DEV)
    dq = ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, q_weight=w)[0]
    ref, _, size, _ = serve_ref.rope_grad(np64(q[idx]), np64(w), np.array(at), f.numpy(), np64(dqo[idx]), eps=1e-6)
    assert (np.abs(np64(dq[idx]) - ref) <= 128 * U * size + 2.0 ** -8 * np.abs(ref)).all()
    del dq, dqo, dko
    stride = (1 << 29) + 8
    buf = torch.empty(4 * stride + 2 * d, dtype=torch.bfloat16, device=DEV)
    far = buf.as_strided((5, 2, d), (stride, d, 1))
    far.copy_(q[:5, :2])
    qo, ko = ra.ra_qk_norm_rope(far, far, ph, q_weight=w)
    check_rope(qo, far, w, np.arange(5), f.numpy())
    assert torch.equal(ko, ra.ra_qk_norm_rope(far.contiguous(), far.contiguous(), ph)[1])
    dy = torch.randn(5, 2, d, generator=g, device=DEV)
    want = ra.ra_qk_norm_rope_backward(far.contiguous(), far.contiguous(), ph, dy, dy, q_weight=w)
    got = ra.ra_qk_norm_rope_backward(far, far.contiguous(), ph, dy, dy, q_weight=w, dq=far)  # dq is q
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_append_offsets_past_32_bits():
    """Slots whose elements lie past 2^32, and q, k, v as views with tokens
    2^29 elements apart."""
    ps, Hkv, d = 256, 8, 128
    n_pages = (1 << 32) // (ps * Hkv * d) + 4
    g = torch.Generator(device=DEV).manual_seed(3)
    kc = torch.empty(n_pages, ps, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    stride = (1 << 29) + 8
    buf = torch.empty(4 * stride + 3 * Hkv * d, dtype=torch.bfloat16, device=DEV)
    q, k, v = (buf.as_strided((5, Hkv, d), (stride, d, 1), i * Hkv * d) for i in range(3))
    for x in (q, k, v):
        x.copy_(torch.randn(5, Hkv, d, generator=g, device=DEV))
    last = n_pages * ps - 1
    slots = torch.tensor([0, last, -1, last - 300, last + 1], device=DEV)
    kc[-3:], vc[-3:] = 3.0, 3.0
    f = ra.rope_freqs(d)[0]
    pos = i32([5, 6, 7, 8, 9])
    qo = ra.ra_paged_append(q, k, v, ra.rope_phases(f).to(DEV), kc, vc, slots, pos)
    at, p = torch.tensor([0, 1, 3], device=DEV), np.array([5, 6, 8])
    page, row = slots[at] // ps, slots[at] % ps
    check_rope(qo[at], q[at], None, p, f.numpy())
    check_rope(kc[page, row], k[at], None, p, f.numpy())
    assert torch.equal(vc[page, row], v[at])
    assert int((vc[-3:] != 3.0).any(-1).any(-1).sum()) == 2  # two rows written there, no other


@pytest.mark.parametrize("n_q, H, Hkv, d", [(1, 4, 1, 64), (40, 4, 1, 64), (1, 4, 1, 128)])
def test_decode_at_the_longest_history(n_q, H, Hkv, d):
    """2^31 - 256 keys, the stated limit, as one page of the cache over and
    over.  With q = 0 every weight is 1 and V of 0 and 1 sums exactly inside a
    CTA (below 2^24); up to 304 partials and a warp's states join in fp32, a
    rounding each, and the LSE is that of the count.  Rows of a request see
    one key more each, which changes a mean by less than 2^-30."""
    ps, max_pages = 256, (1 << 23) - 1
    g = torch.Generator(device=DEV).manual_seed(1)
    kc = torch.randn(1, ps, Hkv, d, generator=g, device=DEV).bfloat16()
    vc = torch.randint(0, 2, (1, ps, Hkv, d), generator=g, device=DEV).bfloat16()
    table = torch.zeros(1, max_pages, dtype=torch.int32, device=DEV)
    q = torch.zeros(n_q, H, d, dtype=torch.bfloat16, device=DEV)
    out, lse = ra.ra_paged_decode(q, kc, vc, table, i32([max_pages * ps]))
    ra.ra_device_status()
    want = vc[0].double().mean(0)  # [Hkv, d], every page the same
    assert ((out.double() - want.repeat_interleave(H // Hkv, 0)).abs() <= 320 * U).all()
    assert (lse.double() - math.log(max_pages * ps)).abs().max().item() <= 320 * U + 2 * U * 22


def test_window_wider_than_any_history():
    q, kc, vc, table, lens, ks, vs = make_decode([300, 7], [2, 2], 8, 2, 128, 16)
    want = ra.ra_paged_decode(q, kc, vc, table, lens)
    for w in (2**31 - 1, 2**31, 2**62):
        got = ra.ra_paged_decode(q, kc, vc, table, lens, window=w)
        assert same(got, want)


def test_pages_out_of_range_stay_with_their_request():
    """A table entry that is no page, inside a request's length: that request's
    result is undefined, the others' are not, and nothing else is read."""
    for n_q, H in ((1, 8), (5, 32)):
        q, kc, vc, table, lens, ks, vs = make_decode([300, 700, 64], [n_q] * 3, H, 2, 128, 16)
        table[1, ::2] = torch.tensor([-1, 2**30, -2**31, kc.shape[0]], dtype=torch.int32,
                                     device=DEV).repeat(table.shape[1])[:table[1, ::2].numel()]
        out, lse = ra.ra_paged_decode(q, kc, vc, table, lens)
        ra.ra_device_status()
        for i in (0, 2):
            rows = slice(i * n_q, (i + 1) * n_q)
            check_decode(out[rows], lse[rows], q[rows], ks[i:i + 1], vs[i:i + 1], [n_q])


def test_extend_and_release_without_a_page_in_the_stack():
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    table = i32([[5, -1], [6, -1]])
    slots, _, cu, ln, count, status = ra.ra_paged_extend(
        i32([3, 0]), i32([2, 1]), table, none, i32([0]), page_size=8, tokens=3)
    assert status.tolist() == [1, 0, 0] and slots.tolist() == [-1] * 3 and ln.tolist() == [3, 0]
    slots, pos, cu, ln, count, status = ra.ra_paged_extend(
        i32([3, 0]), i32([2, 0]), table, none, i32([0]), page_size=8, tokens=3)
    assert status.tolist() == [0, 0, 0] and slots.tolist() == [43, 44, -1] and cu.tolist() == [0, 2, 2]
    ln, count = ra.ra_paged_release(ln, i32([1, 0]), table, none, i32([0]), page_size=8)
    assert ln.tolist() == [0, 0] and count.tolist() == [0]


def test_append_in_place():
    """q_out may be q where that is dense; padding rows of it stay as they are."""
    g = torch.Generator().manual_seed(9)
    T, H, Hkv, d = 50, 8, 2, 128
    q, k, v = (torch.randn(T, h, d, generator=g).bfloat16().to(DEV) for h in (H, Hkv, Hkv))
    kc, vc = (torch.zeros(8, 16, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.randperm(128, generator=g)[:T].to(DEV)
    slots[::7] = -1
    ph, w = ra.rope_phases(ra.rope_freqs(d)[0]).to(DEV), torch.linspace(0.5, 2.0, d, device=DEV)
    want = ra.ra_paged_append(q, k, v, ph, kc, vc, slots, i32(np.arange(T)), q_weight=w,
                              q_out=q.clone())
    old = q.clone()
    got = ra.ra_paged_append(q, k, v, ph, kc, vc, slots, i32(np.arange(T)), q_weight=w, q_out=q)
    assert got is q and torch.equal(q, want) and torch.equal(q[::7], old[::7])


# ------------------------------------------------------------------ two callers

def test_decode_from_two_threads():
    cases = [make_decode([3000, 40, 900], [1] * 3, 32, 8, 128, 16, seed=1),
             make_decode([2000, 700], [16] * 2, 8, 2, 128, 16, seed=2)]
    want = [ra.ra_paged_decode(*c[:5]) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(30):
                out, lse = ra.ra_paged_decode(*cases[i][:5])
                st.synchronize()
                if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])):
                    bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    ra.ra_device_status()
    assert not bad


# ------------------------------------------------------------------ a capture first

FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import blockwise_online_softmax_gb300 as ra
from test_gpu_paged import check_decode, make_decode
q, kc, vc, table, lens, ks, vs = make_decode([700, 64, 3000], [{n_q}] * 3, 32, 8, 128, 16)
f, w = ra.rope_freqs(128)[0], torch.ones(128, device="cuda")
ph, dy = ra.rope_phases(f).cuda(), torch.randn(q.shape, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out, lse = ra.ra_paged_decode(q, kc, vc, table, lens)
    grads = ra.ra_qk_norm_rope_backward(q, q, ph, dy, dy, q_weight=w, k_weight=w)
for _ in range(3):
    g.replay()
torch.cuda.synchronize()
check_decode(out, lse, q, ks, vs, [{n_q}] * 3)
want = ra.ra_qk_norm_rope_backward(q, q, ph, dy, dy, q_weight=w, k_weight=w)
assert all(torch.equal(a, b) for a, b in zip(grads, want))
ra.ra_device_status()
print("captured first")
"""


@pytest.mark.parametrize("n_q", [1, 8])
def test_first_call_of_a_process_may_be_captured(n_q):
    """No call has to run before a capture: pools, attributes and symbols are
    set up inside it."""
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests, n_q=n_q)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr
