"""Pages in 8 bits on the GPU, against the plain forms in 64 bits."""
import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import fp8_ref
import serve_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODE, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu
U = 2.0 ** -24  # an fp32 rounding


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def make_pages(n_pages, ps, hkv, d, fill=0x55, packed=False):
    """Pages of a recognisable byte; packed: k and v halves of one tensor."""
    def one(shape):
        return torch.full(shape, fill, dtype=torch.uint8, device=DEV)
    if packed:
        c, s = one((n_pages, 2, ps, hkv, d)).view(CODE), one((n_pages, 2, hkv, ps)).view(SCALE)
        return c[:, 0], c[:, 1], s[:, 0], s[:, 1]
    c, s = (n_pages, ps, hkv, d), (n_pages, hkv, ps)
    return one(c).view(CODE), one(c).view(CODE), one(s).view(SCALE), one(s).view(SCALE)


def random_pages(n_pages, ps, hkv, d, seed, packed=False):
    """Codes of every kind but NaN, scales 2^-9 .. 2^-3; and what they stand for."""
    kc, vc, ks, vs = make_pages(n_pages, ps, hkv, d, packed=packed)
    rng = np.random.default_rng(seed)
    vals = []
    for c, s in ((kc, ks), (vc, vs)):
        x, e = fp8_ref.quantise(rng.normal(size=(n_pages, ps, hkv, d)))
        e = rng.integers(-9, -2, e.shape)
        c.copy_(torch.from_numpy(x).to(DEV).float().to(CODE))
        s.view(torch.uint8).copy_(torch.from_numpy((e.transpose(0, 2, 1) + 127).astype(np.uint8)))
        vals.append(x * (2.0 ** e)[..., None])
    return kc, vc, ks, vs, vals[0], vals[1]


# ------------------------------------------------------------------ append

def special_rows(d, rng):
    """Rows of v at the type's corners (bf16 values)."""
    x = rng.normal(size=(16, d)).astype(np.float32)
    x[0] = 0
    x[1] = 0
    x[1, d - 1] = 1e-38
    x[2] *= 1e-37
    x[3] *= 3e37
    x[4, 3] = np.inf
    x[5, 0], x[5, 7] = np.nan, -np.inf
    x[6] = np.inf
    x[7] = rng.choice([1, -1], d) * 448.0
    x[8, :] = 1.0
    x[8, 1] = 450.0  # above 448 scales: the next scale
    x[9] = rng.integers(-32, 33, d) / 32 * 1.75  # halves of code steps
    x[10] = rng.integers(-128, 129, d) / 64 * 1.5
    x[11] = rng.normal(size=d) * 2.0 ** rng.integers(-30, 1, d)  # many of them subnormal
    x[12] = -np.abs(x[12])
    x[13, 1:] = 0
    x[14] = 2.0 ** -126
    x[15] = 3.38e38
    return torch.from_numpy(x).bfloat16()


@pytest.mark.parametrize("T, heads, hkv, d, ps, rot, inter, norm, packed", [
    (1, 1, 1, 64, 16, 64, False, False, False),
    (5, 8, 2, 128, 32, 128, False, True, True),
    (37, 12, 3, 64, 16, 32, True, True, False),
    (300, 32, 8, 128, 64, 128, False, True, False),
    (1500, 8, 8, 64, 256, 0, False, False, True),
    (5000, 4, 1, 128, 128, 96, True, True, False),
])
def test_append_fp8(T, heads, hkv, d, ps, rot, inter, norm, packed):
    rng = np.random.default_rng(T + d)
    n_pages = -(-T // ps) + 2
    packed_qkv = torch.from_numpy(rng.normal(size=(T, heads + 2 * hkv, d))).bfloat16()
    q, k, v = packed_qkv.split([heads, hkv, hkv], 1)
    sp = special_rows(d, rng)
    for i in range(min(T, 16)):
        v[i, i % hkv] = sp[i]
    phases = freqs = None
    if rot:
        freqs, _ = ra.rope_freqs(rot)
        phases = ra.rope_phases(freqs).to(DEV)
    qw = torch.from_numpy(1 + 0.2 * rng.normal(size=d)).float() if norm else None
    kw = torch.from_numpy(1 + 0.2 * rng.normal(size=d)).float() if norm else None
    slots = rng.permutation(n_pages * ps)[:T].astype(np.int64)
    if T > 4:
        slots[2], slots[T - 1] = -1, n_pages * ps  # padding
    pos = rng.integers(0, 2 ** 20, T).astype(np.int32)
    kc, vc, ks, vs = make_pages(n_pages, ps, hkv, d, packed=packed)
    dev = packed_qkv.to(DEV)
    dq, dk, dv = dev.split([heads, hkv, hkv], 1)
    qo = torch.full((T, heads, d), 7.0, dtype=torch.bfloat16, device=DEV)
    got = ra.ra_paged_append_fp8(
        dq, dk, dv, phases, kc, vc, ks, vs, torch.from_numpy(slots).to(DEV),
        torch.from_numpy(pos).to(DEV), q_weight=None if qw is None else qw.to(DEV),
        k_weight=None if kw is None else kw.to(DEV), interleaved=inter, q_out=qo)
    assert got is qo
    ra.ra_device_status()
    real = (slots >= 0) & (slots < n_pages * ps)
    page, row = slots[real] // ps, slots[real] % ps
    f = np.zeros(0) if freqs is None else freqs.numpy()
    kx, ksize = serve_ref.rope(k.double().numpy(), None if kw is None else kw.double().numpy(), pos,
                               f, eps=1e-6, interleaved=inter)
    qx, qsize = serve_ref.rope(q.double().numpy(), None if qw is None else qw.double().numpy(), pos,
                               f, eps=1e-6, interleaved=inter)
    # v: every bit is given.
    val, e = fp8_ref.quantise(v[torch.from_numpy(real)].double().numpy())
    held = vc.double().cpu().numpy()[page, row]
    np.testing.assert_array_equal(held, val)
    np.testing.assert_array_equal(bytes_of(vs)[page, :, row], e + 127)
    # k: fp32 arithmetic of some 32 roundings of the terms, then one to a code,
    # at most half a step: 2^-4 of the value or 2^-10 scales.
    kx, err = kx[real], 32 * U * ksize[real]
    byte = bytes_of(ks)[page, :, row].astype(np.int64)
    top = np.abs(kx).max(-1)
    slack = err.max(-1)
    s = 2.0 ** (byte - 127.0)
    assert (top <= 448 * s + slack).all() and ((top > 224 * s - slack) | (byte == 10)).all()
    held = kc.double().cpu().numpy()[page, row] * s[..., None]
    assert (np.abs(held - kx) <= np.maximum(2.0 ** -4 * (np.abs(kx) + err), 2.0 ** -10 * s[..., None]) + err).all()
    # q, and what no row went to.
    qg = qo.double().cpu().numpy()
    assert (np.abs(qg - qx)[real] <= 2.0 ** -8 * np.abs(qx[real]) + 2.0 ** -7 * 32 * U * qsize[real] + 32 * U * qsize[real]).all()
    assert (qg[~real] == 7.0).all()
    touched = np.zeros((n_pages, ps), bool)
    touched[page, row] = True
    for c, sc in ((kc, ks), (vc, vs)):
        assert (bytes_of(c)[~touched] == 0x55).all()
        assert (bytes_of(sc).transpose(0, 2, 1)[~touched] == 0x55).all()


def test_codes_of_k_are_those_of_the_plain_form():
    """Without norm and turn k is held as it came: every bit is given."""
    T, hkv, d, ps = 700, 4, 128, 16
    rng = np.random.default_rng(1)
    k = torch.from_numpy(rng.normal(size=(T, hkv, d)) * 2.0 ** rng.integers(-20, 20, (T, hkv, 1))).bfloat16()
    kc, vc, ks, vs = make_pages(50, ps, hkv, d)
    slots = torch.arange(T, device=DEV)
    ra.ra_paged_append_fp8(k.to(DEV), k.to(DEV), k.to(DEV), None, kc, vc, ks, vs, slots,
                           torch.zeros(T, dtype=torch.int32, device=DEV))
    val, e = fp8_ref.quantise(k.double().numpy())
    for c, s in ((kc, ks), (vc, vs)):
        np.testing.assert_array_equal(c.double().cpu().numpy().reshape(-1, hkv, d)[:T], val)
        np.testing.assert_array_equal(bytes_of(s).transpose(0, 2, 1).reshape(-1, hkv)[:T], e + 127)


@pytest.mark.parametrize("d", [64, 128])
def test_a_row_that_is_not_finite_leaves_its_neighbours_alone(d):
    """Every byte of the other rows is as without it, a zero's sign among them."""
    T, hkv, ps = 6, 8, 16
    x = torch.randn(T, hkv, d).bfloat16()
    x[:, :, ::3] = -0.0
    x[:, :, 1::6] = 0.0
    other = x.clone()
    other[2, 3, 5], other[4, 0, 1], other[4, 7, d - 1] = float("inf"), float("nan"), -float("inf")
    slots = torch.arange(T, device=DEV)
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    held = []
    for y in (x.to(DEV), other.to(DEV)):
        pages = make_pages(1, ps, hkv, d)
        ra.ra_paged_append_fp8(y, y, y, None, *pages, slots, pos)
        held.append([bytes_of(p) for p in pages])
    ra.ra_device_status()
    same = np.ones((1, ps, hkv), bool)
    same[0, [2, 4, 4], [3, 0, 7]] = False
    for a, b in zip(held[0][:2], held[1][:2]):
        np.testing.assert_array_equal(a[same], b[same])
    v = held[0][1][0, :T]
    assert (v[..., ::3] == 0x80).all() and (v[..., 1::6] == 0).all()
    for a, b in zip(held[0][2:], held[1][2:]):
        np.testing.assert_array_equal(a.transpose(0, 2, 1)[same], b.transpose(0, 2, 1)[same])


# ------------------------------------------------------------------ read

def read_expected(vals, table, lens, cu, tokens, ps, before):
    out = before.copy()
    for i, n in enumerate(lens):
        for t in range(max(cu[i], 0), min(cu[i + 1], tokens)):
            pos = n - (cu[i + 1] - t)
            pg = table[i][pos // ps] if 0 <= pos < n else -1
            out[t] = vals[pg, pos % ps] if 0 <= pg < vals.shape[0] else 0
    return out


@pytest.mark.parametrize("hkv, d, ps, packed, lens, rows, extra", [
    (1, 64, 16, False, [1], [1], 0),
    (8, 128, 16, False, [17, 0, 300, 1, 0], None, 3),
    (3, 64, 64, True, [64, 65, 1000], [10, 70, 1000], 5),  # the newest, and more than there are
    (4, 128, 256, False, [700, 5], [0, 5], 0),
    (2, 128, 32, True, list(range(0, 150)), None, 0),
    (8, 64, 32, False, [9000, 33, 4097], [9000, 1, 3000], 0),
])
def test_read_fp8(hkv, d, ps, packed, lens, rows, extra):
    rng = np.random.default_rng(d + ps)
    n_pages = sum(-(-n // ps) for n in lens) + 2
    kc, vc, ks, vs, kv, vv = random_pages(n_pages, ps, hkv, d, 3, packed)
    width = max(1, max(-(-n // ps) for n in lens))
    table = np.full((len(lens), width), -1, np.int32)
    ids = list(rng.permutation(n_pages))
    for i, n in enumerate(lens):
        for c in range(-(-n // ps)):
            table[i, c] = ids.pop()
    cu = np.concatenate([[0], np.cumsum(rows or lens)]).astype(np.int32)
    tokens = int(cu[-1]) + extra
    before = torch.full((tokens, hkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
    ko, vo = before.clone(), before.clone()
    dev = [torch.from_numpy(x).to(DEV) for x in (table, np.array(lens, np.int32), cu)]
    got = ra.ra_paged_read_fp8(kc, vc, ks, vs, *dev, tokens=tokens, k_out=ko, v_out=vo)
    assert got[0] is ko and got[1] is vo
    ra.ra_device_status()
    for out, vals in ((ko, kv), (vo, vv)):
        want = read_expected(vals, table, lens, cu, tokens, ps, before.double().cpu().numpy())
        np.testing.assert_array_equal(out.double().cpu().numpy(), want)
    if not extra:  # outputs of its own
        k2, v2 = ra.ra_paged_read_fp8(kc, vc, ks, vs, *dev, tokens=tokens)
        assert torch.equal(k2, ko) and torch.equal(v2, vo) and k2.dtype == torch.bfloat16


def test_read_fp8_bad_pages_lengths_and_offsets():
    """Pages outside the cache are zeros, lengths past the table count as its
    width, and offsets that are no prefix sums write no row twice outside."""
    ps, hkv, d = 16, 2, 64
    kc, vc, ks, vs, kv, vv = random_pages(6, ps, hkv, d, 5)
    table = np.array([[0, 6, 2], [-1, 4, 5]], np.int32)
    lens, cu, tokens = [60, 33], np.array([0, 48, 81], np.int32), 81
    dev = [torch.from_numpy(x).to(DEV) for x in (table, np.array(lens, np.int32), cu)]
    k, v = ra.ra_paged_read_fp8(kc, vc, ks, vs, *dev, tokens=tokens)
    for out, vals in ((k, kv), (v, vv)):
        want = read_expected(vals, table, [48, 33], cu, tokens, ps, np.zeros((tokens, hkv, d)))
        np.testing.assert_array_equal(out.double().cpu().numpy(), want)
    # Offsets past the output and before it: the rows inside are written, no others.
    whole = torch.full((tokens + 8, hkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
    ko = whole[4:4 + tokens]
    cu2 = torch.tensor([-5, 48, 500], dtype=torch.int32, device=DEV)
    ra.ra_paged_read_fp8(kc, vc, ks, vs, dev[0], dev[1], cu2, tokens=tokens, k_out=ko, v_out=ko.clone())
    ra.ra_device_status()
    assert (whole[:4] == 3).all() and (whole[-4:] == 3).all()


def test_what_is_appended_is_read_back():
    """Append, then read: within half a code step of what went in, and reading
    gives what the codes and scales stand for."""
    T, hkv, d, ps = 333, 2, 128, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(T, hkv, d, device=DEV, dtype=torch.bfloat16, generator=g) for _ in range(2))
    kc, vc, ks, vs = make_pages(30, ps, hkv, d)
    table = torch.randperm(30)[:21].int().to(DEV).view(1, 21)
    t = torch.arange(T, device=DEV)
    slots = table[0, t // ps].long() * ps + t % ps
    ra.ra_paged_append_fp8(k, k, v, None, kc, vc, ks, vs, slots, t.int())
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    got = ra.ra_paged_read_fp8(kc, vc, ks, vs, table, cu[1:], cu, tokens=T)
    for out, x in zip(got, (k, v)):
        val, e = fp8_ref.quantise(x.double().cpu().numpy())
        np.testing.assert_array_equal(out.double().cpu().numpy(), val * (2.0 ** e)[..., None])


@pytest.mark.parametrize("d, hkv", [(64, 3), (128, 1)])
def test_read_fp8_to_outputs_at_16_bytes(d, hkv):
    """Outputs need 16-byte alignment and no more."""
    ps, n = 16, 100
    kc, vc, ks, vs, kv, vv = random_pages(9, ps, hkv, d, 6)
    table = torch.randperm(9)[:7].int().to(DEV).view(1, 7)
    lens, cu = torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV)
    want = ra.ra_paged_read_fp8(kc, vc, ks, vs, table, lens, cu, tokens=n)
    for k_off, v_off in ((8, 0), (0, 8), (8, 8)):
        flat = [torch.full((n * hkv * d + 16,), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        ko, vo = (f[o:o + n * hkv * d].view(n, hkv, d) for f, o in zip(flat, (k_off, v_off)))
        ra.ra_paged_read_fp8(kc, vc, ks, vs, table, lens, cu, tokens=n, k_out=ko, v_out=vo)
        assert torch.equal(ko, want[0]) and torch.equal(vo, want[1])
        for f, o in zip(flat, (k_off, v_off)):
            assert (f[:o] == 3).all() and (f[o + n * hkv * d:] == 3).all()


def test_append_in_place_and_captured():
    """q_out = q; a graph replayed with other slots and inputs; eps = 0."""
    T, heads, hkv, d, ps = 40, 8, 2, 128, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    data = [torch.randn(T, heads + 2 * hkv, d, generator=g, device=DEV).bfloat16() for _ in range(3)]
    w = torch.rand(d, generator=g, device=DEV) + 0.5
    freqs, _ = ra.rope_freqs(d)
    phases = ra.rope_phases(freqs).to(DEV)
    slots = [torch.randperm(64, generator=g, device=DEV)[:T] for _ in range(3)]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)

    def split(x):
        return [y.contiguous() for y in x.split([heads, hkv, hkv], 1)]

    def fresh():
        return make_pages(4, ps, hkv, d)

    kw = dict(q_weight=w, k_weight=w, eps=0.0)
    q, k, v = split(data[0])
    at, pages = slots[0].clone(), fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert ra.ra_paged_append_fp8(q, k, v, phases, *pages, at, pos, q_out=q, **kw) is q
    for x, s in zip(data, slots):
        want = fresh()
        x3 = split(x)
        qw = ra.ra_paged_append_fp8(*x3, phases, *want, s, pos, **kw)
        for y, z in zip((q, k, v), x3):
            y.copy_(z)
        at.copy_(s)
        for p in pages:
            p.view(torch.uint8).fill_(0x55)
        graph.replay()
        ra.ra_device_status()
        assert torch.equal(q, qw) and qw.isfinite().all()
        for a, b in zip(pages, want):
            np.testing.assert_array_equal(bytes_of(a), bytes_of(b))


def test_read_of_more_requests_than_threads_captured():
    """Most of them without a row; replayed with other lengths and offsets."""
    n, ps, hkv, d = 5000, 16, 2, 64
    rng = np.random.default_rng(3)
    kc, vc, ks, vs, kx, vx = random_pages(600, ps, hkv, d, 4)
    table = torch.from_numpy(rng.integers(0, 600, (n, 3)).astype(np.int32)).to(DEV)
    lens = torch.zeros(n, dtype=torch.int32, device=DEV)
    cu = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    tokens = 4000
    ko, vo = (torch.full((tokens, hkv, d), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.ra_paged_read_fp8(kc, vc, ks, vs, table, lens, cu, tokens=tokens, k_out=ko, v_out=vo)
    for seed in range(3):
        r = np.random.default_rng(seed)
        length = r.integers(0, 3 * ps + 1, n)
        rows = np.where(r.random(n) < 0.03, r.integers(0, length + 1), 0)
        lens.copy_(torch.from_numpy(length.astype(np.int32)))
        offs = np.concatenate([[0], np.cumsum(rows)])
        assert 0 < offs[-1] < tokens
        cu.copy_(torch.from_numpy(offs.astype(np.int32)))
        ko.fill_(5.0)
        vo.fill_(5.0)
        graph.replay()
        ra.ra_device_status()
        for out, x in ((ko, kx), (vo, vx)):
            got = out.double().cpu().numpy()
            for i in np.flatnonzero(rows):
                h = x[table[i].cpu().numpy()].reshape(-1, hkv, d)[length[i] - rows[i]:length[i]]
                np.testing.assert_array_equal(got[offs[i]:offs[i + 1]], h)
            assert (got[offs[-1]:] == 5.0).all()


@pytest.mark.parametrize("hkv, d", [(1, 64), (3, 64), (3, 128), (9, 64)])
def test_read_of_long_histories(hkv, d):
    """So many tokens that a warp takes as many rows together as it can."""
    ps, n_pages = 32, 3000
    kc, vc, ks, vs, kx, vx = random_pages(n_pages, ps, hkv, d, hkv)
    rng = np.random.default_rng(d)
    lens = np.array([250000, 1, 0, 99999, 7, 180001])
    table = rng.integers(0, n_pages, (6, 8000)).astype(np.int32)
    rows = lens - np.array([33, 0, 0, 5, 7, 0])
    cu = np.concatenate([[0], np.cumsum(rows)])
    dev = [torch.from_numpy(x.astype(np.int32)).to(DEV) for x in (table, lens, cu)]
    got = ra.ra_paged_read_fp8(kc, vc, ks, vs, *dev, tokens=int(cu[-1]))
    ra.ra_device_status()
    for out, x in zip(got, (kx, vx)):
        pages = torch.from_numpy(x).to(DEV).to(torch.bfloat16)  # exact
        for i in range(6):
            t = torch.arange(int(lens[i] - rows[i]), int(lens[i]), device=DEV)
            want = pages[dev[0][i].long()[t // ps], t % ps]
            assert torch.equal(out[int(cu[i]):int(cu[i + 1])], want)
