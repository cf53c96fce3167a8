"""The q/k norm with rotary positions and its gradient on the GPU against
the plain 64-bit form.

Tolerances.  u = 2^-24.  An output is a c - b s of two fp32 terms whose
size is |a| + |b| (times mscale).  a and b carry the errors of the norm (a
sum of d <= 128 squares in 3 serial and log2(16) tree steps and 8 products,
a reciprocal root good to 2 ulp, two products: under 20 u), c and s those of
the angle (the top 32 bits of the phase to fp32: 2^-25 of at most half a
turn, pi 2^-25 = 1.6 u) and of sincospi (2 ulp), then two products and a
sum: under 32 u of that size together; 64 u is used.  A bf16 result adds its
half step, 2^-8 of the value.  dx has one more product, sum and mean: 128 u
of the sum of its absolute terms.  A weight gradient adds n terms, in any
order at most n u of their absolute sum, plus the terms' own 64 u.
"""
import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import serve_ref
from blockwise_online_softmax_gb300 import binding, inputs

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


def np64(t):
    return t.detach().cpu().double().numpy()


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 0.0


def check_rope(out, x, w, pos, freqs, **kw):
    ref, size = serve_ref.rope(np64(x), None if w is None else np64(w), pos, freqs, eps=1e-6, **kw)
    err = np.abs(np64(out) - ref)
    bar = 64 * U * size + half_step(out.dtype) * np.abs(ref) + 1e-30
    assert np.isfinite(np64(out)).all()
    assert (err <= bar).all(), f"max err / bar = {(err / bar).max():.2f}"


CASES = [
    # T, heads, kv_heads, d, rot, interleaved, dtype, norm q, norm k, weight dtype, mscale
    (1, 1, 1, 64, 64, False, "bf16", True, True, "f32", 1.0),
    (1, 32, 8, 128, 128, False, "bf16", True, True, "bf16", 1.0),
    (3, 3, 1, 64, 16, True, "f32", True, False, "f32", 1.2),
    (7, 5, 5, 128, 96, False, "f32", False, True, "f32", 0.9),
    (257, 8, 1, 128, 48, True, "bf16", True, True, "f32", 1.1),
    (130, 12, 4, 64, 32, False, "bf16", False, False, "f32", 1.0),
    (64, 2, 2, 128, 0, False, "bf16", True, True, "f32", 1.0),
    (65, 64, 8, 64, 48, False, "f32", True, True, "bf16", 1.0),
    (2000, 4, 2, 128, 128, True, "f32", True, True, "f32", 1.0),
    # more tokens than warps: whole ones first, then shares of the rest's rows
    (4099, 32, 8, 128, 128, False, "bf16", True, True, "f32", 1.0),
    (2701, 24, 8, 64, 32, True, "f32", True, True, "f32", 1.1),
]


def make(case, seed=0):
    T, H, Hkv, d, rot, inter, dt, nq, nk, wdt, ms = case
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    g = torch.Generator().manual_seed(seed + T)
    qkv = (torch.randn(T, H + 2 * Hkv, d, generator=g) * 1.5).to(dtype).to(DEV)
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]  # views of a packed projection
    wt = torch.bfloat16 if wdt == "bf16" else torch.float32
    qw = (1 + 0.2 * torch.randn(d, generator=g)).to(wt).to(DEV) if nq else None
    kw = (1 + 0.2 * torch.randn(d, generator=g)).to(wt).to(DEV) if nk else None
    f = ra.rope_freqs(rot)[0].numpy() if rot else np.zeros(0)
    ph = ra.rope_phases(torch.from_numpy(f)).to(DEV) if rot else None
    return q, k, qw, kw, f, ph, dict(mscale=ms, interleaved=inter), g


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_forward(case):
    q, k, qw, kw, f, ph, how, _ = make(case)
    qo, ko = ra.ra_qk_norm_rope(q, k, ph, q_weight=qw, k_weight=kw, **how)
    pos = np.arange(q.shape[0])
    check_rope(qo, q, qw, pos, f, **how)
    check_rope(ko, k, kw, pos, f, **how)


def check_grads(got, q, k, qw, kw, pos, f, dqo, dko, **how):
    for x, w, dy, dx, dw in ((q, qw, dqo, got[0], got[2]), (k, kw, dko, got[1], got[3])):
        ref, rw, size, wsize = serve_ref.rope_grad(
            np64(x), None if w is None else np64(w), pos, f, np64(dy), eps=1e-6, **how)
        err, bar = np.abs(np64(dx) - ref), 128 * U * size + half_step(dx.dtype) * np.abs(ref) + 1e-30
        assert (err <= bar).all(), f"dx: max err / bar = {(err / bar).max():.2f}"
        assert (dw is None) == (w is None)
        if w is not None:
            err, bar = np.abs(np64(dw) - rw), (64 + x.shape[0] * x.shape[1]) * U * wsize
            assert (err <= bar).all(), f"dw: max err / bar = {(err / bar).max():.2f}"


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_backward(case):
    q, k, qw, kw, f, ph, how, g = make(case, seed=50)
    dqo, dko = (torch.randn(x.shape, generator=g).to(DEV) for x in (q, k))
    got = ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, q_weight=qw, k_weight=kw, **how)
    check_grads(got, q, k, qw, kw, np.arange(q.shape[0]), f, dqo, dko, **how)
    again = ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, q_weight=qw, k_weight=kw, **how)
    for a, b in zip(got, again):  # a fixed order of additions
        assert a is b or torch.equal(a, b)


def test_gradient_against_differences():
    """The fp32 gradient against central differences of the plain fp64
    forward (h = 1e-4: error near 1e-7 there; 128 u of terms of size 10)."""
    case = (2, 2, 1, 64, 32, False, "f32", True, True, "f32", 1.1)
    q, k, qw, kw, f, ph, how, g = make(case)
    dqo, dko = (torch.randn(x.shape, generator=g).to(DEV) for x in (q, k))
    dq, _, dqw, _ = ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, q_weight=qw, k_weight=kw, **how)
    x, w, dy = np64(q), np64(qw), np64(dqo)

    def loss(x, w):
        return (dy * serve_ref.rope(x, w, np.arange(2), f, eps=1e-6, **how)[0]).sum()

    h = 1e-4
    for i in range(x.size):
        e = np.zeros(x.size)
        e[i] = h
        e = e.reshape(x.shape)
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - np64(dq).flat[i]) < 1e-4
    for i in range(w.size):
        e = np.zeros(w.size)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - np64(dqw)[i]) < 1e-4


@pytest.mark.parametrize("layout, P", [("contiguous", 4), ("zigzag", 4), ("striped", 6)])
def test_ring_layout_positions(layout, P):
    case = (240, 4, 2, 64, 64, False, "f32", True, True, "f32", 1.0)
    q, k, qw, kw, f, ph, how, g = make(case)
    pos = ra.layout_positions(240, P, layout).numpy()
    qo, ko = ra.ra_qk_norm_rope(q, k, ph, q_weight=qw, k_weight=kw, layout=layout, P=P, **how)
    check_rope(qo, q, qw, pos, f, **how)
    check_rope(ko, k, kw, pos, f, **how)
    dqo, dko = (torch.randn(x.shape, generator=g).to(DEV) for x in (q, k))
    got = ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, q_weight=qw, k_weight=kw, layout=layout,
                                      P=P, **how)
    check_grads(got, q, k, qw, kw, pos, f, dqo, dko, **how)


def test_far_and_negative_positions():
    """int32 positions to both ends: the phase product wraps exactly, so far
    positions have the tolerance of near ones.  The fp64 reference's angle is
    off by 2^-53 of 2^31 radians = 2.4e-7 at most, 4 u."""
    case = (6, 2, 1, 128, 128, False, "f32", False, False, "f32", 1.0)
    q, k, _, _, f, ph, how, _ = make(case)
    pos = torch.tensor([0, 1, 1048575, 2**31 - 1, -5, -2**31], dtype=torch.int32, device=DEV)
    qo, ko = ra.ra_qk_norm_rope(q, k, ph, positions=pos, **how)
    check_rope(qo, q, None, pos.cpu().numpy(), f, **how)
    check_rope(ko, k, None, pos.cpu().numpy(), f, **how)


def test_in_place_and_strided_outputs():
    case = (33, 4, 2, 128, 64, False, "bf16", True, True, "f32", 1.0)
    q, k, qw, kw, f, ph, how, g = make(case)
    want = ra.ra_qk_norm_rope(q, k, ph, q_weight=qw, k_weight=kw, **how)
    qc, kc = q.contiguous().clone(), k.contiguous().clone()
    ra.ra_qk_norm_rope(qc, kc, ph, q_weight=qw, k_weight=kw, q_out=qc, k_out=kc, **how)
    assert torch.equal(qc, want[0]) and torch.equal(kc, want[1])
    dqo, dko = (torch.randn(x.shape, generator=g).to(DEV) for x in (q, k))
    ref = ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, q_weight=qw, k_weight=kw, **how)
    packed = torch.full((33, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, q_weight=qw, k_weight=kw, dq=packed[:, :4],
                                dk=packed[:, 4:6], **how)
    assert torch.equal(packed[:, :4], ref[0]) and torch.equal(packed[:, 4:6], ref[1])
    assert (packed[:, 6:] == 7.0).all()


def test_infinity_stays_in_its_column_without_norm():
    """An infinite column that is not rotated must not touch the others, and
    an infinite pair only itself."""
    case = (1, 1, 1, 128, 64, False, "f32", False, False, "f32", 1.0)
    q, k, _, _, f, ph, how, _ = make(case)
    q = q.contiguous().clone()
    q[0, 0, 100] = float("inf")
    qo, _ = ra.ra_qk_norm_rope(q, k, ph, **how)
    assert torch.isinf(qo[0, 0, 100]) and torch.isfinite(qo).sum() == 127


def test_no_rows():
    q = torch.zeros(0, 4, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    qo, ko = ra.ra_qk_norm_rope(q, q, None, q_weight=w)
    assert qo.shape == (0, 4, 64)
    dw = torch.full((64,), 3.0, device=DEV)
    ra.ra_qk_norm_rope_backward(q, q, None, q, q, q_weight=w, dq_weight=dw)
    assert (dw == 0).all()


def test_other_stream_and_captured_backward():
    """Forward and backward captured into a graph and replayed on new inputs
    give what eager calls give; two graphs do not share their scratch."""
    case = (500, 8, 2, 128, 128, False, "bf16", True, True, "f32", 1.0)
    q, k, qw, kw, f, ph, how, g = make(case)
    how.update(q_weight=qw, k_weight=kw)
    dqo, dko = (torch.randn(x.shape, generator=g).to(DEV) for x in (q, k))
    ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, **how)  # the pool exists before a capture
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a = ra.ra_qk_norm_rope(q, k, ph, **how)
            b = ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, **how)
        graphs.append(graph)
        outs.append(a + b)
    q.mul_(0.5)
    dqo.add_(1.0)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for s, graph in zip(streams, graphs):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    want = ra.ra_qk_norm_rope(q, k, ph, **how) + ra.ra_qk_norm_rope_backward(q, k, ph, dqo, dko, **how)
    for out in outs:
        for x, y in zip(out, want):
            assert torch.equal(x, y)


def test_training_step_around_the_ring():
    """norm and rotation -> ring forward -> ring backward -> their gradient,
    in zigzag order, against the plain 64-bit chain (which takes the GPU's
    own rotated bf16 q and k, so the ring's tested bar applies between)."""
    import oracle
    from parity import check_grad, check_output

    N, P, H, Hkv, d = 256, 2, 4, 2, 64
    q0, k0, v = inputs.make_random(N, H, Hkv, d, seed=5)
    g = inputs.randn_chunked((N, H, d), 5, 3).to(torch.bfloat16)
    qw, kw = (1 + 0.2 * inputs.randn_chunked((d,), 6, i) for i in (0, 1))
    f = ra.rope_freqs(64)[0]
    ph = ra.rope_phases(f).to(DEV)
    how = dict(q_weight=qw.to(DEV), k_weight=kw.to(DEV), layout="zigzag", P=P)
    qd, kd, vd, gd = (t.to(DEV) for t in (q0, k0, v, g))
    q, k = ra.ra_qk_norm_rope(qd, kd, ph, **how)
    out, lse = ra.ra_ring_forward_masked(q, k, vd, P=P, layout="zigzag", causal=True)
    dq, dk, dv = ra.ra_ring_backward_masked(q, k, vd, out, lse, gd, P=P, layout="zigzag", causal=True)
    got = ra.ra_qk_norm_rope_backward(qd, kd, ph, dq, dk, **how)
    ra.ra_device_status()
    pos = ra.layout_positions(N, P, "zigzag").numpy()
    check_rope(q, q0, qw, pos, f.numpy())
    kwpos = dict(causal=True, q_pos=pos, k_pos=pos)
    check_output(out, lse, *oracle.attention(q.cpu(), k.cpu(), v, **kwpos), "bf16")
    refs, scales, _ = oracle.backward_with_scales(q.cpu(), k.cpu(), v, g, **kwpos)
    for x, r, s in zip((dq, dk, dv), refs, scales):
        check_grad(x, r, s)
    check_grads(got, q0, k0, qw, kw, pos, f.numpy(), dq, dk)
