"""The serving calls without a GPU: refusals of the C ABI and of the binding
(every check runs before any CUDA call; the pointers are never dereferenced),
the rotary tables, and the tests' own plain gradient against differences."""
import math

import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import serve_ref
from blockwise_online_softmax_gb300 import binding

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from blockwise_online_softmax_gb300 import build

    build.build()
    return binding.lib()


def refused(lib, rc, code, msg):
    assert rc == code, (rc, lib.ra_last_error())
    assert msg in lib.ra_last_error(), lib.ra_last_error()


ROPE = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, T=8, d=128, heads=4, kv_heads=2, q_stride=512,
            k_stride=256, positions=0, layout=0, P=1, rot_dim=128, interleaved=0, phases=FAKE,
            mscale=1.0, q_weight=0, k_weight=0, w_dtype=0, eps=1e-6, dtype=1, stream=None)


@pytest.mark.parametrize("change, code, msg", [
    (dict(d=96), -2, b"head dim"),
    (dict(heads=3), -1, b"multiple of kv_heads"),
    (dict(dtype=5), -1, b"dtype"),
    (dict(T=-1), -1, b"T=-1"),
    (dict(T=7, P=2), -1, b"multiple of P"),
    (dict(P=0), -1, b"P=0"),
    (dict(T=6, P=2, layout=1), -1, b"odd"),
    (dict(layout=3), -1, b"layout"),
    (dict(rot_dim=136), -2, b"rot_dim"),
    (dict(rot_dim=24), -2, b"rot_dim"),
    (dict(rot_dim=-16), -2, b"rot_dim"),
    (dict(interleaved=2), -1, b"interleaved"),
    (dict(phases=0), -1, b"NULL"),
    (dict(phases=FAKE + 4), -1, b"8-byte"),
    (dict(positions=FAKE + 2), -1, b"positions"),
    (dict(w_dtype=9), -1, b"w_dtype"),
    (dict(q_weight=FAKE + 4), -1, b"weight"),
    (dict(eps=-1.0), -1, b"eps"),
    (dict(eps=float("nan")), -1, b"eps"),
    (dict(mscale=float("inf")), -1, b"mscale"),
    (dict(q_stride=504), -1, b"q_stride"),
    (dict(k_stride=260), -1, b"k_stride"),
    (dict(q=0), -1, b"NULL"),
    (dict(k_out=FAKE + 8), -1, b"aligned"),
])
def test_rope_refusals(lib, change, code, msg):
    refused(lib, lib.ra_qk_norm_rope(*{**ROPE, **change}.values()), code, msg)


def test_rope_of_no_rows_is_a_no_op(lib):
    assert lib.ra_qk_norm_rope(*{**ROPE, "T": 0, "q": 0, "q_out": 0}.values()) == 0


def rope_backward(lib, **change):
    a = dict(q=FAKE, k=FAKE, dqo=FAKE, dko=FAKE, dq=FAKE, dk=FAKE, dqw=0, dkw=0, T=8, d=128,
             heads=4, kv_heads=2, q_stride=512, k_stride=256, dq_stride=512, dk_stride=256,
             positions=0, layout=0, P=1, rot=128, inter=0, phases=FAKE, mscale=1.0, qw=0, kw=0,
             w_dtype=0, eps=1e-6, dtype=1, stream=None)
    return lib.ra_qk_norm_rope_backward(*{**a, **change}.values())


@pytest.mark.parametrize("change, code, msg", [
    (dict(qw=FAKE), -1, b"together"),
    (dict(dkw=FAKE), -1, b"together"),
    (dict(qw=FAKE, dqw=FAKE + 4), -1, b"weight gradient"),
    (dict(dq_stride=256), -1, b"dq_stride"),
    (dict(dk_stride=257), -1, b"dk_stride"),
    (dict(dqo=0), -1, b"NULL"),
])
def test_rope_backward_refusals(lib, change, code, msg):
    refused(lib, rope_backward(lib, **change), code, msg)


EXTEND = dict(lengths=FAKE, new_tokens=FAKE, n_req=4, table=FAKE, max_pages=8, free=FAKE,
              capacity=32, count=FAKE, page_size=16, tokens=4, lengths_out=FAKE, count_out=FAKE,
              slots=FAKE, positions=FAKE, cu=FAKE, status=FAKE, stream=None)


@pytest.mark.parametrize("change, code, msg", [
    (dict(page_size=12), -2, b"page_size"),
    (dict(page_size=4), -2, b"page_size"),
    (dict(page_size=512), -2, b"page_size"),
    (dict(n_req=-1), -1, b"n_req"),
    (dict(max_pages=0), -1, b"max_pages"),
    (dict(n_req=1 << 16, max_pages=1 << 16), -2, b"n_req * max_pages"),
    (dict(n_req=1, max_pages=1 << 28), -2, b"max_pages * page_size"),
    (dict(capacity=-1), -1, b"free_capacity"),
    (dict(tokens=-1), -1, b"tokens"),
    (dict(tokens=1 << 31), -1, b"tokens"),
    (dict(status=0), -1, b"NULL"),
    (dict(cu=FAKE + 2), -1, b"4-byte"),
    (dict(slots=FAKE + 4), -1, b"8-byte"),
    (dict(lengths=0), -1, b"NULL"),
])
def test_extend_refusals(lib, change, code, msg):
    refused(lib, lib.ra_paged_extend(*{**EXTEND, **change}.values()), code, msg)


def test_release_refusals(lib):
    def call(page_size=16, free=FAKE, finished=FAKE, capacity=32):
        return lib.ra_paged_release(FAKE, finished, 4, FAKE, 8, free, capacity, FAKE, page_size,
                                    FAKE, FAKE, None)

    refused(lib, call(page_size=0), -2, b"page_size")
    refused(lib, call(free=0), -1, b"NULL")
    refused(lib, call(finished=0), -1, b"NULL")
    refused(lib, call(capacity=-2), -1, b"free_capacity")


def append(lib, **change):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, kc=FAKE, vc=FAKE, T=8, d=128, heads=4, kv_heads=2,
             q_stride=512, k_stride=256, v_stride=256, n_pages=10, page_size=16, kps=4096,
             vps=4096, slots=FAKE, positions=FAKE, rot=64, inter=0, phases=FAKE, mscale=1.0, qw=0,
             kw=0, w_dtype=0, eps=1e-6, dtype=1, stream=None)
    return lib.ra_paged_append(*{**a, **change}.values())


@pytest.mark.parametrize("change, code, msg", [
    (dict(dtype=0), -2, b"bf16"),
    (dict(page_size=20), -2, b"page_size"),
    (dict(n_pages=-1), -1, b"n_pages"),
    (dict(kps=4088), -1, b"k_page_stride"),
    (dict(vps=4100), -1, b"v_page_stride"),
    (dict(v_stride=128), -1, b"v_stride"),
    (dict(slots=FAKE + 4), -1, b"8-byte"),
    (dict(positions=0), -1, b"NULL"),
    (dict(vc=0), -1, b"NULL"),
])
def test_append_refusals(lib, change, code, msg):
    refused(lib, append(lib, **change), code, msg)


def decode(lib, **change):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, out=FAKE, lse=FAKE, T=8, n_req=4, n_q=2, cu_q=0, table=FAKE,
             max_pages=8, lengths=FAKE, n_pages=10, page_size=16, kps=4096, vps=4096, window=0,
             d=128, heads=4, kv_heads=2, dtype=1, out_dtype=0, stream=None)
    return lib.ra_paged_decode(*{**a, **change}.values())


@pytest.mark.parametrize("change, code, msg", [
    (dict(dtype=0), -2, b"bf16"),
    (dict(out_dtype=2), -1, b"out_dtype"),
    (dict(d=80), -2, b"head dim"),
    (dict(heads=5), -1, b"multiple of kv_heads"),
    (dict(heads=258, kv_heads=2), -2, b"exceeds 128"),
    (dict(T=7), -1, b"n_req * n_q"),
    (dict(n_q=-1), -1, b"n_q"),
    (dict(T=1 << 30, n_req=1 << 29, max_pages=1), -2, b"T * heads"),
    (dict(window=-1), -1, b"window"),
    (dict(kps=4095), -1, b"k_page_stride"),
    (dict(cu_q=FAKE + 1), -1, b"cu_q"),
    (dict(table=0), -1, b"NULL"),
    (dict(q=FAKE + 8), -1, b"aligned"),
])
def test_decode_refusals(lib, change, code, msg):
    refused(lib, decode(lib, **change), code, msg)


def test_empty_steps_are_no_ops(lib):
    assert decode(lib, T=0, n_req=0, n_q=0, q=0, table=0) == 0
    assert decode(lib, T=0, cu_q=FAKE, q=0) == 0
    assert append(lib, T=0, q=0, slots=0) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    q, k = torch.zeros(4, 2, 64), torch.zeros(4, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_qk_norm_rope(q, k, None)
    with pytest.raises(ValueError, match="share"):
        ra.ra_qk_norm_rope(q, k[:3], None)
    with pytest.raises(ValueError, match="q_out"):
        ra.ra_qk_norm_rope(q, k, None, q_out=q[:2])
    with pytest.raises(ValueError, match="dq_out"):
        ra.ra_qk_norm_rope_backward(q, k, None, q[:2], k)
    with pytest.raises(ValueError, match="without its weight"):
        ra.ra_qk_norm_rope_backward(q, k, None, q, k, dq_weight=torch.zeros(64))
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_table"):
        ra.ra_paged_extend(i, i, i.view(1, 3), i, i[:1], page_size=16, tokens=3)
    cache = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="multiple of 3"):
        ra.ra_paged_decode(q.bfloat16(), cache, cache, i.view(3, 1), i)
    with pytest.raises(ValueError, match="v must match"):
        ra.ra_paged_append(q, k, q, None, cache, cache, i, i)


# ------------------------------------------------------------------ rotary tables

@pytest.mark.parametrize("rot, base", [(128, 10000.0), (64, 500000.0), (16, 1e7)])
def test_phases_hold_the_angles(rot, base):
    """The table's angle at a position, as the kernel forms it, against
    pos * f in extended integers: the table truncates to 2^-64 turns."""
    f, m = ra.rope_freqs(rot, base)
    assert m == 1.0 and f.dtype == torch.float64 and f.shape == (rot // 2,)
    ph = ra.rope_phases(f)
    assert ph.dtype == torch.int64
    for pos in (1, 4097, 1048575, 2**31 - 1):
        got = (pos * ph.numpy().astype(object)) % 2**64
        want = np.array([(pos * int(x * 2**80)) % 2**80 for x in (f / (2 * math.pi)).tolist()],
                        dtype=object)
        err = np.array([min((int(g) * 2**16 - w) % 2**80, (w - int(g) * 2**16) % 2**80)
                        for g, w in zip(got, want)], dtype=object)
        assert max(err) <= pos * 2**17  # turns in units of 2^-80: a unit of 2^-64 per position


def test_scaled_frequencies():
    f, _ = ra.rope_freqs(64, 10000.0)
    lin, m = ra.rope_freqs(64, 10000.0, scaling="linear", factor=4.0)
    assert torch.allclose(lin * 4, f, rtol=1e-15) and m == 1.0
    ntk, m = ra.rope_freqs(64, 10000.0, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and torch.allclose(ntk[-1] * 4, f[-1], rtol=1e-12) and m == 1.0
    yarn, m = ra.rope_freqs(64, 10000.0, scaling="yarn", factor=4.0)
    assert m == pytest.approx(0.1 * math.log(4.0) + 1.0)
    ratio = f / yarn
    assert ratio[0] == 1.0 and ratio[-1] == pytest.approx(4.0)
    assert (ratio.diff() >= -1e-12).all()
    one, m = ra.rope_freqs(64, 10000.0, scaling="yarn", factor=1.0)
    assert torch.allclose(one, f, rtol=1e-15) and m == 1.0
    for bad in (dict(scaling="other"), dict(factor=0.5)):
        with pytest.raises(ValueError):
            ra.rope_freqs(64, **bad)
    with pytest.raises(ValueError):
        ra.rope_freqs(15)


@pytest.mark.parametrize("inter", [False, True])
def test_plain_gradient_against_differences(inter):
    """Central differences of the plain forward in fp64: their error is of
    order h^2 = 1e-8 relative to second differences, plus 1e-16 / h."""
    rng = np.random.default_rng(3)
    x, dy = rng.normal(size=(2, 2, 64)), rng.normal(size=(2, 2, 64))
    w = 1 + 0.2 * rng.normal(size=64)
    pos, f = np.array([5, 123456]), ra.rope_freqs(32)[0].numpy()
    kw = dict(eps=1e-6, mscale=1.1, interleaved=inter)
    dx, dw, _, _ = serve_ref.rope_grad(x, w, pos, f, dy, **kw)

    def loss(x, w):
        return (dy * serve_ref.rope(x, w, pos, f, **kw)[0]).sum()

    h = 1e-4
    for at in [(0, 0, 0), (0, 1, 17), (1, 0, 33), (1, 1, 63)]:
        e = np.zeros_like(x)
        e[at] = h
        assert (loss(x + e, w) - loss(x - e, w)) / (2 * h) == pytest.approx(dx[at], abs=1e-6)
    for i in (0, 20, 63):
        e = np.zeros_like(w)
        e[i] = h
        assert (loss(x, w + e) - loss(x, w - e)) / (2 * h) == pytest.approx(dw[i], abs=1e-6)
