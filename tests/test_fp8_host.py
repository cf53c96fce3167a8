"""Pages in 8 bits without a GPU: refusals of the C ABI and of the binding
(every check runs before any CUDA call; the pointers are never dereferenced),
and the tests' own quantisation against torch's type."""
import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import fp8_ref
from test_serve_host import FAKE, lib, refused  # noqa: F401

APPEND = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, T=8, d=128,
              heads=4, kv_heads=2, q_stride=512, k_stride=256, v_stride=256, n_pages=10,
              page_size=16, kps=4096, vps=4096, kss=32, vss=32, slots=FAKE, positions=FAKE, rot=64,
              inter=0, phases=FAKE, mscale=1.0, qw=0, kw=0, w_dtype=0, eps=1e-6, dtype=1,
              stream=None)
READ = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, k_out=FAKE, v_out=FAKE, tokens=8, n_req=4, cu=FAKE,
            table=FAKE, max_pages=8, lengths=FAKE, n_pages=10, page_size=16, kps=4096, vps=4096,
            kss=32, vss=32, d=128, kv_heads=2, stream=None)


@pytest.mark.parametrize("change, code, msg", [
    (dict(dtype=0), -2, b"bf16"),
    (dict(page_size=8), -2, b"page_size=8 (pages in 8 bits"),
    (dict(page_size=20), -2, b"page_size"),
    (dict(n_pages=-1), -1, b"n_pages"),
    (dict(kps=4080), -1, b"k_page_stride"),
    (dict(vps=4104), -1, b"v_page_stride"),
    (dict(kss=16), -1, b"k_scale_stride"),
    (dict(vss=40), -1, b"v_scale_stride"),
    (dict(q_stride=504), -1, b"q_stride"),
    (dict(v_stride=128), -1, b"v_stride"),
    (dict(slots=FAKE + 4), -1, b"8-byte"),
    (dict(positions=0), -1, b"NULL"),
    (dict(vs=0), -1, b"NULL"),
    (dict(ks=FAKE + 8), -1, b"aligned"),
    (dict(kc=FAKE + 8), -1, b"aligned"),
])
def test_append_refusals(lib, change, code, msg):  # noqa: F811
    refused(lib, lib.ra_paged_append_fp8(*{**APPEND, **change}.values()), code, msg)


@pytest.mark.parametrize("change, code, msg", [
    (dict(d=96), -2, b"head dim"),
    (dict(kv_heads=0), -1, b"heads"),
    (dict(page_size=8), -2, b"page_size=8 (pages in 8 bits"),
    (dict(n_req=-1), -1, b"n_req"),
    (dict(tokens=-1), -1, b"tokens"),
    (dict(tokens=1 << 31), -1, b"tokens"),
    (dict(n_pages=-2), -1, b"n_pages"),
    (dict(n_req=1 << 16, max_pages=1 << 16), -2, b"n_req * max_pages"),
    (dict(kps=4080), -1, b"k_page_stride"),
    (dict(vss=24), -1, b"v_scale_stride"),
    (dict(k_out=FAKE + 8), -1, b"aligned"),
    (dict(cu=0), -1, b"NULL"),
    (dict(lengths=FAKE + 2), -1, b"4-byte"),
    (dict(vc=0), -1, b"NULL"),
])
def test_read_refusals(lib, change, code, msg):  # noqa: F811
    refused(lib, lib.ra_paged_read_fp8(*{**READ, **change}.values()), code, msg)


def test_empty_calls_are_no_ops(lib):  # noqa: F811
    assert lib.ra_paged_append_fp8(*{**APPEND, "T": 0, "q": 0, "slots": 0}.values()) == 0
    assert lib.ra_paged_read_fp8(*{**READ, "tokens": 0, "k_out": 0}.values()) == 0
    assert lib.ra_paged_read_fp8(*{**READ, "n_req": 0, "cu": 0}.values()) == 0


def test_binding_refusals():
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 16, 1, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(2, 1, 16, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="v must match"):
        ra.ra_paged_append_fp8(q, k, q, None, c, c, s, s, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_paged_append_fp8(q, k, k, None, c, c, s, s, i, i)
    with pytest.raises(ValueError, match="k_cache"):
        ra.ra_paged_read_fp8(c[0], c, s, s, i.view(3, 1), i, i, tokens=4)
    with pytest.raises(ValueError, match="negative"):
        ra.ra_paged_read_fp8(c, c, s, s, i.view(3, 1), i, i, tokens=-1)
    with pytest.raises(ValueError, match="v_out must have shape"):
        ra.ra_paged_read_fp8(c, c, s, s, i.view(3, 1), i, i, tokens=4, v_out=k[:3])


def test_the_plain_quantisation_is_the_types():
    """Code values and rounding as torch's e4m3 has them (its cast rounds
    halves to even); scaling by a power of two is exact."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(fp8_ref.code_values(), codes)
    rng = np.random.default_rng(0)
    x = (rng.normal(size=(4000, 64)) * 2.0 ** rng.integers(-30, 30, (4000, 1))).astype(np.float32)
    x[::7] = np.float32(1.0) * (rng.integers(-64, 65, x[::7].shape) / 32)  # halves
    x[5] = 0
    val, e = fp8_ref.quantise(x)
    y = torch.from_numpy(x).double() / torch.from_numpy(2.0 ** e.astype(np.float64))[:, None]
    assert float(y.abs().max()) <= 448 and (y.abs().amax(1) > 224)[np.arange(4000) != 5][:4].all()
    np.testing.assert_array_equal(val, y.float().to(torch.float8_e4m3fn).double().numpy())
    assert e[5] == -117


DECODE = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, out=FAKE, lse=FAKE, T=8, n_req=4, n_q=2,
              cu_q=0, table=FAKE, max_pages=8, lengths=FAKE, n_pages=10, page_size=16, kps=4096,
              vps=4096, kss=32, vss=32, window=0, d=128, heads=4, kv_heads=2, dtype=1, out_dtype=0,
              stream=None)


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
    (dict(page_size=8), -2, b"page_size=8 (pages in 8 bits"),
    (dict(kps=4095), -1, b"k_page_stride"),
    (dict(vss=16), -1, b"v_scale_stride"),
    (dict(cu_q=FAKE + 1), -1, b"cu_q"),
    (dict(table=0), -1, b"NULL"),
    (dict(q=FAKE + 8), -1, b"aligned"),
    (dict(ks=FAKE + 4), -1, b"aligned"),
])
def test_decode_refusals(lib, change, code, msg):  # noqa: F811
    refused(lib, lib.ra_paged_decode_fp8(*{**DECODE, **change}.values()), code, msg)


def test_empty_decode_is_a_no_op(lib):  # noqa: F811
    assert lib.ra_paged_decode_fp8(*{**DECODE, "T": 0, "n_req": 0, "n_q": 0, "q": 0}.values()) == 0
    assert lib.ra_paged_decode_fp8(*{**DECODE, "T": 0, "cu_q": FAKE, "ks": 0}.values()) == 0


def test_two_halves_hold_a_weight():
    """The weight's two fp16 terms, as the decode forms them: what they leave is
    at most 2^-23 of it where the first is in fp16's normal range, else 2^-25
    absolute, of weights scaled to at most 2^15."""
    rng = np.random.default_rng(2)
    w = (rng.uniform(1, 2, 200000) * 2.0 ** rng.integers(-30, 15, 200000)).astype(np.float32)
    hi = w.astype(np.float16).astype(np.float32)
    lo = (w - hi).astype(np.float16).astype(np.float32)
    left = np.abs(w.astype(np.float64) - hi - lo)
    assert (left <= np.maximum(2.0 ** -23 * w, 2.0 ** -25)).all()
    assert np.abs(w - hi).max() > 2.0 ** -13 * 2.0 ** 14  # one term alone does not
