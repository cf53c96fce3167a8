"""The serving and rotary calls at their edges.

u = 2^-24 throughout (half a step of fp32, relative).
"""
import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import serve_ref
from blockwise_online_softmax_gb300 import binding
from test_gpu_rope import np64

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
