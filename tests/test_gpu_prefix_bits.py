"""What is kept of the weights over a shared prefix: 24 bits with an fp32 output,
2^-17 of each with a bf16 one, where rounding to one bf16 term would leave 2^-9."""
import math

import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import fp8_ref
from test_gpu_prefix import DEV, U, make
from test_gpu_rope import np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_that_cancel(d, room):
    """Half of the keys have a weight exp(-a / sqrt d) and a value of 1, half exp(-b /
    sqrt d) and -1, and a prefix's last key, the largest score, a value of 0: the
    output, half the difference of two weights near each other, shows what is lost
    of a weight as the bf16 rounding of a larger output would not.  Scores are one
    product each: a weight is off by 6.4 u (as in test_gpu_prefix.py's test of 24
    bits), sums of n terms by n u on either side of the fraction, and the terms by
    2^-24 or 2^-17."""
    n, ps, H, Hkv = 301, 16, 8, 2
    args, ks, vs = make([(n, [1] * 40)], [1] * 40, H, Hkv, d, ps, room=room)
    q, kc, vc, ptab, _, _, table, _ = args
    q.zero_()
    q[:, :, 0] = 1.0
    # Two scores near each other whose weights one term would round apart.
    grid = torch.arange(0.25, 1.0, 2.0 ** -8).double().numpy()
    w = np.exp(-grid / math.sqrt(d))
    lost = torch.from_numpy(w).bfloat16().double().numpy() / w - 1
    i, j = np.unravel_index((lost[:, None] - lost - 2.0 ** -6 * np.abs(w[:, None] - w)).argmax(), (len(w), len(w)))
    a, b = grid[i], grid[j]
    k = torch.zeros(n, Hkv, d)
    v = torch.zeros(n, Hkv, d)
    k[0::2, :, 0], v[0::2] = -a, 1.0
    k[1::2, :, 0], v[1::2] = -b, -1.0
    k[n - 1], v[n - 1] = 0.0, 0.0
    k, v = k.bfloat16(), v.bfloat16()
    for t in range(n):
        kc[int(ptab[0, t // ps]), t % ps] = k[t].to(DEV)
        vc[int(ptab[0, t // ps]), t % ps] = v[t].to(DEV)
    own_k, own_v = torch.full((1, Hkv, d), -1.0), torch.zeros(1, Hkv, d)
    for r in range(40):
        kc[int(table[r, 0]), 0] = own_k.bfloat16().to(DEV)
        vc[int(table[r, 0]), 0] = own_v.bfloat16().to(DEV)
    kd = np.concatenate((np64(k), np64(own_k)))
    vd = np.concatenate((np64(v), np64(own_v)))
    want, _, size = fp8_ref.attention(np64(q[:1]), kd, vd)
    sums = (2 * 6.4 + 2 * (n + 1)) * U
    bar = (sums + 2.0 ** -17) * size + 2.0 ** -8 * np.abs(want)
    assert (0.4 * (lost[i] - lost[j]) * size > 2 * bar).all()  # one term would show
    out, _ = ra.ra_paged_decode_prefix(*args)
    bf, _ = ra.ra_paged_decode_prefix(*args, out=torch.empty(q.shape, dtype=torch.bfloat16, device=DEV))
    ra.ra_device_status()
    assert (np.abs(np64(out) - want) <= (sums + 2.0 ** -24) * size).all()
    assert (np.abs(np64(bf) - want) <= bar).all()
