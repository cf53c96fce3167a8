"""Reading the histories of a few requests of a large batch: the others have no
rows."""
import numpy as np
import pytest
import torch

import blockwise_online_softmax_gb300 as ra
from test_gpu_fp8 import DEV, random_pages

pytestmark = pytest.mark.gpu


def call(rows, lens, hkv, d, ps, seed=0):
    """The newest rows[i] of lens[i] tokens of every request i."""
    rng = np.random.default_rng(seed)
    kc, vc, ks, vs, kx, vx = random_pages(64, ps, hkv, d, seed)
    table = rng.integers(0, 64, (len(rows), -(-max(lens) // ps))).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    dev = [torch.from_numpy(x).to(DEV) for x in (table, np.asarray(lens, dtype=np.int32), cu)]
    outs = [torch.full((int(cu[-1]), hkv, d), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    def run():
        ra.ra_paged_read_fp8(kc, vc, ks, vs, *dev, tokens=int(cu[-1]), k_out=outs[0], v_out=outs[1])

    return run, outs, (kx, vx), table, cu


@pytest.mark.parametrize("hkv, d", [(1, 64), (3, 128)])
@pytest.mark.parametrize("idle", [[0, 1, 2, 3, 4, 5, 6, 7, 8, 9], [31, 32, 33, 1023, 1024, 1025], [2900, 0, 1, 700]])
def test_rows_on_both_sides_of_idle_requests(idle, hkv, d):
    """Requests of 4001 rows, or of one to three, with runs of idle ones before,
    between and behind: so many tokens that a warp takes several rows."""
    rows = []
    for j, n in enumerate(idle):
        rows += [0] * n + [4001, 1, 2, 0, 3]
    rows += [4001] * 3 + [0] * idle[0]
    lens = [n + j % 7 for j, n in enumerate(rows)]
    run, outs, vals, table, cu = call(rows, lens, hkv, d, 16, seed=len(rows))
    run()
    ra.ra_device_status()
    for out, x in zip(outs, vals):
        got = out.double().cpu().numpy()
        for i in np.flatnonzero(rows):
            want = x[table[i]].reshape(-1, hkv, d)[lens[i] - rows[i]:lens[i]]
            np.testing.assert_array_equal(got[cu[i]:cu[i + 1]], want)


def test_idle_requests_cost_a_search_and_not_a_walk():
    """Two histories of 30K tokens with 4998 idle requests between them, against the
    two alone: a walk over the idle ones took 300 us where the rows take 8."""
    times = []
    for between in (0, 4998):
        rows = [30001] + [0] * between + [30001]
        run = call(rows, rows, 1, 64, 16)[0]
        for _ in range(3):
            run()
        best = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                run()
            b.record()
            b.synchronize()
            best.append(a.elapsed_time(b) * 100)  # us a call
        times.append(min(best))
    assert times[1] < 4 * times[0] + 20, f"{times[0]:.1f} us alone, {times[1]:.1f} with idle requests"
