"""The first call of a thread, with everything passed in: nothing in it has made the
device's context the thread's own yet."""
import threading

import pytest
import torch

import blockwise_online_softmax_gb300 as ra
import test_gpu_fp8_decode as fp8
import test_gpu_prefix as prefix

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ring():
    q = torch.randn(256, 4, 64, device=DEV).bfloat16()
    return lambda **kw: ra.ra_ring_forward(q, q, q, P=2, causal=True, **kw), (256, 4, 64)


def split():
    q, k = (torch.randn(n, 4, 64, device=DEV).bfloat16() for n in (2, 500))
    return lambda **kw: ra.ra_decode_forward(q, k, k, P=2, **kw), (2, 4, 64)


def paged():
    q, kc, vc, table, lens, _, _ = prefix.make_decode([70, 5], [1, 1], 4, 2, 64, 16)
    return lambda **kw: ra.ra_paged_decode(q, kc, vc, table, lens, **kw), q.shape


def shared(room):
    args, _, _ = prefix.make([(300, [3] * 20)], [1] * 20, 4, 2, 64, 16, room=room)
    return lambda **kw: ra.ra_paged_decode_prefix(*args, **kw), args[0].shape


def codes():
    q, pages, table, lens, _, _ = fp8.make8([70, 5], [1, 1], 4, 2, 64, 16)
    return lambda **kw: ra.ra_paged_decode_fp8(q, *pages, table, lens, **kw), q.shape


@pytest.mark.parametrize("make", [ring, split, paged, lambda: shared(False), lambda: shared(True), codes])
def test_first_call_of_a_thread(make):
    run, shape = make()
    want = run()
    out, lse = torch.empty(shape, device=DEV), torch.empty(shape[:2], device=DEV)
    stream = torch.cuda.Stream().cuda_stream
    torch.cuda.synchronize()
    raised = []

    def work():
        try:
            run(out=out, lse=lse, stream=stream)
        except Exception as e:  # noqa: BLE001
            raised.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not raised, raised[0]
    torch.cuda.synchronize()
    ra.ra_device_status()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
