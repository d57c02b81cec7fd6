"""The SM-limited dispatch from two threads with rows of different lengths, one call
after the other: the shared memory that one thread's calls ask for is not what
another thread's calls left."""
import threading

import pytest
import torch

from test_gpu_smlimit import _dispatch, _setup

pytestmark = pytest.mark.gpu


def test_dispatch_of_short_rows_by_another_thread_in_between():
    from gpu_path import B
    T, E, K, R = 400, 16, 4, 4
    cases = {H: _setup(T, H, E, K, R, seed=H) for H in (512, 7168)}

    def call(H, num_sms):
        _, idx, w, x, lay = cases[H]
        return _dispatch(B, x, idx, w, E, R, lay, lay.num_recv, H, K, False, num_sms, False)

    def in_a_thread(H):
        failed = []

        def work():
            try:
                call(H, 8)
            except Exception as e:      # noqa: BLE001
                failed.append(repr(e))
        t = threading.Thread(target=work)
        t.start()
        t.join()
        assert not failed, failed

    want = call(7168, 0)
    call(7168, 8)
    in_a_thread(512)
    for got, ok in zip(call(7168, 8), want):
        assert torch.equal(got, ok)
