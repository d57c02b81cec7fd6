"""Calls from several threads at once, each on a stream of its own, of sizes that
want different amounts of shared memory of one kernel."""
import threading

import pytest
import torch

from test_gpu_route import gen, make_logits, status

import route_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [(2048, 1552, 1792), (2048, 1040, 1400)])
def test_threads_with_different_numbers_of_experts(sizes):
    from gpu_path import B
    B.library()
    T, K, calls = 8, 4, 2000
    errors, results = [], {}
    inputs = {E: make_logits(gen(E), T, E, "fp32").contiguous() for E in sizes}
    start = threading.Barrier(len(sizes))

    def work(E):
        try:
            l = inputs[E]
            idx, w = torch.empty((T, K), dtype=torch.int64, device="cuda"), torch.empty((T, K), device="cuda")
            loss, load = torch.empty(1, device="cuda"), torch.empty((1, E), device="cuda")
            ws = torch.empty(B.ep_balance_loss_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
            st, stream = status(), torch.cuda.Stream()
            torch.cuda.synchronize()
            start.wait()
            for _ in range(calls):
                B.ep_route(l, idx, w, st, score=B.EP_SCORE_SIGMOID, num_groups=8, topk_groups=4, stream=stream)
                B.ep_balance_loss(l, idx, ws, loss, load, st, score=B.EP_SCORE_SIGMOID, stream=stream)
            stream.synchronize()
            results[E] = (idx, loss, int(st.item()))
        except Exception as e:      # noqa: BLE001
            errors.append((E, repr(e)))

    threads = [threading.Thread(target=work, args=(E,)) for E in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for E in sizes:
        idx, loss, st = results[E]
        want = ref.route(inputs[E], K, "sigmoid", groups=8, topk_groups=4)[0]
        assert st == 0 and torch.equal(idx, want)
        want_loss, _, _ = ref.balance(inputs[E], idx, "sigmoid")
        assert abs(float(loss) - float(want_loss)) <= 1e-4 * float(want_loss)
