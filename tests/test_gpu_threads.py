"""Host threads that share a stream have workspaces of their own."""
import threading

import pytest
import torch

from test_gpu_varlen import check, make, run
from test_gpu_workspaces import dense_step

pytestmark = pytest.mark.gpu


def test_two_threads_on_one_stream():
    cases = [make("bf16", [1, 1], [9000, 4000], 64, seed=66), make("bf16", [1], [12000], 128, seed=67)]
    steps = [dense_step(cases[0]), lambda: run(cases[1], dev=dev)]
    dev = {k: v.cuda() for k, v in cases[1].items() if isinstance(v, torch.Tensor)}
    torch.cuda.synchronize()
    results, errors = [None, None], []
    gate = threading.Barrier(2)

    def work(i):
        try:
            gate.wait()
            results[i] = [steps[i]() for _ in range(100)]
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for s, res in zip(cases, results):
        check(s, *res[0])
        for o, lse in res[1:]:
            assert torch.equal(o, res[0][0]) and torch.equal(lse, res[0][1])
