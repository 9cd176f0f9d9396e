"""Other Python threads run while a call waits for room in the stream's queue
(a launch waits once about a thousand are ahead of it)."""

import threading
import time

import pytest
import torch

from tests import serving_cases as sc

pytestmark = pytest.mark.gpu


def test_a_waiting_call_lets_other_threads_run(lib):
    x = sc.to_cuda(sc.layer_inputs([1, 1], 2, 4, 128, True, seed=1), True)
    a = {n: v if v is None else torch.from_numpy(v).cuda() for n, v in sc.accept_inputs(2, 4, 50, seed=1).items()}
    layer = [x[n] for n in ("q", "k", "v", "g", "beta")]
    ws = lib.prefill_workspace(2, 2, 4, 128)
    o, S = torch.empty(2, 4, 128, device="cuda"), torch.empty_like(x["S0"])
    calls = {"step": lambda: lib.step(*layer, x["S0"], out=o, S_out=S),
             "prefill": lambda: lib.prefill(*layer, x["S0"], x["starts"], ws, out=o, S_out=S),
             "accept": lambda: lib.accept(a["p"], a["tokens"], a["parent"], a["u"], a["noise"], q=a["q"])}
    for name, call in calls.items():
        call()
        torch.cuda.synchronize()
        longest, done = 0.0, threading.Event()

        def tick():
            nonlocal longest
            last = time.perf_counter()
            while not done.is_set():
                time.sleep(0.001)
                now = time.perf_counter()
                longest, last = max(longest, now - last), now

        thread = threading.Thread(target=tick)
        thread.start()
        time.sleep(0.01)
        start = time.perf_counter()
        torch.cuda._sleep(1_500_000_000)  # some 0.8 s on the GPU
        for _ in range(3000):
            call()
        waited = time.perf_counter() - start
        done.set()
        thread.join()
        torch.cuda.synchronize()
        assert waited > 0.5, "no call had to wait"
        assert longest < 0.25, (name, longest)
