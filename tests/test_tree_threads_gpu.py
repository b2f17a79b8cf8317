"""Other threads of the interpreter go on while a call waits in its launch, as it
does when the device's queue of launches is full."""
import threading
import time

import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def test_a_waiting_launch_leaves_other_threads_free():
    parents, cu_q, cu_k = i32([-1, 0, 0, 1]), i32([0, 4]), i32([0, 40])
    msa.msa_tree_mask(parents, cu_q, cu_k, 4)
    torch.cuda.synchronize()
    gaps, done = [], threading.Event()

    def watch():
        last = time.monotonic()
        while not done.is_set():
            time.sleep(0.001)
            now = time.monotonic()
            gaps.append(now - last)
            last = now

    thread = threading.Thread(target=watch)
    thread.start()
    longest = 0.0
    try:
        torch.cuda._sleep(1_500_000_000)  # about a second of the device
        for _ in range(4000):
            at = time.monotonic()
            msa.msa_tree_mask(parents, cu_q, cu_k, 4)
            longest = max(longest, time.monotonic() - at)
    finally:
        done.set()
        thread.join()
    torch.cuda.synchronize()
    if longest < 0.3:
        pytest.skip("no launch waited")
    assert max(gaps) < longest / 2, (max(gaps), longest)
