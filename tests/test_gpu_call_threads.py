"""The native calls beside other Python threads, streams and devices."""
import threading
import time

import pytest
import torch

from trellis_quantized_moe_exl3_gb300 import (PagedBatch, PagedKVCache, PagePool, kv_append, paged_attention,
                                               verify_drafts)

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def calls():
    """Each native operator as a call without arguments."""
    pool = PagePool(9, 16, 2, 4)
    seqs, q = ints([1, 0]), ints([1, 1])
    cache = PagedKVCache(*[torch.zeros(9, 16, 1, 64, dtype=BF, device="cuda") for _ in range(2)])
    batch = PagedBatch(ints([0, 1, 2]), ints([5, 9]), ints([[0], [1]]), 1)
    x = torch.randn(2, 1, 64, device="cuda").to(BF)
    p, u = torch.full((2, 8), 0.125, device="cuda"), torch.zeros(2, device="cuda")
    none, cu = ints([]), ints([0, 0, 0])
    return {"extend": lambda: pool.extend(seqs, q, 1, 2), "trim": lambda: pool.trim(seqs, q),
            "append": lambda: kv_append(cache, batch, x, x, q=x),
            "attention": lambda: paged_attention(x, cache, batch),
            "verify": lambda: verify_drafts(p, none, cu, u[:0], u)}


@pytest.mark.parametrize("name", ["extend", "trim", "append", "attention", "verify"])
def test_other_threads_run_while_a_call_waits_for_the_queue(name):
    """A call that waits for room among the launches under way (behind half a second of
    work) leaves the interpreter to other threads."""
    call = calls()[name]
    call()
    torch.cuda.synchronize()
    gaps, stop = [], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    ticker = threading.Thread(target=tick)
    ticker.start()
    try:
        torch.cuda._sleep(1_000_000_000)
        t0 = time.perf_counter()
        for _ in range(3000):
            call()
        took = time.perf_counter() - t0
    finally:
        stop.set()
        ticker.join()
    torch.cuda.synchronize()
    assert took > 0.2, "the queue never filled"
    assert max(gaps) < 0.1, max(gaps)
