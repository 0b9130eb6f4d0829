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
    """A call that waits for room among the launches under way (behind a second of
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
        torch.cuda._sleep(2_000_000_000)
        t0 = time.perf_counter()
        for _ in range(3000):
            call()
        took = time.perf_counter() - t0
    finally:
        stop.set()
        ticker.join()
    torch.cuda.synchronize()
    assert took > 0.6, "the queue never filled"
    assert max(gaps) < 0.3, max(gaps)


def given(g):
    """Calls by name: fresh tensors, and the call on them with stream=."""
    from trellis_quantized_moe_exl3_gb300 import qk_norm_rope
    n = 60000  # (sizes of their own, larger than what small tensors share)

    def cache():
        return PagedKVCache(*[torch.zeros(40, 16, 2, 64, dtype=BF, device="cuda") for _ in range(2)])

    def batch(rows):
        return PagedBatch(ints([0, rows]), ints([rows]), ints([list(range(40))]), rows)

    def x(rows, heads):
        return torch.randn(rows, heads, 64, generator=g, device="cuda").to(BF)

    fixed = cache()
    plain = batch(600)
    w = lambda: 1 + torch.rand(64, generator=g, device="cuda").to(BF)  # noqa: E731
    f = lambda: torch.rand(32, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    pos = lambda: torch.arange(600, dtype=torch.int32, device="cuda")  # noqa: E731
    return {
        "verify": (lambda: [torch.rand(3, n, device="cuda"), ints([1, 2]), ints([0, 2]),
                            torch.rand(2, device="cuda"), torch.rand(1, device="cuda"),
                            torch.rand(2, n, device="cuda")],
                   lambda t, st: verify_drafts(*t[:5], q=t[5], stream=st)),
        "append": (lambda: [x(600, 2), x(600, 2), f(), w(), x(600, 4), w(), x(600, 4), pos()],
                   lambda t, st: kv_append(fixed, plain, t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7],
                                           stream=st)),
        "append to a handle": (lambda: (lambda c, b: [c, b, c.k, c.v, b.cu_q, b.seq_lens, b.block_table])(
                                   cache(), batch(600)),
                               lambda t, st: kv_append(t[0], t[1], kept[0], kept[1], stream=st)),
        "attention": (lambda: [x(600, 4), torch.empty(600, 4, 64, dtype=BF, device="cuda"),
                               torch.zeros(fixed.workspace_size(600, 4, 1), dtype=torch.uint8, device="cuda")],
                      lambda t, st: paged_attention(t[0], fixed, plain, out=t[1], ws=t[2], stream=st)),
        "attention of a handle": (lambda: (lambda c, b: [c, b, c.k, c.v, b.cu_q, b.seq_lens, b.block_table])(
                                      cache(), batch(600)),
                                  lambda t, st: paged_attention(kept[2], t[0], t[1], stream=st)),
        "norm": (lambda: [x(600, 4), x(600, 2), pos(), f(), w(), w()],
                 lambda t, st: qk_norm_rope(*t, stream=st)),
        "extend": (lambda: (lambda p: [p, ints([0, 1]), ints([5, 3]), p.table, p.lens, p.free, p.count])(
                       PagePool(90000, 16, 30, 900)),
                   lambda t, st: t[0].extend(t[1], t[2], 5, 8, stream=st)),
        "trim": (lambda: (lambda p: [p, ints([0, 1]), ints([0, 0]), p.table, p.lens, p.free, p.count])(
                     PagePool(90000, 16, 30, 900)),
                 lambda t, st: t[0].trim(t[1], t[2], stream=st)),
    }


kept = []


@pytest.mark.parametrize("name", ["verify", "append", "append to a handle", "attention",
                                  "attention of a handle", "norm", "extend", "trim"])
def test_tensors_freed_after_a_call_on_another_stream(name):
    """Tensors (a handle's own among them) that the program drops right after a call with
    stream= are not handed out again while that stream has yet to run it."""
    g = torch.Generator(device="cuda").manual_seed(3)
    kept[:] = [torch.randn(600, h, 64, generator=g, device="cuda").to(BF) for h in (2, 2, 4)]
    make, call = given(g)[name]
    side = torch.cuda.Stream()
    call(make(), side)                        # (workspaces made)
    t = make()
    torch.cuda.synchronize()
    tensors = [x for x in t if isinstance(x, torch.Tensor)]
    at = {(x.untyped_storage().data_ptr()): x.untyped_storage().nbytes() for x in tensors}
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)      # half a second before the call's turn
    out = call(t, side)
    del t, tensors
    again = []
    for size in list(at.values()) * 3:
        again.append(torch.empty(size, dtype=torch.uint8, device="cuda"))
    assert not side.query(), "the stream was done too early for the test to say anything"
    taken = {x.data_ptr() for x in again} & set(at)
    torch.cuda.synchronize()
    assert not taken
    del out


class _Elsewhere:
    """A tensor that says it is on the next device."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.t.get_device() + 1


@pytest.mark.parametrize("which", ["k", "positions", "inv_freq", "q_weight", "k_weight", "q_out", "k_out"])
def test_norm_refuses_tensors_of_another_device(which):
    """Before anything is launched (there may be one device only)."""
    from trellis_quantized_moe_exl3_gb300 import _lib, qk_norm_rope
    x = torch.randn(4, 2, 64, device="cuda").to(BF)
    a = dict(q=x, k=x.clone(), positions=torch.arange(4, dtype=torch.int32, device="cuda"),
             inv_freq=torch.ones(32, dtype=torch.float64, device="cuda"),
             q_weight=torch.ones(64, device="cuda").to(BF), k_weight=torch.ones(64, device="cuda").to(BF),
             q_out=torch.empty_like(x), k_out=torch.empty_like(x))
    want = [t.clone() for t in qk_norm_rope(**a)]
    n = _lib.lib().exl3_launch_count()
    with pytest.raises(ValueError, match="another device"):
        qk_norm_rope(**{**a, which: _Elsewhere(a[which])})
    assert _lib.lib().exl3_launch_count() == n
    assert all(torch.equal(g, w) for g, w in zip(qk_norm_rope(**a), want))


def test_norm_makes_its_tensors_device_current(monkeypatch):
    """Where another device is current, the launch is inside a guard of the tensors'."""
    from trellis_quantized_moe_exl3_gb300 import attention, qk_norm_rope
    x = torch.randn(4, 2, 64, device="cuda").to(BF)
    w = torch.ones(64, device="cuda").to(BF)
    want = qk_norm_rope(x, None, q_weight=w)[0]
    entered = []
    real = torch.cuda.device

    class Guard(real):
        def __enter__(self):
            entered.append(self.idx)
            return super().__enter__()

    monkeypatch.setattr(torch.cuda, "device", Guard)
    assert torch.equal(qk_norm_rope(x, None, q_weight=w)[0], want) and not entered
    monkeypatch.setattr(attention, "_current_device", lambda: x.get_device() + 1)
    assert torch.equal(qk_norm_rope(x, None, q_weight=w)[0], want)
    assert entered == [x.get_device()]


class _NoTruth:
    def __bool__(self):
        raise KeyError("neither true nor false")


def test_errors_of_arguments_come_through():
    """What an argument raises when it is looked at is what the caller sees."""
    cache = PagedKVCache(*[torch.zeros(2, 16, 1, 64, dtype=BF, device="cuda") for _ in range(2)])
    batch = PagedBatch(ints([0, 1]), ints([5]), ints([[0, 1]]), 1)
    x = torch.randn(1, 1, 64, device="cuda").to(BF)
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    want = paged_attention(x, cache, batch)
    for kw in (dict(causal=_NoTruth()), dict(return_lse=_NoTruth())):
        with pytest.raises(KeyError):
            paged_attention(x, cache, batch, **kw)
    with pytest.raises(KeyError):
        kv_append(cache, batch, x, x, inv_freq=f, interleaved=_NoTruth())
    for kw in (dict(window="3"), dict(scale="1"), dict(path=None)):
        with pytest.raises(TypeError):
            paged_attention(x, cache, batch, **kw)
    assert torch.equal(paged_attention(x, cache, batch, causal=5, window=0), want)
    assert cache.status() == 0
