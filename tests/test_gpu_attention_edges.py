"""Edges of the attention operators: values that are not finite in places that
every row of a unit sees, scales of zero, workspaces, streams, inconsistent
batches.  Tolerances are those of test_gpu_attention.py."""
import math

import pytest
import torch

import _attention_ref as R
from test_gpu_attention import BF, E4, FP, PATHS, check_attention, freqs, gen, setup
from trellis_quantized_moe_exl3_gb300 import (PagedBatch, PagedKVCache, _lib, device_status, kv_append,
                                              paged_attention)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ values that are not finite
def plant(cache, step, page, spots):
    """NaN (infinities too in a 16-bit cache) in V of the given (sequence,
    position) places, a channel of its own for each, in kv head 0."""
    tab = step.table.cpu()
    for i, (b, pos) in enumerate(spots):
        at = (int(tab[b, pos // page]), pos % page, 0, (7 * i + 3) % cache.head_dim)
        if cache.dtype == E4:
            cache.v.view(torch.uint8)[at] = 0x7F
        else:
            cache.v[at] = (math.nan, math.inf, -math.inf)[i % 3]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype,cdt", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)],
                         ids=["bf16", "fp16", "bf16_e4m3", "fp16_e4m3"])
@pytest.mark.parametrize("c,spots", [
    # one token: the last tile is part filled, and every row sees what it holds
    (([1], [300], 16, 4, 1, 128), [(0, 299), (0, 256), (0, 130)]),
    (([1, 2], [70, 513], 32, 8, 2, 64), [(0, 69), (0, 0), (1, 512), (1, 511)]),
    # 65 tokens of 4 heads: a unit of 256 rows and one of 4, of one token
    (([65], [420], 16, 4, 1, 128), [(0, 419), (0, 384), (0, 400), (0, 355)]),
    # every row sees every key
    (([40, 7], [333, 150], 16, 8, 2, 128, False), [(0, 332), (0, 260), (1, 149), (1, 128), (0, 5)]),
    (([70], [200], 48, 4, 4, 64, False), [(0, 199), (0, 129)]),
    # a window that begins inside a tile, seen by one token and by several
    (([1], [500], 16, 4, 1, 128, True, 200), [(0, 299), (0, 300), (0, 303), (0, 499)]),
    (([1, 1], [459, 260], 16, 4, 1, 64, True, 150), [(0, 308), (0, 309), (0, 315), (0, 319), (1, 110), (1, 111)]),
    (([3, 80], [700, 300], 16, 4, 1, 64, True, 130), [(0, 567), (0, 570), (0, 699), (1, 91), (1, 120), (1, 299)]),
], ids=lambda x: f"q{x[0]}_len{x[1]}_d{x[5]}{'_full' if len(x) == 7 else ''}{'_w' if len(x) > 7 else ''}"
    .replace(" ", "") if isinstance(x, tuple) else "")
def test_nonfinite_values_reach_those_that_see_them(c, spots, dtype, cdt, path):
    c = c[:6] + (dtype, cdt) + (c[6:] + (True, 0)[len(c) - 6:])
    cache, step, q = setup(c)
    plant(cache, step, c[2], spots)
    check_attention(cache, step, q, c[2], c[5] ** -0.5, c[8], c[9], path)


# ------------------------------------------------------------ scales
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("ks,vs", [(0.0, 0.02), (-0.02, -0.01), (1e-45, 0.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_zero_and_below(D, ks, vs, dtype, path):
    """A stored x stands for x * scale whatever the scale: with 0 every key a
    token sees weighs the same, and what it does not see weighs nothing."""
    c = ([1, 70, 3], [77, 301, 200], 16, 8, 2, D, dtype, E4, True, 0)
    cache, step, q = setup(c)
    cache.k_scale[0], cache.v_scale[1] = ks, vs
    check_attention(cache, step, q, c[2], D ** -0.5, True, 0, path)


def test_append_with_a_scale_of_zero():
    """A head whose scale is 0 holds zeros (a NaN stays one), not 0 / 0."""
    cache = PagedKVCache(*[torch.zeros(1, 16, 2, 16, dtype=E4, device="cuda") for _ in range(2)],
                         *[torch.tensor([0.0, 0.5], device="cuda") for _ in range(2)])
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    batch = PagedBatch(one, one[1:], one[:1].view(1, 1), 1)
    x = torch.tensor([0.0, 1.0, -2.0, math.inf, math.nan] + [0.5] * 11, dtype=BF, device="cuda")
    x = x.expand(1, 2, 16).contiguous()
    kv_append(cache, batch, x, x)
    for t in (cache.k, cache.v):
        got = t[0, 0].float().cpu()
        assert got[0, :4].tolist() == [0, 0, 0, 0] and math.isnan(got[0, 4]) and not got[0, 5:].any()
        assert got[1, :4].tolist() == [0, 2, -4, 448] and math.isnan(got[1, 4])
        assert bool((got[1, 5:] == 1).all())


# ------------------------------------------------------------ softmax terms
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype,cdt", [(FP, FP), (BF, BF), (FP, E4)], ids=["fp16", "bf16", "fp16_e4m3"])
@pytest.mark.parametrize("n,L,D", [(1, 3000, 64), (70, 1500, 128)])
def test_small_terms_count(n, L, D, dtype, cdt, path):
    """One key outweighs every other one by about 2^25 and its value is 0: the
    output is what the others add.  Terms are rounded to 16 bits: half a step
    of theirs, or in fp16 (below 2^-14) 2^-25, against a largest term that
    stands at 2^7; so an output is off by at most 2^-32 of the values' sum."""
    step, pages = R.make_step(gen(1), [n], [L], 16)
    k = torch.zeros(pages, 16, 1, D, dtype=cdt, device="cuda")
    v = torch.full_like(k, 64.0, dtype=torch.float32).to(cdt)
    at = (int(step.table[0, 0]), 0, 0)
    k[at] = torch.tensor([17.5 if cdt != E4 else 18.0] + [0.0] * (D - 1), device="cuda").to(cdt)
    v[at] = torch.zeros(D, device="cuda").to(cdt)
    q = torch.zeros(n, 2, D, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    batch = PagedBatch(step.cu_q, step.seq_lens, step.table, n)
    got = paged_attention(q, PagedKVCache(k, v), batch, scale=1.0, path=path).double().cpu()
    e = math.exp(-float(k[at][0]))
    others = torch.arange(L - n, L, dtype=torch.float64)[:, None, None]  # keys a token sees but the first
    ref = 64 * others * e / (1 + others * e)
    u = R.U[dtype]
    tol = 2 * u * ref + 1e-4 * ref + 2.0 ** -25 + (64 * others * 2.0 ** -32 if dtype == FP or cdt == E4 else 0)
    assert bool(((got - ref).abs() <= tol).all()), float(((got - ref).abs() / tol).max())


# ------------------------------------------------------------ workspaces and streams
LONG = ([1, 2], [9000, 4000], 32, 16, 1, 128, BF, BF, True, 0)  # units of many parts


def batch_of(step):
    return PagedBatch(step.cu_q, step.seq_lens, step.table, step.max_q)


@pytest.mark.parametrize("path", PATHS)
def test_a_workspace_needs_its_head_zeroed_and_no_more(path):
    """Through the ABI and with ws=: 0xFF everywhere but in the first
    EXL3_ATTENTION_HEAD_BYTES."""
    cache, step, q = setup(LONG, pad=0)
    batch = batch_of(step)
    want, lse = paged_attention(q, cache, batch, return_lse=True, path=path)
    n = cache.workspace_size(3, 16, 2)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:_lib.EXL3_ATTENTION_HEAD_BYTES] = 0
    for _ in range(2):
        got, glse = paged_attention(q, cache, batch, return_lse=True, path=path, ws=ws)
        assert torch.equal(got, want) and torch.equal(glse, lse) and device_status(ws) == 0
    out = torch.full_like(q, 7.0)
    torch.cuda.synchronize()
    assert _lib.lib().exl3_paged_attention(
        cache._ref, batch._ref, q.data_ptr(), q.stride(0), q.stride(1), _lib.EXL3_BF16, 3, 16, 128 ** -0.5,
        1, 0, out.data_ptr(), None, path, ws.data_ptr(), n, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_workspaces_that_are_refused():
    cache, step, q = setup(LONG, pad=0)
    batch = batch_of(step)
    n = cache.workspace_size(3, 16, 2)
    for ws, error in ((torch.zeros(n, dtype=torch.uint8), ValueError),
                      (torch.zeros(n, dtype=torch.float32, device="cuda"), TypeError),
                      (torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2], ValueError),
                      (torch.zeros(n - 1, dtype=torch.uint8, device="cuda"), _lib.Exl3Error)):
        with pytest.raises(error):
            paged_attention(q, cache, batch, ws=ws)


def dirty(*sizes):
    """Blocks of 0xFF that the allocator will hand out next."""
    torch.cuda.empty_cache()
    junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    del junk


def test_first_call_on_another_stream():
    """stream= on a new handle, while the current stream is busy: the workspace
    is zeroed, and the output belongs, where the kernels run."""
    cache, step, q = setup(LONG, pad=0)
    batch = batch_of(step)
    want, wlse = paged_attention(q, cache, batch, return_lse=True, path=1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    dirty(64 << 20, 8 << 20, 4096, q.numel() * 2)
    fresh = PagedKVCache(cache.k, cache.v)
    late = torch.empty_like(q)  # freed while a write to it is still to come
    torch.cuda._sleep(40_000_000)
    late.fill_(5.0)
    del late
    got, lse = paged_attention(q, fresh, batch, return_lse=True, path=1, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(lse, wlse)
    assert fresh.status() == 0


def test_append_on_another_stream():
    cache, step, q = setup(LONG, pad=0)
    batch = batch_of(step)
    k, v = [torch.randn(3, 1, 128, device="cuda").to(BF) for _ in range(2)]
    want = kv_append(cache, batch, k, v, q=q, inv_freq=freqs(128))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    dirty(8 << 20, 8192, 4096, q.numel() * 2)
    fresh = PagedKVCache(cache.k, cache.v)
    late = torch.empty_like(q)
    torch.cuda._sleep(40_000_000)
    late.fill_(5.0)
    del late
    got = kv_append(fresh, batch, k, v, q=q, inv_freq=freqs(128), stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and fresh.status() == 0


@pytest.mark.parametrize("path", PATHS)
def test_one_handle_on_two_streams(path):
    """Calls in flight on two streams do not meet in the handle's workspace."""
    cases = [setup(c, pad=0) for c in (LONG, ([2, 1, 1, 40], [3000, 5000, 12000, 700], 32, 16, 1, 128, BF, BF,
                                              True, 0))]
    cache, n0 = cases[0][0], cases[0][0].k.shape[0]
    # one cache with the pages of both cases
    k, v = [torch.cat([getattr(c[0], x) for c in cases]) for x in "kv"]
    cache = PagedKVCache(k, v)
    cases[1][1].table.add_(n0)
    work = [(q, batch_of(step)) for _, step, q in cases]
    want = [paged_attention(q, cache, b, path=path) for q, b in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, (q, b) in enumerate(work):
            got[i].append(paged_attention(q, cache, b, path=path, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
    assert cache.status() == 0
    assert torch.equal(paged_attention(work[0][0], cache, work[0][1], path=path), want[0])


def test_growth_inside_a_capture_is_refused():
    cache, step, q = setup(LONG, pad=0)
    batch = batch_of(step)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="workspace"):
        with torch.cuda.graph(graph):
            paged_attention(q, cache, batch)
    torch.cuda.synchronize()
    want = paged_attention(q, cache, batch)   # the handle is as good as before
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = paged_attention(q, cache, batch)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and cache.status() == 0


def test_append_captured_first():
    """An append needs no workspace but its status word: a new handle's first
    call may be a captured one."""
    cache, step, q = setup(LONG, pad=0)
    k, v = [torch.randn(3, 1, 128, device="cuda").to(BF) for _ in range(2)]
    batch, f = batch_of(step), freqs(128)
    want = kv_append(cache, batch, k, v, q=q, inv_freq=f)
    fresh = PagedKVCache(torch.zeros_like(cache.k), torch.zeros_like(cache.v))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kv_append(fresh, batch, k, v, q=q, inv_freq=f)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and fresh.status() == 0
    step.table[0, 0] = 1 << 20
    step.table[0, (9000 - 1) // 32] = 1 << 20
    graph.replay()
    graph.replay()
    assert fresh.status() == 1


def test_a_graph_beside_calls_on_the_stream_it_was_warmed_up_on():
    """A replay on one stream and calls on another, both in flight."""
    cache, step, q = setup(LONG, pad=0)
    batch, q2 = batch_of(step), q.flip(0).contiguous()
    want = [paged_attention(x, cache, batch, path=1) for x in (q, q2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = paged_attention(q, cache, batch, path=1)
    paged_attention(q2, cache, batch, path=1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs, got = [], []
    for _ in range(30):
        with torch.cuda.stream(s):
            graph.replay()
            outs.append(out.clone())
        got.append(paged_attention(q2, cache, batch, path=1))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[0]) for g in outs) and all(torch.equal(g, want[1]) for g in got)
    assert cache.status() == 0


def test_a_growing_step_holds_one_workspace():
    """Steps of more and more tokens: the handle does not keep a block for each."""
    k = torch.zeros(64, 16, 2, 64, dtype=BF, device="cuda")
    cache = PagedKVCache(k, k.clone())
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for n in range(8):
        T = 100 << n
        q = torch.zeros(T, 8, 64, dtype=BF, device="cuda")
        cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
        paged_attention(q, cache, PagedBatch(cu, cu[1:], table, 100))
    del q, cu
    need = cache.workspace_size(T, 8, 1)
    assert torch.cuda.memory_allocated() - before <= need + (2 << 20) + 65536


# ------------------------------------------------------------ inconsistent batches
def test_append_of_tokens_outside_the_sequence_found():
    """cu_q that does not ascend: a token whose sequence cannot be told is
    dropped and reported; nothing is read or written past a sequence's end."""
    pages, table = 8, [[0, 1], [2, 3], [4, 5], [6, 7]]
    k, v = [torch.zeros(pages, 16, 1, 16, dtype=BF, device="cuda") for _ in range(2)]
    cache = PagedKVCache(k, v)
    new = (1 + torch.arange(12, device="cuda")).view(12, 1, 1).expand(12, 1, 16).to(BF).contiguous()

    def run(cu, lens):
        k.zero_()
        v.zero_()
        b = PagedBatch(*[torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, lens, table)], 12)
        kv_append(cache, b, new, new)
        bits = cache.status()
        cache.clear_status()
        assert torch.equal(k, v)
        at = k[:, :, 0, 0].flatten().cpu()
        return bits, {int(i): int(at[i]) for i in at.nonzero()[:, 0]}

    # sequences [0, 10), backwards, [2, 3), [3, 12): tokens 0, 1 fall to the
    # first, 2 to the second, 3 to 9 to the third, past its end, the rest to the last
    assert run([0, 10, 2, 3, 12], [10, 5, 32, 31]) == (2, {0: 1, 1: 2, 96 + 29: 11, 96 + 30: 12})
    assert run([0, 0, 9, 1, 12], [0, 31, 32, 32])[0] == 2
    # (ascending, the same tokens find their places)
    assert run([0, 3, 3, 5, 12], [3, 0, 32, 7]) == \
        (0, {0: 1, 1: 2, 2: 3, 64 + 30: 4, 64 + 31: 5, **{96 + i: 6 + i for i in range(7)}})


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("c", [([6, 9], [3, 0], 16, 4, 2, 128, BF, BF), ([300, 2, 40], [299, 1, 500], 16, 24, 8, 128, BF, BF),
                               ([7, 1], [4, 100], 32, 4, 2, 64, BF, E4)], ids=["bf16", "bf16_long", "e4m3"])
def test_the_widest_window_is_none(c, path):
    """A window of 2^31 - 1, with tokens that stand before position 0."""
    cache, step, q = setup(c + (True, 0), pad=0)
    want = paged_attention(q, cache, batch_of(step), return_lse=True, path=path)
    for window in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30 + 1):
        got = paged_attention(q, cache, batch_of(step), return_lse=True, window=window, path=path)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("path", PATHS)
def test_lengths_are_held_to_a_billion(path):
    """A table of 2^31 places of one page, and a length of 2^31 - 1: clamped to
    2^30 and reported; the window at its end is read where it should be."""
    g = gen(3)
    k, v = [torch.randn(1, 4096, 1, 64, generator=g).to(BF).cuda() for _ in range(2)]
    cache = PagedKVCache(k, v)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros(1, 1 << 19, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 4, 64, generator=g).to(BF).cuda()
    near = PagedBatch(ints(0, 1), ints(4096), table, 1)
    want = paged_attention(q, cache, near, window=64, path=path)
    assert cache.status() == 0
    got = paged_attention(q, cache, PagedBatch(ints(0, 1), ints(2 ** 31 - 1), table, 1), window=64, path=path)
    assert cache.status() == 2
    assert torch.equal(got, want)


def test_overlapping_sequences_that_count_past_32_bits():
    """65535 sequences, every other one of all 2^22 tokens of 8 heads (the rest
    run backwards): 2^32 units claimed where the rows make 2^17.  The units past
    those are left out; the first sequence is answered."""
    T, B = 1 << 22, 65535
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = [torch.randn(1, 16, 1, 64, generator=gen(8)).to(BF).cuda() for _ in range(2)]
    cache = PagedKVCache(k, v)
    q = torch.ones(T, 8, 64, dtype=BF, device="cuda")
    q[-16:] = torch.randn(16, 8, 64, generator=gen(9)).to(BF).cuda()
    want = paged_attention(q, cache, PagedBatch(ints(0, T), ints(16), ints([0]), T), path=2)
    assert cache.status() == 0 and not bool(want[:-16].any()) and bool(want[-16:].any())
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    lens, table = torch.full((B,), 16, dtype=torch.int32, device="cuda"), torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    got = paged_attention(q, cache, PagedBatch(cu, lens, table, T), path=2)
    assert cache.status() == 2
    assert torch.equal(got, want)


# ------------------------------------------------------------ bounded waits
@pytest.mark.parametrize("dtype,cdt,D", [(BF, BF, 128), (FP, FP, 64), (BF, E4, 128), (FP, E4, 64)],
                         ids=["bf16_128", "fp16_64", "e4m3_128", "e4m3_64"])
def test_attention_waits_run_out(dtype, cdt, D):
    """Each of the tile kernel's barriers in turn never completes, with a budget
    of 2,000,000 cycles, about 1 ms (nothing that was issued is held back, so
    copies and products end by themselves): the call returns, with status bit 4
    if it waits on that barrier, and once the bit is cleared the next call on
    the workspace is right."""
    c = ([700, 300, 1], [9000, 300, 2000], 64, 8, 2, D, dtype, cdt, True, 0)
    cache, step, q = setup(c, pad=0)
    batch = batch_of(step)
    want = paged_attention(q, cache, batch, path=2)
    assert cache.status() == 0
    L, seen = _lib.lib(), []
    for barrier in range(64):
        assert L.exl3_test_set_attention_wait_fault(barrier, 2_000_000) == 0
        try:
            paged_attention(q, cache, batch, path=2)
            seen.append(cache.status())
        finally:
            assert L.exl3_test_set_attention_wait_fault(-1, 0) == 0
        cache.clear_status()
        assert torch.equal(paged_attention(q, cache, batch, path=2), want) and cache.status() == 0
    # k_full, k_empty, v_full, v_empty; queries, scores, outputs, terms; units
    n = 4 if D == 64 else 2
    assert set(seen) == {0, 4} and all(seen[i] == 4 for i in range(4 * n)), seen
    assert seen.count(4) >= 4 * n + 14 and not any(seen[5 * n + 26:]), seen
