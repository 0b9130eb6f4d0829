"""Pages of a step and verification of drafts on the GPU, against lists and
whole-number arithmetic: every output is a whole number and has to be equal."""
import math

import numpy as np
import pytest
import torch

import _speculate_ref as R
from trellis_quantized_moe_exl3_gb300 import PagePool, verify_drafts

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ pages
def same_state(pool, ref):
    table, lens, free = ref.state()
    assert pool.table.tolist() == table and pool.lens.tolist() == lens
    assert int(pool.count) == len(free) and pool.free[:len(free)].tolist() == free
    assert pool.status() == ref.status


def step_both(pool, ref, seqs, q, max_tokens):
    step = pool.extend(ints(seqs), ints(q), max_q=max(q + [1]), max_tokens=max_tokens)
    cu, lens, table, pos, slots = ref.extend(seqs, q, max_tokens)
    assert step.cu_q.tolist() == cu and step.seq_lens.tolist() == lens
    assert step.block_table.tolist() == table
    assert step.positions.tolist() == pos and step.slots.tolist() == slots
    same_state(pool, ref)


@pytest.mark.parametrize("page,rows,cols,pages,steps", [
    (16, 1, 8, 8, 6), (16, 9, 12, 80, 12), (64, 40, 7, 200, 12), (48, 13, 5, 30, 15),
    (4096, 3, 2, 5, 4),
])
def test_pages_over_many_steps(page, rows, cols, pages, steps):
    """Steps, drops and releases at random, running out of pages on the way."""
    g = np.random.default_rng(page + rows)
    pool, ref = PagePool(pages, page, rows, cols), R.Pool(pages, page, rows, cols)
    for _ in range(steps):
        n = int(g.integers(1, rows + 1))
        seqs = g.permutation(rows)[:n].tolist()
        top = int(g.choice([1, 5, page, 2 * page + 3]))
        q = g.integers(0, top + 1, n).tolist()
        step_both(pool, ref, seqs, q, sum(q) + int(g.integers(0, 9)))
        if g.random() < 0.6:
            drop = [int(g.integers(0, ref.lens[s] + 1)) if g.random() < 0.7 else 0 for s in seqs]
            pool.trim(ints(seqs), ints(drop))
            ref.trim(seqs, drop)
            same_state(pool, ref)
        if g.random() < 0.2:
            gone = seqs[:max(1, n // 2)]
            pool.trim(ints(gone))
            ref.trim(gone)
            same_state(pool, ref)


def test_pages_of_a_step_taken_back():
    """A step taken back whole leaves every bit of the pool."""
    pool = PagePool(500, 16, 64, 40)
    g = gen(3)
    seqs = torch.randperm(64, generator=g)[:50].int().cuda()
    pool.extend(seqs, torch.randint(0, 90, (50,), generator=g).int().cuda(), 90, 5000)
    before = [t.clone() for t in (pool.table, pool.lens, pool.free, pool.count)]
    q = torch.randint(0, 40, (50,), generator=g).int().cuda()
    step = pool.extend(seqs, q, 40, 2000)
    assert int(pool.count) < int(before[3]) and int(step.cu_q[-1]) == int(q.sum())
    pool.trim(seqs, q)
    for t, b in zip((pool.table, pool.lens, pool.free, pool.count), before):
        assert torch.equal(t, b)
    assert pool.status() == 0


def test_pages_refused_on_the_device():
    """Rows out of range, named twice or with a negative count; too few pages;
    too long; rows past max_tokens: each leaves the others' results alone."""
    for q, seqs, max_tokens, pages in [
        ([3, 4, 5], [0, 7, 1], 12, 20),             # row 7 of 4
        ([3, 4, 5], [0, -1, 1], 20, 20),
        ([3, 4, 5, 6], [2, 0, 2, 2], 18, 20),       # the same row three times
        ([3, -4, 5], [0, 1, 2], 8, 20),
        ([20, 40, 1, 16], [0, 1, 2, 3], 77, 4),     # 2 + 3 pages of 4: the second gets none, nor later ones
        ([20, 40, 0, 16], [0, 1, 2, 3], 77, 4),
        ([49, 3], [1, 0], 60, 20),                  # 49 tokens of 48
        ([5, 5, 0, 5], [0, 1, 2, 3], 9, 20),        # rows 5 .. 9 of 9
        ([0, 0], [0, 1], 0, 0),
        ([1], [0], 1, 0),                           # a pool without pages
    ]:
        pool, ref = PagePool(pages, 16, 4, 3), R.Pool(pages, 16, 4, 3)
        step_both(pool, ref, seqs, q, max_tokens)
        step_both(pool, ref, [3, 0], [1, 1], 2)
        pool.clear_status()
        ref.status = 0
        for drop in ([1, 2], [100, 1], [-3, 0]):
            pool.trim(ints([0, 3]), ints(drop))
            ref.trim([0, 3], drop)
            same_state(pool, ref)
        pool.trim(ints([1, 9, 1]))
        ref.trim([1, 9, 1])
        same_state(pool, ref)


def test_pages_of_many_sequences():
    """More sequences than threads of a block; every one twice over the steps."""
    n = 1700
    pool, ref = PagePool(9000, 16, 2000, 6), R.Pool(9000, 16, 2000, 6)
    g = np.random.default_rng(0)
    for top in (30, 9):
        seqs = g.permutation(2000)[:n].tolist()
        q = g.integers(0, top, n).tolist()
        step_both(pool, ref, seqs, q, sum(q) + 3)


def test_pages_of_a_pool_with_many_rows():
    """Claims of more rows than fit shared memory, rows named twice among them."""
    n = 700
    pool, ref = PagePool(2500, 16, 9000, 4), R.Pool(2500, 16, 9000, 4)
    g = np.random.default_rng(4)
    seqs = g.permutation(9000)[:n].tolist()
    seqs[300], seqs[650], seqs[651] = seqs[2], 9000, seqs[2]
    for top in (20, 5):
        q = g.integers(0, top, n).tolist()
        step_both(pool, ref, seqs, q, sum(q))
        drop = [min(1, x) for x in q]
        for i in (300, 650, 651):
            drop[i] = 0
        pool.trim(ints(seqs), ints(drop))
        ref.trim(seqs, drop)
        same_state(pool, ref)


def test_pages_of_a_pool_that_makes_no_sense():
    """Whatever a program has written to the pool, its calls stay inside it."""
    g = gen(1)
    for count, lens, table in ((10 ** 6, 5, 0), (-7, 1 << 30, 99), (4, -5, -1), (1 << 31 - 1, 1 << 30, 1 << 30)):
        pool = PagePool(6, 16, 3, 4)
        pool.count.fill_(min(count, (1 << 31) - 1))
        pool.lens.fill_(lens)
        pool.table.fill_(table)
        pool.free.copy_(torch.randint(-1 << 31, 1 << 31, (6,), generator=g).int())
        for _ in range(3):
            step = pool.extend(ints([0, 1, 2]), ints([30, 1, 0]), 30, 31)
            pool.trim(ints([2, 1, 0]), ints([5, 70, 1]))
            pool.trim(ints([1]))
            assert 0 <= int(pool.count) <= 6
            assert bool((step.seq_lens >= 0).all()) and bool((step.seq_lens <= 64).all())


def test_pages_no_sequences_and_captured_steps():
    pool = PagePool(64, 16, 4, 9)
    step = pool.extend(ints([]), ints([]), 1, 3)
    assert step.cu_q.tolist() == [0] and step.slots.tolist() == [-1] * 3 and step.num_seqs == 0
    pool.trim(ints([]))
    seqs, q, drop = ints([2, 0]), ints([5, 3]), ints([2, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = pool.extend(seqs, q, 8, 8)
        pool.trim(seqs, drop)
    ref = R.Pool(64, 16, 4, 9)
    for k in range(9):
        q.copy_(ints([5 + k % 3, 3 - k % 2]))
        graph.replay()
        cu, lens, table, pos, slots = ref.extend([2, 0], [5 + k % 3, 3 - k % 2], 8)
        assert step.cu_q.tolist() == cu and step.seq_lens.tolist() == lens
        assert step.block_table.tolist() == table and step.slots.tolist() == slots
        ref.trim([2, 0], [2, 1])
        same_state(pool, ref)


# ------------------------------------------------------------ verification
def make_drafts(g, ds, vocab, dtype, given, sharp=2.0, pad=0):
    n = sum(ds)
    logits = torch.randn(n + len(ds) + pad, vocab, generator=g) * sharp
    p = logits.softmax(-1).to(dtype)
    row = [c + j for b, c in enumerate(np.cumsum([0] + [d + 1 for d in ds])[:-1]) for j in range(ds[b])]
    near = (logits[row] + 0.7 * torch.randn(n, vocab, generator=g)).softmax(-1).to(dtype)
    draft = torch.multinomial(near.float(), 1, generator=g)[:, 0].int() if n else torch.zeros(0).int()
    draft = torch.cat([draft, torch.zeros(pad, dtype=torch.int32)])
    near = torch.cat([near, torch.zeros(pad, vocab, dtype=dtype)])
    cu = [0] + np.cumsum(ds).tolist()
    return (p, draft, cu, torch.rand(n + pad, generator=g), torch.rand(len(ds), generator=g),
            near if given else None)


def run_both(p, draft, cu, au, su, q):
    got = verify_drafts(p.cuda(), draft.cuda(), ints(cu), au.cuda(), su.cuda(),
                        q=q.cuda() if q is not None else None)
    want = R.verify(p, draft, cu, au, su, q)
    tail = [-1] * (len(draft) + len(su) - len(want[0]))
    assert got[0].tolist() == want[0] + tail
    assert got[1].tolist() == want[1] and got[2].tolist() == want[2]
    return want


@pytest.mark.parametrize("ds,vocab,dtype,given,pad", [
    ([4], 32000, F32, True, 0), ([0], 100, F32, True, 0), ([1], 1, F32, True, 0),
    ([3, 0, 7, 1], 50001, BF, False, 0), ([5] * 30, 777, FP, True, 2), ([2] * 9, 8191, F32, False, 3),
    ([40, 1, 70], 301, F32, True, 0),                    # more drafts than a warp's lanes
    ([0, 0, 0], 33, BF, True, 0), ([3, 2], 131072, F32, True, 0), ([2, 3], 199999, BF, True, 0),
    ([1] * 200, 64, F32, True, 0), ([1, 2], 1000003, F32, True, 0), ([1], 300001, FP, True, 1),
])
@pytest.mark.parametrize("sharp", [0.5, 4.0])
def test_verify(ds, vocab, dtype, given, pad, sharp):
    run_both(*make_drafts(gen(sum(ds) + vocab), ds, vocab, dtype, given, sharp, pad))


def test_verify_accepts_and_refuses_all():
    g = gen(2)
    p, draft, cu, au, su, q = make_drafts(g, [5, 5, 5], 1000, F32, True)
    same = torch.cat([p[:5], p[6:11], p[12:17]])
    want = run_both(p, draft, cu, au, su, same)          # q = p: all stand
    assert want[1] == [5, 5, 5]
    p[:, :] = 0
    p[:, 7] = 1
    assert run_both(p, draft.fill_(8), cu, au, su, q)[0][0] == 7   # p(x) = 0: none stands
    assert run_both(p, draft.fill_(7), cu, au, su, None)[1] == [5, 5, 5]


def test_verify_borders():
    """Draws on and beside the borders between tokens, ties of the acceptance."""
    v = 512
    p = torch.full((6, v), 1.0 / v)
    q = torch.full((3, v), 2.0 / v)
    q[:, v // 2:] = 0
    draft = torch.tensor([3, 5, v - 1], dtype=torch.int32)
    cu = [0, 1, 2, 3]
    for au in (0.5, 0.5 - 2.0 ** -25, 0.0, 1 - 2.0 ** -24):         # u q = p refuses
        for su in (0.0, 2.0 ** -8, 2.0 ** -8 - 2.0 ** -32, 1 - 2.0 ** -24, 0.5):
            run_both(p, draft, cu, torch.full((3,), au), torch.full((3,), su), q)
            run_both(p, draft, cu, torch.full((3,), au), torch.full((3,), su), None)


def test_verify_rows_without_weight():
    """p <= q everywhere falls back to p; a row of zeros gives -1; NaN and
    negative probabilities count as 0; drafts outside the vocabulary are refused."""
    v = 100
    p, q = torch.full((2, v), 0.25 / v), torch.full((1, v), 1.0 / v)
    one = torch.ones(1)
    want = run_both(p, torch.tensor([4], dtype=torch.int32), [0, 1], 0.9 * one, 0.5 * one, q)
    assert want[0] == [50, -1]
    z = torch.zeros(2, v)
    assert run_both(z, torch.tensor([4], dtype=torch.int32), [0, 1], 0 * one, 0.5 * one, q)[0] == [-1, -1]
    z[0, 9], z[0, 10], z[0, 11] = math.nan, -1.0, 0.5
    assert run_both(z, torch.tensor([4], dtype=torch.int32), [0, 1], 0 * one, 0.5 * one, None)[0] == [11, -1]
    for x in (-1, v, 1 << 30, -(1 << 31)):
        assert run_both(p, torch.tensor([x], dtype=torch.int32), [0, 1], 0 * one, 0.3 * one, q)[1] == [0]
        assert run_both(p, torch.tensor([x], dtype=torch.int32), [0, 1], 0 * one, 0.3 * one, None)[1] == [0]


def test_verify_inconsistent_bounds_are_left_out():
    g = gen(9)
    p, draft, _, au, su, q = make_drafts(g, [2, 2, 2], 50, F32, True)
    for cu in ([0, 4, 2, 6], [0, 2, 9, 6], [-1, 2, 4, 6]):
        got = verify_drafts(p.cuda(), draft.cuda(), ints(cu), au.cuda(), su.cuda(), q=q.cuda())
        bad = [b for b in range(3) if not 0 <= cu[b] <= cu[b + 1] <= 6]
        assert bad and all(int(got[1][b]) == 0 and int(got[2][b]) == 0 for b in bad)


def test_verify_strided_rows_and_streams():
    """Rows inside a wider buffer, and a call on another stream than the current one."""
    g = gen(4)
    p, draft, cu, au, su, q = make_drafts(g, [3, 1, 2], 1003, BF, True)
    wide_p, wide_q = (torch.full((x.shape[0], 1100), 9.0, dtype=BF).cuda() for x in (p, q))
    wide_p[:, 5:1008], wide_q[:, 90:1093] = p.cuda(), q.cuda()
    args = draft.cuda(), ints(cu), au.cuda(), su.cuda()
    torch.cuda.synchronize()
    want = R.verify(p, draft, cu, au, su, q)
    got = verify_drafts(wide_p[:, 5:1008], *args, q=wide_q[:, 90:1093])
    assert [x.tolist() for x in got] == list(want)
    st = torch.cuda.Stream()
    got = verify_drafts(wide_p[:, 5:1008], *args, q=wide_q[:, 90:1093], stream=st)
    torch.cuda.synchronize()
    assert [x.tolist() for x in got] == list(want)


def test_verify_no_sequences():
    e = torch.zeros(0, device="cuda")
    t, a, d = verify_drafts(torch.zeros(0, 10, device="cuda"), ints([]), ints([0]), e, e)
    assert t.shape == (0,) and a.shape == (0,) and d.shape == (0,)


# ------------------------------------------------------------ a step of all of them
@pytest.mark.parametrize("captured", [False, True])
def test_speculative_steps_over_a_block_scaled_cache(captured):
    """Pages, append, attention, verification and the way back, step after step:
    lengths follow what was accepted, every token's attention is that of the cache
    as it is then, and refused drafts leave no page behind."""
    import _attention_ref as A
    from trellis_quantized_moe_exl3_gb300 import PagedKVCache, kv_append, paged_attention
    n, drafts, heads, hk, d, page, vocab = 5, 3, 8, 2, 64, 16, 97
    g = gen(77)
    cache = PagedKVCache(*[torch.zeros(60, page, hk, d, dtype=R.E4M3, device="cuda") for _ in range(2)],
                         *[torch.zeros(60, hk, device="cuda") for _ in range(2)])
    pool, ref = PagePool(60, page, 9, 12), R.Pool(60, page, 9, 12)
    rows_of = [4, 0, 8, 2, 7]
    seqs, rows = ints(rows_of), drafts + 1
    T = n * rows
    table = torch.randn(vocab, heads + 2 * hk, d, generator=g).to(BF).cuda()
    head = (torch.randn(heads * d, vocab, generator=g) * 0.3).cuda()
    f = (500000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    tokens_in = torch.zeros(n, rows, dtype=torch.int64, device="cuda")
    au, su = torch.zeros(n * drafts, device="cuda"), torch.zeros(n, device="cuda")
    cu = ints([b * drafts for b in range(n + 1)])
    q_probs = torch.full((n * drafts, vocab), 1.0 / vocab, device="cuda")
    q_lens = ints([rows] * n)

    def step():
        qkv = table[tokens_in.flatten()]
        s = pool.extend(seqs, q_lens, rows, T)
        q = kv_append(cache, s, qkv[:, heads:heads + hk], qkv[:, heads + hk:], inv_freq=f,
                      q=qkv[:, :heads])
        out = paged_attention(q, cache, s)
        p = (out.view(T, -1).float() @ head).softmax(-1)
        t, accepted, dropped = verify_drafts(p, tokens_in[:, 1:].int().flatten(), cu, au, su, q=q_probs)
        return s, q, out, p, t, accepted, dropped

    def whole():
        got = step()
        pool.trim(seqs, got[-1])
        return got

    # prompts of odd lengths first
    start = [17, 3, 40, 16, 1]
    s = pool.extend(seqs, ints(start), max(start), sum(start))
    ref.extend(rows_of, start, sum(start))
    kv = table[torch.randint(0, vocab, (sum(start),), generator=g).cuda()]
    kv_append(cache, s, kv[:, heads:heads + hk], kv[:, heads + hk:], inv_freq=f)
    cache.workspace(T, heads, n)
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = whole()
    total = 0
    for k in range(6):
        tokens_in.copy_(torch.randint(0, vocab, (n, rows), generator=g))
        au.copy_(torch.rand(n * drafts, generator=g) * 0.7)
        su.copy_(torch.rand(n, generator=g))
        if captured:
            graph.replay()
        else:
            got = whole()
        s, q, out, p, t, accepted, dropped = got
        cu_r, lens, tab, pos, slots = ref.extend(rows_of, [rows] * n, T)
        assert s.cu_q.tolist() == cu_r and s.seq_lens.tolist() == lens
        assert s.block_table.tolist() == tab and s.slots.tolist() == slots and s.positions.tolist() == pos
        want = R.verify(p.cpu(), tokens_in[:, 1:].flatten().cpu(), cu.tolist(), au.cpu(), su.cpu(),
                        q_probs.cpu())
        assert t.tolist() == want[0] and accepted.tolist() == want[1] and dropped.tolist() == want[2]
        # (nothing is appended between the attention and this look: the cache still holds the step)
        o, mag, _ = R.attention(q, R.values(cache.k, cache.k_scale), R.values(cache.v, cache.v_scale),
                                torch.tensor(tab), [rows] * n, lens, page, d ** -0.5, True, 0)
        tol = A.U[BF] * (o.abs() + mag) + 1e-4 * mag + 2.0 ** -25
        assert bool(((out.double().cpu() - o).abs() <= tol).all())
        ref.trim(rows_of, want[2])
        same_state(pool, ref)
        total += sum(want[1])
    assert total > 0 and cache.status() == 0
    pool.trim(seqs)
    ref.trim(rows_of)
    same_state(pool, ref)
    assert int(pool.count) == 60


def test_verify_drafts_of_no_sequence_and_padding():
    """Rows that belong to no sequence give -1, also where there is none at all."""
    p = torch.rand(7, 33, device="cuda")
    e = torch.zeros(0, device="cuda")
    t, a, d = verify_drafts(p, ints([1] * 7), ints([0]), torch.rand(7, device="cuda"), e)
    assert t.tolist() == [-1] * 7 and a.shape == d.shape == (0,)


def test_pool_on_another_stream():
    side = torch.cuda.Stream()
    seqs, q = ints([1, 0]), ints([20, 3])
    torch.cuda.synchronize()
    pool = PagePool(9, 16, 2, 4)
    step = pool.extend(seqs, q, 20, 23, stream=side)
    pool.trim(seqs, ints([7, 0]), stream=None)  # (ints waits for the device)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        pool.trim(seqs, q)
    assert step.cu_q.tolist() == [0, 20, 23] and pool.lens.tolist() == [0, 0]
    assert int(pool.count) == 9 and pool.status() == 1      # (7 of the 20 were gone already)


def test_tensors_of_another_device_are_refused():
    """Before anything is launched.  (The handles say that they live elsewhere: there
    may be one device only.)"""
    from trellis_quantized_moe_exl3_gb300 import PagedBatch, PagedKVCache, kv_append, paged_attention
    pool = PagePool(9, 16, 2, 4)
    seqs, q = ints([1, 0]), ints([20, 3])
    here = pool._device
    assert here == torch.cuda.current_device()
    pool._device = here + 1
    with pytest.raises(ValueError, match="another device"):
        pool.extend(seqs, q, 20, 23)
    with pytest.raises(ValueError, match="another device"):
        pool.trim(seqs)
    pool._device = here
    step = pool.extend(seqs, q, 20, 23)
    t = torch.zeros(9, 16, 1, 64, device="cuda").to(torch.float8_e4m3fn)
    s = torch.zeros(9, 1, device="cuda")
    cache = PagedKVCache(t, t.clone(), s, s.clone())
    x = torch.randn(23, 1, 64, device="cuda").to(BF)
    for both in (False, True):  # the batch beside the cache, then the tensors beside both
        cache._device = here + 1
        step._device = here + both
        with pytest.raises(ValueError, match="another device"):
            kv_append(cache, step, x, x)
        with pytest.raises(ValueError, match="another device"):
            paged_attention(x, cache, step)
    cache._device = step._device = here
    kv_append(cache, step, x, x)
    assert bool((paged_attention(x, cache, step) != 0).any())
    assert cache.status() == pool.status() == 0 and pool.lens.tolist() == [3, 20]
    with pytest.raises(ValueError, match="CUDA"):
        pool.extend(seqs, q.cpu(), 20, 23)
    with pytest.raises(ValueError, match="one device"):
        PagedBatch(step.cu_q.cpu().cuda(), step.seq_lens, _Elsewhere(step.block_table), 20)


class _Elsewhere:
    """A tensor that says it is on the next device."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.t.get_device() + 1
