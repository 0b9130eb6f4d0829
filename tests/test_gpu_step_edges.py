"""What a speculative step does where its calls meet: sequences without pages,
bounds that make no sense, odd probabilities, tensors that are freed or saved."""
import io
import math

import pytest
import torch

import _speculate_ref as R
from trellis_quantized_moe_exl3_gb300 import PagedKVCache, PagePool, kv_append, paged_attention, verify_drafts

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def state(pool):
    return [t.clone() for t in (pool.table, pool.lens, pool.free, pool.count)]


# ------------------------------------------------------------ sequences that a step does not serve
@pytest.mark.parametrize("captured", [False, True])
def test_sequences_without_pages_keep_their_tokens(captured):
    """The whole loop with a pool that runs out: a sequence that gets no pages gets no
    token and no counts, and its row, length and pages stay as they were."""
    page, rows, cols, hk, d, drafts, vocab = 16, 4, 4, 1, 64, 3, 50
    start, pages = [15, 14, 16, 3], 6              # four pages taken, two left
    need = drafts + 1
    g = gen(1)
    cache = PagedKVCache(*[torch.zeros(pages, page, hk, d, dtype=R.E4M3, device="cuda") for _ in range(2)],
                         *[torch.zeros(pages, hk, device="cuda") for _ in range(2)])
    pool, ref = PagePool(pages, page, rows, cols), R.Pool(pages, page, rows, cols)
    seqs, n, T = [0, 1, 2, 3], 4, 4 * need
    kv = torch.randn(sum(start), 2 * hk, d, generator=g).to(BF).cuda()
    kv_append(cache, pool.extend(ints(seqs), ints(start), 16, sum(start)), kv[:, :hk], kv[:, hk:])
    ref.extend(seqs, start, sum(start))
    x = torch.randn(T, 3 * hk, d, generator=g).to(BF).cuda()
    p = torch.rand(T, vocab, generator=g).cuda()
    p /= p.sum(-1, keepdim=True)
    q = torch.full((n * drafts, vocab), 1.0 / vocab, device="cuda")
    draft = torch.randint(0, vocab, (n * drafts,), generator=g).int().cuda()
    cu = ints([drafts * b for b in range(n + 1)])
    au, su = torch.rand(n * drafts, generator=g).cuda(), torch.rand(n, generator=g).cuda()
    seqs_d, q_lens = ints(seqs), ints([need] * n)

    def whole():
        s = pool.extend(seqs_d, q_lens, need, T)
        kv_append(cache, s, x[:, :hk], x[:, hk:2 * hk])
        out = paged_attention(x[:, 2 * hk:], cache, s)
        got = verify_drafts(p, draft, cu, au, su, q=q, step=s)
        pool.trim(seqs_d, got[2])
        return s, out, got

    cache.workspace(T, 1, n)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s, out, got = whole()
    unserved = 0
    for _ in range(3):
        before = state(pool)
        _, lens, table, _, _ = ref.extend(seqs, [need] * n, T)
        if captured:
            graph.replay()
        else:
            s, out, got = whole()
        assert s.seq_lens.tolist() == lens and s.block_table.tolist() == table
        want = R.verify(p.cpu(), draft.cpu(), cu.tolist(), au.cpu(), su.cpu(), q.cpu())
        for b in range(n):
            at = need * b
            if lens[b]:
                assert got[0][at:at + need].tolist() == want[0][at:at + need]
                assert int(got[1][b]) == want[1][b] and int(got[2][b]) == want[2][b]
            else:
                unserved += 1
                assert got[0][at:at + need].tolist() == [-1] * need
                assert int(got[1][b]) == int(got[2][b]) == 0
                assert bool((out[at:at + need] == 0).all())
                assert torch.equal(pool.table[b], before[0][b]) and int(pool.lens[b]) == int(before[1][b])
        ref.trim(seqs, [want[2][b] if lens[b] else 0 for b in range(n)])
        table, lens, free = ref.state()
        assert pool.table.tolist() == table and pool.lens.tolist() == lens
        assert pool.free[:len(free)].tolist() == free and int(pool.count) == len(free)
    assert unserved and pool.status() == 2


@pytest.mark.parametrize("q,seqs,max_tokens,pages", [
    ([3, 4, 5], [0, 1, 2], 12, 20),             # all of them served
    ([5, 40, 1, 16], [0, 1, 2, 3], 70, 7),      # too few pages for the second and the last
    ([3, 4, 5], [0, 7, 1], 12, 20),             # row 7 of 4
    ([3, 4, 5, 6], [2, 0, 2, 2], 18, 20),       # the same row three times
    ([49, 3], [1, 0], 60, 20),                  # past its row of the table
    ([5, 5, 0, 5], [0, 1, 2, 3], 9, 20),        # past max_tokens
])
def test_a_step_taken_back_whole_whatever_was_served(q, seqs, max_tokens, pages):
    pool = PagePool(pages, 16, 4, 3)
    pool.extend(ints([0, 1, 2, 3]), ints([16, 2, 15, 9]), 16, 42)
    assert pool.status() == 0
    before = state(pool)
    step = pool.extend(ints(seqs), ints(q), max(q), max_tokens)
    pool.trim(ints(seqs), ints(q), step=step)
    # (a refused sequence's request is a request that makes no sense to trim as well)
    for b, now in zip(before, state(pool)):
        assert torch.equal(b, now)
    # rows that were served are released, the others keep what they have
    step = pool.extend(ints(seqs), ints(q), max(q), max_tokens)
    served = {s for s, n in zip(seqs, step.seq_lens.tolist()) if n}
    pool.trim(ints(seqs), step=step)
    want = [0 if s in served else n for s, n in enumerate([16, 2, 15, 9])]
    assert pool.lens.tolist() == want
    assert int(pool.count) == pages - sum(-(-n // 16) for n in want)


def test_steps_of_another_size_are_refused():
    pool = PagePool(9, 16, 4, 3)
    step = pool.extend(ints([0, 1]), ints([3, 3]), 3, 6)
    with pytest.raises(ValueError, match="seq_lens"):
        pool.trim(ints([0]), ints([1]), step=step)
    p, z = torch.full((3, 9), 1 / 9, device="cuda"), torch.zeros(2, device="cuda")
    with pytest.raises(ValueError, match="seq_lens"):
        verify_drafts(p, ints([1, 2]), ints([0, 2]), z, z[:1], step=step)


# ------------------------------------------------------------ verification: bounds that make no sense
def verify_into_garbage(p, draft, cu, au, su, q):
    """verify_drafts with its outputs in memory that has held something else."""
    B, D = len(su), len(draft)
    n = sum((x + 3) // 4 * 4 for x in (D + B, B, B))
    torch.cuda.synchronize()
    for _ in range(4):
        held = [torch.full((n,), 0x5EED, dtype=torch.int32, device="cuda") for _ in range(8)]
        del held
    got = verify_drafts(p.cuda(), draft.cuda(), ints(cu), au.cuda(), su.cuda(), q=q.cuda())
    return [x.tolist() for x in got]


@pytest.mark.parametrize("D,cu", [
    (6, [0, 2, 4, 6]), (6, [1, 3, 5]), (6, [0, 3]), (6, [2, 2, 2]),          # rows before and behind
    (6, [0, 2, 9, 6]), (6, [-1, 2, 4, 6]), (6, [0, 2, 4, 7]), (6, [0, 2, -5, 6]),
    (6, [0, 2, 4, -1]), (6, [9, 2, 4, 6]), (6, [5, 0]), (6, [0, 6, 2]), (6, [9, 9, 9]), (6, [-3, -2, -1]),
    (6, [0, 1 << 30, 1 << 30, 6]), (6, [-(1 << 31), (1 << 31) - 1, 3, 6]), (0, [0, 5, 0]), (0, [0]),
    (6, [0, 4, 2, 6]), (100, [0, 50, 40, 90]), (100, [0, 1000, 10, 70]),
])
def test_every_token_is_written(D, cu):
    """Places of no sequence and of those left out hold -1, whatever was there."""
    B, vocab = len(cu) - 1, 40
    g = gen(D + B)
    p = torch.rand(D + B, vocab, generator=g)
    p /= p.sum(-1, keepdim=True).clamp(min=1e-9)
    q = torch.full((D, vocab), 1.0 / vocab)
    draft = torch.randint(0, vocab, (D,), generator=g).int()
    au, su = torch.rand(D, generator=g), torch.rand(B, generator=g)
    tokens, accepted, dropped = verify_into_garbage(p, draft, cu, au, su, q)
    lo, hi = cu[0] if 0 <= cu[0] <= D else 0, cu[-1] if 0 <= cu[-1] <= D else D
    want = [{-1} for _ in range(D + B)]
    claimed = [[] for _ in range(D + B)]
    for b in range(B):
        c0, c1 = cu[b], cu[b + 1]
        if lo <= c0 <= c1 <= hi:
            t, a, d = R.verify(p[b:], draft, [c0, c1], au, su[b:], q)
            assert accepted[b] == a[0] and dropped[b] == d[0]
            for j, x in enumerate(t):
                claimed[c0 + b + j].append(x)
        else:
            assert accepted[b] == dropped[b] == 0
    # (a place that bounds up and down give to two of them: either's)
    twice = any(x > y for x, y in zip(cu, cu[1:]))
    for j, x in enumerate(claimed):
        if x:
            want[j] = set(x) | ({-1} if twice else set())
    assert all(t in w for t, w in zip(tokens, want)), (tokens, want)


# ------------------------------------------------------------ verification: odd probabilities
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, BF])
@pytest.mark.parametrize("u", [0.0, 0.25, 0.75])
def test_acceptance_holds_probabilities_to_0_and_1(dtype, u):
    """NaN and what is negative count as 0, what is above 1 as 1, in the decision on a
    draft as in the weights of the token that follows."""
    values = [math.nan, -math.inf, -2.0, -0.0, 0.0, 0.125, 0.5, 1.0, 2.0, 1000.0, math.inf]
    pairs = [(a, b) for a in values for b in values]
    n, vocab = len(pairs), 5
    p = torch.zeros(2 * n, vocab)
    p[0::2, 1], p[1::2, 4] = 0.25, 1.0
    q = torch.zeros(n, vocab)
    for i, (a, b) in enumerate(pairs):
        p[2 * i, 3], q[i, 3] = a, b

    def held(x):
        return min(max(x, 0.0), 1.0) if x == x else 0.0

    p, q = p.to(dtype), q.to(dtype)
    draft = torch.full((n,), 3, dtype=torch.int32)
    t, accepted, dropped = verify_drafts(p.cuda(), draft.cuda(), ints(list(range(n + 1))),
                                         torch.full((n,), u, device="cuda"),
                                         torch.full((n,), 0.5, device="cuda"), q=q.cuda())
    t = t.view(n, 2).tolist()
    for i, (a, b) in enumerate(pairs):
        stands = u * held(b) < held(a)
        # refused: of token 1 (0.25) and token 3 (what is left of it), the one at half of the sum
        rest = max(held(a) - held(b), 0.0)
        want = [3, 4] if stands else [1 if 0.5 * (0.25 + rest) < 0.25 else 3, -1]
        assert t[i] == want and int(accepted[i]) == stands and int(dropped[i]) == 1 - stands, (a, b, t[i])
    # without q a draft is certain: refused only where it has no probability, or u is past it
    t, accepted, _ = verify_drafts(p.cuda(), draft.cuda(), ints(list(range(n + 1))),
                                   torch.full((n,), u, device="cuda"), torch.full((n,), 0.5, device="cuda"))
    assert accepted.tolist() == [int(u < held(a)) for a, _ in pairs]


# ------------------------------------------------------------ a step's tensors afterwards
def test_a_step_can_be_saved():
    """All of a step's and of a verification's tensors, together and one by one."""
    pool = PagePool(500, 16, 64, 40)
    step = pool.extend(ints(list(range(0, 64, 2))), ints([3] * 32), 3, 100)
    p, u = torch.full((5, 9), 1 / 9, device="cuda"), torch.full((3,), 0.5, device="cuda")
    got = verify_drafts(p, ints([1, 2, 3]), ints([0, 1, 3]), u, u[:2])
    of = {n: getattr(step, n) for n in ("cu_q", "seq_lens", "block_table", "positions", "slots")}
    of |= dict(zip(("tokens", "accepted", "dropped"), got))
    for what in [of] + [{n: t} for n, t in of.items()]:
        f = io.BytesIO()
        torch.save(what, f)
        f.seek(0)
        back = torch.load(f)
        assert all(torch.equal(back[n], t) and back[n].dtype == t.dtype for n, t in what.items())
        if "block_table" not in what:
            assert len(f.getvalue()) < 4000     # (the table is 5120 bytes)


def test_what_is_kept_of_a_step_does_not_keep_its_table():
    pool = PagePool(100, 16, 64, 60000)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    step = pool.extend(ints(list(range(64))), ints([1] * 64), 1, 64)
    assert torch.cuda.memory_allocated() - before > 64 * 60000 * 4
    kept = step.cu_q, step.seq_lens, step.positions, step.slots
    del step
    assert torch.cuda.memory_allocated() - before < 100000
    assert kept[0].tolist() == list(range(65)) and kept[1].tolist() == [1] * 64


def test_outputs_are_ordinary_tensors():
    """Also made inside torch.inference_mode, of no elements, and on another stream."""
    pool = PagePool(9, 16, 4, 3)
    side = torch.cuda.Stream()
    seqs, q = ints([0, 1]), ints([2, 1])
    torch.cuda.synchronize()
    step = pool.extend(seqs, q, 2, 3)
    t = step.block_table
    assert t.device == pool.table.device and t.is_contiguous() and not t.requires_grad and t._version == 0
    assert torch.equal(t + 0, t) and t.stride() == (3, 1) and step.slots.dtype == torch.int64
    t += 1                                    # (versions count, memory can be resized)
    assert t._version == 1
    t.resize_(7, 3)
    f = torch.zeros(3, device="cuda", requires_grad=True)
    (f * step.positions).sum().backward()
    assert f.grad.tolist() == [0.0, 1.0, 0.0]
    with torch.inference_mode():
        step = pool.extend(seqs, q, 2, 0)
        assert step.slots.is_inference() and step.slots.shape == step.positions.shape == (0,)
    with pytest.raises(RuntimeError, match="[Ii]nference"):
        step.slots.requires_grad_(False).add_(1)
    pool.clear_status()
    step = pool.extend(seqs, q, 2, 3, stream=side)
    torch.cuda.synchronize()
    assert step.cu_q.tolist() == [0, 2, 3] and step.block_table.cpu()[:, 0].min() >= 0
    n = torch.cuda.memory_allocated()
    del step, t
    assert torch.cuda.memory_allocated() < n


def test_pages_of_a_pool_whose_count_is_the_largest():
    """A count of 2^31 - 1 and the like is held to the pool's pages."""
    for count in ((1 << 31) - 1, -(1 << 31), 7):
        pool = PagePool(6, 16, 3, 4)
        pool.count.fill_(count)
        for _ in range(3):
            step = pool.extend(ints([0, 1, 2]), ints([30, 1, 0]), 30, 31)
            assert step.seq_lens.tolist() in ([30, 1, 0], [0, 0, 0])
            pool.trim(ints([2, 1, 0]), ints([5, 70, 1]))
            pool.trim(ints([0, 1, 2]))
            assert 0 <= int(pool.count) <= 6 and pool.lens.tolist() == [0, 0, 0]


def test_a_step_of_another_pools_pages_is_refused():
    """A pool whose pages have another size than the cache's, or of which the cache has
    fewer, would put tokens into the wrong places, or nowhere."""
    x = torch.randn(5, 1, 64, device="cuda").to(BF)
    cache = PagedKVCache(*[torch.zeros(9, 32, 1, 64, dtype=BF, device="cuda") for _ in range(2)])
    for pool in (PagePool(9, 16, 2, 4), PagePool(9, 64, 2, 4), PagePool(10, 32, 2, 4)):
        step = pool.extend(ints([0, 1]), ints([2, 3]), 3, 5)
        with pytest.raises(ValueError, match="pages of another size"):
            kv_append(cache, step, x, x)
        with pytest.raises(ValueError, match="pages of another size"):
            paged_attention(x, cache, step)
    for pages in (9, 5):
        step = PagePool(pages, 32, 2, 4).extend(ints([0, 1]), ints([2, 3]), 3, 5)
        kv_append(cache, step, x, x)
        assert bool((paged_attention(x, cache, step) != 0).all()) and cache.status() == 0
