"""Block scales at the ends of what is allowed: strided scales, offsets past 31 bits,
the largest pages, many sequences."""
import pytest
import torch

import _attention_ref as A
import test_gpu_block_scales as T
from trellis_quantized_moe_exl3_gb300 import PagedBatch, PagedKVCache, kv_append, paged_attention

pytestmark = pytest.mark.gpu


def fill(cache, seed):
    g = T.gen(seed)
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x.copy_((torch.randn(x.shape, generator=g) * 60).to(T.E4))
        s.copy_(2.0 ** torch.randint(-9, -4, s.shape, generator=g).float())


def run(cache, step, qkv, heads, hk, path=0):
    q, k, v = qkv.split([heads, hk, hk], 1)
    q = kv_append(cache, T.batch_of(step), k, v, q=q, inv_freq=T.freqs(64))
    return paged_attention(q, cache, T.batch_of(step), path=path)


def same(a, b):
    for x in ("k", "v", "k_scale", "v_scale"):
        p, q = getattr(a, x), getattr(b, x)
        assert torch.equal(T.u8(p) if x in "kv" else p, T.u8(q) if x in "kv" else q)


@pytest.mark.parametrize("path", T.PATHS)
def test_strided_scales(path):
    """k and v scales side by side in one buffer, wider than they need."""
    g = T.gen(3)
    qs, lens, page, heads, hk = [3, 40, 1], [30, 300, 17], 32, 8, 2
    step, pages = A.make_step(g, qs, lens, page)
    qkv = torch.randn(sum(qs), heads + 2 * hk, 64, generator=g).to(T.BF).cuda()
    plain = T.blank(pages, page, hk, 64)
    fill(plain, 9)
    both = torch.full((pages, 2, hk + 3), -1.0, device="cuda")
    strided = PagedKVCache(plain.k.clone(), plain.v.clone(), both[:, 0, 1:1 + hk], both[:, 1, 1:1 + hk])
    strided.k_scale.copy_(plain.k_scale)
    strided.v_scale.copy_(plain.v_scale)
    want, got = (run(c, step, qkv, heads, hk, path) for c in (plain, strided))
    assert torch.equal(got, want) and strided.status() == plain.status() == 0
    same(strided, plain)
    assert bool((both[:, :, 0] == -1).all()) and bool((both[:, :, 1 + hk:] == -1).all())


@pytest.mark.parametrize("path", T.PATHS)
def test_pages_past_31_bits(path):
    """The last pages of a cache of 2.4 GB a side against the first of a small one."""
    g = T.gen(4)
    qs, lens, page, heads, hk = [2, 50], [200, 130], 64, 8, 8
    step, pages = A.make_step(g, qs, lens, page)
    qkv = torch.randn(sum(qs), heads + 2 * hk, 128, generator=g).to(T.BF).cuda()
    small = T.blank(pages, page, hk, 128)
    fill(small, 11)
    many = 36000
    assert (many - pages) * page * hk * 128 > 1 << 31
    kv = [torch.zeros(many, page, hk, 128, dtype=T.E4, device="cuda") for _ in range(2)]
    large = PagedKVCache(*kv, *[torch.zeros(many, hk, device="cuda") for _ in range(2)])
    for x in ("k", "v", "k_scale", "v_scale"):
        getattr(large, x)[many - pages:].copy_(getattr(small, x))
    table = step.table + (step.table >= 0) * (many - pages)
    far = A.Step(step.cu_q, step.seq_lens, table.to(torch.int32), step.max_q, qs, lens)
    want, got = run(small, step, qkv, heads, hk, path), run(large, far, qkv, heads, hk, path)
    assert torch.equal(got, want) and large.status() == small.status() == 0
    tail = PagedKVCache(*[getattr(large, x)[many - pages:] for x in ("k", "v", "k_scale", "v_scale")])
    same(tail, small)
    assert not bool(T.u8(large.k[:many - pages]).any()) and not bool(large.v_scale[:many - pages].any())


@pytest.mark.parametrize("page,D,rot", [(4096, 64, 64), (4096, 256, 0), (4080, 128, 64)])
def test_append_to_the_largest_pages(page, D, rot):
    g = T.gen(page + D)
    qs, lens = [5000, 1, 300], [5300, 4097, 8000]
    step, pages = A.make_step(g, qs, lens, page)
    cache = T.blank(pages, page, 1, D)
    fill(cache, 2)
    k, v = ((torch.randn(sum(qs), 1, D, generator=g) * 30).to(T.BF).cuda() for _ in range(2))
    before = {x: (getattr(cache, x).cpu(), getattr(cache, x + "_scale").cpu()) for x in "kv"}
    kv_append(cache, T.batch_of(step), k, v, inv_freq=T.freqs(rot))
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(qs, lens)]).int()
    T.expect(cache, before, step, page, A.norm_rope(k, pos, T.freqs(rot), None, 1e-6, False), v,
             exact_keys=rot == 0)
    assert cache.status() == 0


@pytest.mark.parametrize("n,rows", [(2000, 1), (700, 3)])
def test_many_sequences(n, rows):
    """All at once as in parts: a sequence's results do not depend on the others."""
    g = T.gen(n)
    page, heads, hk = 16, 4, 1
    lens = [rows + (i * 37) % 40 for i in range(n)]
    step, pages = A.make_step(g, [rows] * n, lens, page)
    qkv = torch.randn(n * rows, heads + 2 * hk, 64, generator=g).to(T.BF).cuda()
    all_at_once, parts = T.blank(pages, page, hk, 64), T.blank(pages, page, hk, 64)
    for c in (all_at_once, parts):
        fill(c, 6)
    got = run(all_at_once, step, qkv, heads, hk, 1)
    size = 100
    for i in range(0, n, size):
        m = min(size, n - i)
        cu = torch.arange(0, m * rows + 1, rows, dtype=torch.int32, device="cuda")
        part = A.Step(cu, step.seq_lens[i:i + m].contiguous(), step.table[i:i + m].contiguous(), rows,
                      [rows] * m, lens[i:i + m])
        want = run(parts, part, qkv[i * rows:(i + m) * rows], heads, hk, 1)
        # (parts of a sequence may be cut elsewhere: softmax terms and the output are 16 bits)
        d = (got[i * rows:(i + m) * rows].float() - want.float()).abs()
        assert float(d.max()) <= 4 * 2.0 ** -8 * float(want.float().abs().max())
    same(all_at_once, parts)
    assert all_at_once.status() == parts.status() == 0
