"""Refusals of block scales, page pools and verification, made on the host before
any launch (no GPU: the pointers are never read)."""
import ctypes

import pytest
import torch

from test_attention_abi import P, R, batch, cache, heads, rope
from trellis_quantized_moe_exl3_gb300 import PagedKVCache, PagePool, _lib, build, verify_drafts

ARG, SHAPE, WS = _lib.EXL3_ERR_ARG, _lib.EXL3_ERR_SHAPE, _lib.EXL3_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def e4m3(**kw):
    return cache(**{**dict(dtype=2), **kw})


def scales(**kw):
    s = _lib.KVScales(P, 2 * P, 2)
    for k, x in kw.items():
        setattr(s, k, x)
    return s


BAD_SCALES = [dict(s=None), dict(s=scales(k=None)), dict(s=scales(v=None)), dict(s=scales(k=P + 2)),
              dict(s=scales(v=P + 1)), dict(s=scales(page_stride=1)), dict(s=scales(page_stride=-2)),
              dict(c=cache()), dict(c=cache(dtype=0)), dict(c=e4m3(k_scale=P)), dict(c=e4m3(v_scale=P))]


def attend(L, c="e4m3", s="scales", b=None, q=P, dt=1, T=8, h=4, scale=0.1, causal=1, window=0, out=P,
           lse=None, path=0, ws=P, n=1 << 40):
    c, s = e4m3() if c == "e4m3" else c, scales() if s == "scales" else s
    return L.exl3_paged_attention_blocks(R(c), R(s), R(b or batch()), q, 512, 64, dt, T, h, scale, causal,
                                         window, out, lse, path, ws, n, None)


def test_attention_blocks_refusals(L):
    for kw in BAD_SCALES + [dict(dt=2), dict(dt=3), dict(scale=0.0), dict(causal=2), dict(q=None),
                            dict(c=e4m3(head_stride=72)), dict(b=batch(cu_q=None)), dict(path=3)]:
        assert attend(L, **kw) == ARG, kw
    for kw in (dict(T=-1), dict(h=5), dict(c=e4m3(head_dim=80)), dict(c=e4m3(page_size=8)),
               dict(b=batch(num_seqs=65536))):
        assert attend(L, **kw) == SHAPE, kw
    assert attend(L, ws=None) == WS and attend(L, n=100) == WS
    n = L.exl3_launch_count()
    assert attend(L, T=0, q=None, out=None, ws=None) == 0
    assert attend(L, b=batch(num_seqs=0)) == 0
    assert L.exl3_launch_count() == n


def append(L, c="e4m3", s="scales", b=None, q=None, k=None, v=None, dt=1, T=8, r=None, status=P, eps=1e-6):
    c, s = e4m3() if c == "e4m3" else c, scales() if s == "scales" else s
    return L.exl3_kv_append_blocks(R(c), R(s), R(b or batch()), R(q), R(k or heads()), R(v or heads()), dt,
                                   T, R(r), None, eps, status, None)


def test_append_blocks_refusals(L):
    for kw in BAD_SCALES + [dict(dt=2), dict(dt=3), dict(status=None), dict(k=heads(x=None)),
                            dict(q=heads(out=None)), dict(b=batch(cu_q=None)), dict(eps=-1.0),
                            dict(r=rope(inv_freq=None))]:
        assert append(L, **kw) == ARG, kw
    for kw in (dict(T=-1), dict(k=heads(heads=3)), dict(c=e4m3(head_dim=264)), dict(r=rope(rotary_dim=72)),
               dict(b=batch(num_seqs=70000))):
        assert append(L, **kw) == SHAPE, kw
    n = L.exl3_launch_count()
    assert append(L, T=0) == 0 and append(L, b=batch(num_seqs=0)) == 0
    assert L.exl3_launch_count() == n


def pool(**kw):
    p = _lib.PagePool(100, 16, 8, 20, P, P, P, P)
    for k, x in kw.items():
        setattr(p, k, x)
    return p


def extend(L, p="pool", num=4, seqs=P, q=P, T=16, cu=P, lens=P, table=P, pos=P, slots=P, ws=P, n=1 << 40):
    return L.exl3_pages_extend(R(pool() if p == "pool" else p), num, seqs, q, T, cu, lens, table, pos, slots,
                               ws, n, None)


def trim(L, p="pool", num=4, seqs=P, drop=P, ws=P, n=1 << 40):
    return L.exl3_pages_trim(R(pool() if p == "pool" else p), num, seqs, drop, ws, n, None)


def test_pool_refusals(L):
    for kw in (dict(p=None), dict(seqs=None), dict(q=None), dict(cu=None), dict(lens=None), dict(table=None),
               dict(pos=None), dict(slots=None), dict(slots=P + 4), dict(p=pool(table=None)),
               dict(p=pool(lens=None)), dict(p=pool(free=None)), dict(p=pool(count=None))):
        assert extend(L, **kw) == ARG, kw
    shapes = [dict(num=-1), dict(num=65536), dict(p=pool(num_pages=-1)), dict(p=pool(page_size=0)),
              dict(p=pool(page_size=24)), dict(p=pool(page_size=8192)), dict(p=pool(max_seqs=0)),
              dict(p=pool(max_seqs=70000)), dict(p=pool(max_pages=0)), dict(p=pool(max_pages=1 << 27))]
    for kw in shapes + [dict(T=-1), dict(T=(1 << 30) + 1)]:
        assert extend(L, **kw) == SHAPE, kw
    for kw in shapes:
        assert trim(L, **kw) == SHAPE, kw
    assert trim(L, p=None) == ARG and trim(L, seqs=None) == ARG
    for f in (extend, trim):
        assert f(L, ws=None) == WS and f(L, ws=P + 4) == WS and f(L, n=100) == WS
    assert trim(L, num=0, seqs=None) == 0
    f = L.exl3_pages_workspace_size
    assert f(8, 4) > 0 and f(8, 0) <= f(8, 4) <= f(1000, 4)
    assert f(0, 1) == f(70000, 1) == f(8, -1) == f(8, 70000) == 0


def verify(L, p=P, ps=100, q=P, qs=100, dt=3, vocab=100, B=2, D=6, cu=P, draft=P, au=P, su=P, t=P, a=P, d=P):
    return L.exl3_verify_drafts(p, ps, q, qs, dt, vocab, B, D, cu, draft, au, su, t, a, d, None)


def test_verify_refusals(L):
    for kw in (dict(dt=2), dict(dt=4), dict(ps=99), dict(qs=99), dict(p=None), dict(p=P + 2), dict(q=P + 1),
               dict(dt=1, p=P + 1), dict(cu=None), dict(draft=None), dict(au=None), dict(su=None),
               dict(t=None), dict(a=None), dict(d=None)):
        assert verify(L, **kw) == ARG, kw
    for kw in (dict(vocab=0), dict(vocab=(1 << 24) + 1, ps=1 << 25, qs=1 << 25), dict(B=-1), dict(B=65536),
               dict(D=-1)):
        assert verify(L, **kw) == SHAPE, kw
    assert verify(L, B=0, D=0, p=None, q=None, cu=None, su=None, t=None, a=None, d=None) == 0


def test_python_refusals():
    with pytest.raises(ValueError):
        PagePool(10, 16, 4, 4, device="cpu")
    for bad in ((-1, 16, 4, 4), (10, 16, 0, 4), (10, 16, 4, 0)):
        with pytest.raises(ValueError):
            PagePool(*bad)
    z = torch.zeros(3)
    with pytest.raises(ValueError):
        verify_drafts(torch.zeros(4, 9), z.int()[:2], z.int(), z[:2], z[:2])
    t = torch.zeros(2, 16, 1, 64, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        PagedKVCache(t, t, torch.zeros(2, 1), torch.zeros(2, 1))


def test_structs_match(L):
    assert ctypes.sizeof(_lib.KVScales) == 24 and ctypes.sizeof(_lib.PagePool) == 48
