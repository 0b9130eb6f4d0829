"""Refusals of the attention operators, made on the host before any launch
(no GPU: the pointers are never read)."""
import ctypes

import pytest
import torch

from trellis_quantized_moe_exl3_gb300 import PagedBatch, PagedKVCache, _lib, build, paged_attention

ARG, SHAPE, WS = _lib.EXL3_ERR_ARG, _lib.EXL3_ERR_SHAPE, _lib.EXL3_ERR_WORKSPACE
P = 1 << 20  # a pointer that is aligned and never read


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def cache(**kw):
    c = _lib.KVCache(k=P, v=2 * P, dtype=_lib.EXL3_BF16, num_pages=10, page_size=16, kv_heads=2,
                     head_dim=64, page_stride=2048, token_stride=128, head_stride=64)
    for k, x in kw.items():
        setattr(c, k, x)
    return c


def batch(**kw):
    b = _lib.KVBatch(num_seqs=2, max_q=4, max_pages=8, table_stride=8, cu_q=P, seq_lens=P,
                     block_table=P)
    for k, x in kw.items():
        setattr(b, k, x)
    return b


def heads(**kw):
    h = _lib.Heads(x=P, out=3 * P, weight=None, heads=2, token_stride=512, head_stride=64,
                   out_token_stride=512, out_head_stride=64)
    for k, x in kw.items():
        setattr(h, k, x)
    return h


def rope(**kw):
    r = _lib.Rope(P, 64, 0)
    for k, x in kw.items():
        setattr(r, k, x)
    return r


def R(x):
    return ctypes.byref(x) if x is not None else None


def attend(L, c=None, b=None, q=P, qt=512, qh=64, dt=1, T=8, h=4, scale=0.1, causal=1, window=0,
           out=P, lse=None, path=0, ws=P, n=1 << 40):
    return L.exl3_paged_attention(R(c or cache()), R(b or batch()), q, qt, qh, dt, T, h, scale, causal,
                                  window, out, lse, path, ws, n, None)


def test_attention_refusals(L):
    inf, nan = float("inf"), float("nan")
    for kw in (dict(dt=2), dict(dt=7), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf),
               dict(scale=nan), dict(causal=2), dict(window=-1), dict(window=5, causal=0),
               dict(path=3), dict(path=-1), dict(q=None), dict(q=P + 8), dict(out=None),
               dict(out=P + 2), dict(lse=P + 2), dict(qt=12), dict(qh=-64),
               dict(c=cache(dtype=0)), dict(c=cache(dtype=5)), dict(c=cache(k=None)),
               dict(c=cache(v=P + 4)), dict(c=cache(token_stride=100)), dict(c=cache(page_stride=-2048)),
               dict(c=cache(k_scale=P)), dict(c=cache(dtype=2, head_stride=72)),
               dict(b=batch(cu_q=None)), dict(b=batch(block_table=None)), dict(b=batch(seq_lens=None))):
        assert attend(L, **kw) == ARG, kw
    for kw in (dict(T=-1), dict(h=0), dict(h=5), dict(T=1 << 30), dict(c=cache(head_dim=80)),
               dict(c=cache(head_dim=192)), dict(c=cache(page_size=8)), dict(c=cache(page_size=24)),
               dict(c=cache(page_size=8192)), dict(c=cache(kv_heads=0)), dict(c=cache(num_pages=-1)),
               dict(b=batch(num_seqs=-1)), dict(b=batch(num_seqs=65536)), dict(b=batch(max_pages=-1))):
        assert attend(L, **kw) == SHAPE, kw
    assert attend(L, ws=None) == WS and attend(L, n=1000) == WS
    assert L.exl3_paged_attention(None, R(batch()), P, 512, 64, 1, 8, 4, 0.1, 1, 0, P, None, 0, P,
                                  1 << 40, None) == ARG
    assert L.exl3_paged_attention(R(cache()), None, P, 512, 64, 1, 8, 4, 0.1, 1, 0, P, None, 0, P,
                                  1 << 40, None) == ARG
    # nothing to do is no error, and launches nothing
    n = L.exl3_launch_count()
    assert attend(L, T=0, q=None, out=None, ws=None) == 0
    assert attend(L, b=batch(num_seqs=0, cu_q=None, seq_lens=None, block_table=None)) == 0
    assert L.exl3_launch_count() == n


def test_workspace_size(L):
    f = L.exl3_paged_attention_workspace_size
    assert f(8, 8, 2, 128, 4) > 256 and f(8, 8, 2, 128, 4) == f(8, 8, 2, 128, 4)
    assert f(100000, 8, 2, 128, 4) >= f(8, 8, 2, 128, 4)
    assert f(-1, 8, 2, 128, 4) == f(8, 9, 2, 128, 4) == f(8, 8, 2, 96, 4) == f(8, 8, 2, 128, -1) == 0


def norm(L, q=None, k=None, dt=1, T=8, dim=64, pos=P, r=None, eps=1e-6):
    return L.exl3_qk_norm_rope(R(q or heads()), R(k), dt, T, dim, pos, R(r), eps, None)


def test_norm_rope_refusals(L):
    for kw in (dict(dt=2), dict(q=heads(x=None)), dict(q=heads(out=None)), dict(q=heads(x=P + 2)),
               dict(q=heads(weight=P + 2)), dict(q=heads(token_stride=100)),
               dict(q=heads(out_head_stride=4)), dict(k=heads(x=None)), dict(r=rope(inv_freq=None)),
               dict(r=rope(interleaved=2)), dict(r=rope(), pos=None), dict(eps=-1.0),
               dict(eps=float("nan"))):
        assert norm(L, **kw) == ARG, kw
    for kw in (dict(T=-1), dict(dim=0), dict(dim=60), dict(dim=264), dict(q=heads(heads=0)),
               dict(r=rope(rotary_dim=8)), dict(r=rope(rotary_dim=40)), dict(r=rope(rotary_dim=80))):
        assert norm(L, **kw) == SHAPE, kw
    assert L.exl3_qk_norm_rope(None, None, 1, 8, 64, P, None, 1e-6, None) == ARG
    assert norm(L, T=0, q=heads(x=None, out=None)) == 0


def append(L, c=None, b=None, q=None, k=None, v=None, dt=1, T=8, r=None, status=P, eps=1e-6):
    return L.exl3_kv_append(R(c or cache()), R(b or batch()), R(q), R(k or heads()), R(v or heads()),
                            dt, T, R(r), None, eps, status, None)


def test_append_refusals(L):
    for kw in (dict(dt=2), dict(dt=0), dict(status=None), dict(k=heads(x=None)), dict(v=heads(x=P + 2)),
               dict(q=heads(out=None)), dict(c=cache(k=None)), dict(c=cache(v_scale=P)),
               dict(c=cache(head_stride=60)), dict(b=batch(cu_q=None)), dict(eps=-1.0),
               dict(r=rope(inv_freq=None))):
        assert append(L, **kw) == ARG, kw
    for kw in (dict(T=-1), dict(k=heads(heads=3)), dict(v=heads(heads=1)), dict(c=cache(head_dim=264)),
               dict(c=cache(page_size=0)), dict(r=rope(rotary_dim=72)), dict(b=batch(num_seqs=70000))):
        assert append(L, **kw) == SHAPE, kw
    assert L.exl3_kv_append(R(cache()), R(batch()), None, None, R(heads()), 1, 8, None, None, 1e-6, P,
                            None) == ARG
    assert append(L, T=0) == 0


def test_python_refuses_cpu_tensors():
    t = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        PagedKVCache(t, t)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        PagedBatch(i, i[:2], i.view(1, 3), 1)
    with pytest.raises(ValueError):
        paged_attention(torch.zeros(1, 1, 64, dtype=torch.bfloat16), None, None)
