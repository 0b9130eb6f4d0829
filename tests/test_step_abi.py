"""Refusals of the calls that know their step, made on the host before any launch
(no GPU: the pointers are never read)."""
import pytest

from test_attention_abi import P, R
from test_speculate_abi import pool
from trellis_quantized_moe_exl3_gb300 import _lib, build

ARG, SHAPE, WS = _lib.EXL3_ERR_ARG, _lib.EXL3_ERR_SHAPE, _lib.EXL3_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def trim(L, p="pool", num=4, seqs=P, drop=P, lens=P, ws=P, n=1 << 40):
    return L.exl3_pages_trim_step(R(pool() if p == "pool" else p), num, seqs, drop, lens, ws, n, None)


def test_trim_step_refusals(L):
    assert trim(L, p=None) == ARG and trim(L, seqs=None) == ARG
    for kw in (dict(num=-1), dict(num=65536), dict(p=pool(page_size=24)), dict(p=pool(max_seqs=0))):
        assert trim(L, **kw) == SHAPE, kw
    assert trim(L, ws=None) == WS and trim(L, ws=P + 4) == WS and trim(L, n=100) == WS
    assert trim(L, num=0, seqs=None, lens=None) == 0


def verify(L, p=P, ps=100, q=P, qs=100, dt=3, vocab=100, B=2, D=6, cu=P, draft=P, au=P, su=P, lens=P, t=P,
           a=P, d=P):
    return L.exl3_verify_drafts_step(p, ps, q, qs, dt, vocab, B, D, cu, draft, au, su, lens, t, a, d, None)


def test_verify_step_refusals(L):
    for kw in (dict(dt=2), dict(ps=99), dict(p=None), dict(cu=None), dict(su=None), dict(t=None),
               dict(a=None), dict(d=None)):
        assert verify(L, **kw) == ARG, kw
    for kw in (dict(vocab=0), dict(B=-1), dict(D=-1)):
        assert verify(L, **kw) == SHAPE, kw
    assert verify(L, B=0, D=0, p=None, q=None, cu=None, su=None, lens=None, t=None, a=None, d=None) == 0
