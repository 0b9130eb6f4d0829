"""The attention operators on the GPU against their 64-bit forms.

Tolerances.  u is half a step of the output's type.
  norm/rotation: y is rounded once from fp32; the fp32 chain (mean of up to
    256 squares, one square root and division, three products, a two-term
    sum, cos and sin to 2^-22) is off by less than 3e-6 of the pair's or
    row's magnitude.
  attention: softmax terms are rounded to the 16-bit type of the products
    (fp16 with an E4M3 cache, never coarser than the output's type u), the
    output once more; scores are fp32 sums of D products, off by at most
    D * 2^-24 * sum |q k| * scale < 1e-4 for the data here, which moves a term
    by that much of itself."""
import math

import numpy as np
import pytest
import torch

import _attention_ref as R
from trellis_quantized_moe_exl3_gb300 import (PagedBatch, PagedKVCache, kv_append, paged_attention,
                                              qk_norm_rope)

pytestmark = pytest.mark.gpu

BF, FP, E4 = torch.bfloat16, torch.float16, R.E4M3
NAMES = {BF: "bf16", FP: "fp16", E4: "e4m3"}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def freqs(rot, theta=500000.0):
    return (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).cuda()


def close_rotated(got, ref, dtype):
    got = got.double().cpu()
    row = ref.abs().amax(-1, keepdim=True)
    tol = R.U[dtype] * ref.abs() + 3e-6 * row + (2.0 ** -25 if dtype == FP else 0)
    bad = ((got - ref).abs() > tol)
    assert not bad.any(), f"{int(bad.sum())} off, worst {float(((got - ref).abs() - tol).max()):.3e}"


# ------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("T,H,Hk,D,rot,inter,norm,dtype", [
    (1, 32, 8, 128, 128, False, True, BF),
    (3, 5, 1, 128, 64, True, True, FP),
    (2, 4, 2, 64, 64, False, True, BF),
    (7, 3, 3, 80, 48, False, True, FP),       # lanes of a row that hold nothing
    (5, 2, 1, 256, 256, True, True, BF),
    (4, 6, 2, 192, 64, False, False, FP),
    (9, 1, 1, 8, 0, False, True, BF),         # norm alone, one lane per row
    (6, 2, 2, 24, 16, True, True, BF),
    (1000, 8, 2, 64, 32, True, True, BF),
    (5001, 8, 2, 128, 128, False, True, BF),  # blocks of several tokens, a ragged last one
])
def test_norm_rope(T, H, Hk, D, rot, inter, norm, dtype):
    g = gen(T * 31 + D)
    fused = randn(g, T, H + 2 * Hk, D).to(dtype).cuda()  # strided inputs
    q, k = fused[:, :H], fused[:, H:H + Hk]
    wq, wk = [(1 + 0.2 * randn(g, D)).to(dtype).cuda() if norm else None for _ in range(2)]
    pos = torch.randint(-1000, 200000, (T,), generator=g, dtype=torch.int32).cuda()
    f = freqs(rot) if rot else None
    gq, gk = qk_norm_rope(q, k, pos if rot else None, f, wq, wk, eps=1e-5, interleaved=inter)
    for x, w, got in ((q, wq, gq), (k, wk, gk)):
        close_rotated(got, R.norm_rope(x, pos, f, w, 1e-5, inter), dtype)
    # in place gives the same bits
    buf = fused.clone()
    qk_norm_rope(buf[:, :H], buf[:, H:H + Hk], pos if rot else None, f, wq, wk, eps=1e-5,
                 interleaved=inter, q_out=buf[:, :H], k_out=buf[:, H:H + Hk])
    assert torch.equal(buf[:, :H], gq) and torch.equal(buf[:, H:H + Hk], gk)
    assert torch.equal(buf[:, H + Hk:], fused[:, H + Hk:])


def test_rotation_of_far_positions():
    """The angle is exact modulo a turn: positions up to 2^31 - 1."""
    pos = torch.tensor([0, 1, -1, 65535, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)],
                       dtype=torch.int32).cuda()
    g = gen(5)
    q = randn(g, len(pos), 2, 64).to(FP).cuda()
    f = freqs(64, 10000.0)
    got, none = qk_norm_rope(q, None, pos, f)
    assert none is None
    close_rotated(got, R.norm_rope(q, pos, f, None, 0, False), FP)
    assert torch.equal(got[0], q[0])


def test_norm_of_zero_and_nonfinite_rows():
    q = torch.zeros(3, 1, 64, dtype=BF, device="cuda")
    q[1, 0, 5], q[2, 0, 7] = math.inf, math.nan
    w = torch.ones(64, dtype=BF, device="cuda")
    got, _ = qk_norm_rope(q, None, None, None, w)
    assert bool((got[0] == 0).all()) and bool(got[1:].isnan().any(-1).all())


def test_norm_rope_no_tokens():
    q = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    assert qk_norm_rope(q, q[:, :2], torch.empty(0, dtype=torch.int32, device="cuda"),
                        freqs(64))[0].shape == (0, 4, 64)


# ------------------------------------------------------------ append
def make_cache(g, pages, page, hk, D, dtype, layout="NHD", fill=None):
    shape = (pages, page, hk, D) if layout == "NHD" else (pages, hk, page, D)

    def one():
        t = torch.empty(shape) if fill is not None else randn(g, *shape)
        if fill is not None:
            t.fill_(fill)
        t = t.to(dtype).cuda()
        return t if layout == "NHD" else t.permute(0, 2, 1, 3)

    ks, vs = [(0.01 + 0.02 * torch.rand(hk, generator=g)).cuda() if dtype == E4 else None
              for _ in range(2)]
    k, v = one(), one()
    return PagedKVCache(k, v, ks, vs)


def u8(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("qs,lens,page,H,Hk,D,rot,inter,dtype,cdt,layout", [
    ([1], [1], 16, 4, 1, 128, 128, False, BF, BF, "NHD"),
    ([1, 1, 1], [17, 1, 160], 16, 8, 2, 128, 128, False, BF, E4, "NHD"),
    ([5, 0, 33, 1], [5, 0, 100, 64], 32, 6, 2, 64, 32, True, FP, FP, "HND"),
    ([40, 3], [41, 300], 48, 3, 3, 80, 48, False, FP, E4, "HND"),
    ([700, 900, 1200], [700, 901, 4000], 64, 8, 2, 128, 64, True, BF, BF, "NHD"),
])
def test_append(qs, lens, page, H, Hk, D, rot, inter, dtype, cdt, layout):
    g = gen(sum(lens) + D)
    step, pages = R.make_step(g, qs, lens, page)
    cache = make_cache(g, pages, page, Hk, D, cdt, layout)
    k0, v0 = cache.k.clone(), cache.v.clone()
    T, pad = sum(qs), 3                                  # rows past the last sequence
    qkv = randn(g, T + pad, H + 2 * Hk, D).to(dtype).cuda()
    q, k, v = qkv.split([H, Hk, Hk], 1)
    wq, wk = [(1 + 0.2 * randn(g, D)).to(dtype).cuda() for _ in range(2)]
    f = freqs(rot)
    q_out = torch.full((T + pad, H, D), 7.0, dtype=dtype, device="cuda")
    batch = PagedBatch(step.cu_q, step.seq_lens, step.table, step.max_q)
    kv_append(cache, batch, k, v, inv_freq=f, k_weight=wk, q=q, q_weight=wq, q_out=q_out,
              interleaved=inter)
    assert cache.status() == 0
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(qs, lens)]).int()
    close_rotated(q_out[:T], R.norm_rope(q[:T], pos, f, wq, 1e-6, inter), dtype)
    assert bool((q_out[T:] == 7.0).all())
    page_of = torch.cat([step.table[b].cpu()[torch.arange(L - n, L) // page]
                         for b, (n, L) in enumerate(zip(qs, lens))]).long()
    at = (page_of, pos.long() % page)
    want_k = R.norm_rope(k[:T], pos, f, wk, 1e-6, inter)
    want_v = v[:T].double().cpu()
    for got, old, want, sc, name in ((cache.k, k0, want_k, cache.k_scale, "k"),
                                     (cache.v, v0, want_v, cache.v_scale, "v")):
        new = got.cpu()[at] if cdt != E4 else u8(got).cpu().view(got.shape)[at].view(E4)
        if cdt == E4:
            s = sc.double().cpu()[:, None]
            x = want / s
            # rounded once from a value that is off by 3e-6 of its row
            err = (new.double() - x.clamp(-448, 448)).abs()
            assert bool((err <= R.U[E4] * x.abs() + 2.0 ** -10 + 3e-6 * x.abs().amax(-1, keepdim=True)).all())
        elif name == "v":
            assert torch.equal(new.double(), want)
        else:
            close_rotated(new, want, dtype)
        # nothing else changed
        mask = torch.zeros(got.shape[:2], dtype=torch.bool)
        mask[at] = True
        same = (u8(got) == u8(old)).view(*got.shape[:2], -1).all(-1).cpu()
        assert bool(same[~mask].all())
    # without q, and with explicit positions, the same keys land in the same places
    again = make_cache(g, pages, page, Hk, D, cdt, layout, fill=0.0)
    again = PagedKVCache(again.k, again.v, cache.k_scale, cache.v_scale)
    kv_append(again, batch, k, v, inv_freq=f, k_weight=wk, interleaved=inter,
              positions=torch.cat([pos, torch.zeros(pad, dtype=torch.int32)]).cuda())
    assert torch.equal(u8(again.k).view(*again.k.shape[:2], -1)[at[0].cuda(), at[1].cuda()],
                       u8(cache.k).view(*cache.k.shape[:2], -1)[at[0].cuda(), at[1].cuda()])


def test_append_e4m3_saturates_and_keeps_nan():
    g = gen(1)
    cache = PagedKVCache(*[torch.zeros(1, 16, 1, 16, dtype=E4, device="cuda") for _ in range(2)])
    step, _ = R.make_step(g, [1], [1], 16)
    step.table[0, 0] = 0
    v = torch.tensor([1e4, -1e4, math.inf, -math.inf, math.nan, 448, 464, 0.5, 2.0 ** -9, 2.0 ** -11]
                     + [0.0] * 6, dtype=BF, device="cuda").view(1, 1, 16)
    kv_append(cache, PagedBatch(step.cu_q, step.seq_lens, step.table, 1), torch.zeros_like(v), v)
    got = cache.v[0, 0, 0].float().cpu().tolist()
    assert got[:4] == [448, -448, 448, -448] and math.isnan(got[4])
    assert got[5:10] == [448, 448, 0.5, 2.0 ** -9, 0]


def test_append_reports_bad_pages_and_batches():
    g = gen(2)
    k = torch.ones(3, 1, 16, dtype=BF, device="cuda")

    def run(cu, lens, table):
        cache = make_cache(g, 4, 16, 1, 16, BF, fill=0.0)
        b = PagedBatch(*[torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, lens, table)], 3)
        kv_append(cache, b, k, k)
        return cache.status(), cache.k.float().sum().item() / 16

    assert run([0, 3], [3], [[1, 2]]) == (0, 3)
    assert run([0, 3], [18], [[1, 4]]) == (1, 1)        # the second page does not exist
    assert run([0, 3], [18], [[-1, 3]]) == (1, 2)
    assert run([0, 3], [2], [[1, 2]]) == (2, 2)         # the first token stands before position 0
    assert run([0, 3], [40], [[1, 2]])[0] == 2          # longer than its table
    assert run([0, 4], [4], [[1, 2]]) == (2, 0)         # past the rows
    assert run([1, 3], [2], [[1, 2]])[0] == 2           # rows before the first sequence


# ------------------------------------------------------------ attention
def values(cache):
    """The cache as float64 values on the CPU."""
    out = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = t.float().cpu().double()
        out.append(x * s.cpu().double()[:, None] if s is not None else x)
    return out


def check_attention(cache, step, q, page, scale, causal, window, path=0, pad=0):
    T = sum(step.qs)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    batch = PagedBatch(step.cu_q, step.seq_lens, step.table, step.max_q)
    got, lse = paged_attention(q, cache, batch, scale=scale, causal=causal, window=window, out=out,
                               return_lse=True, path=path)
    assert cache.status() == 0
    k, v = values(cache)
    ref, mag, rlse = R.attention(q[:T], k, v, step.table.cpu(), step.qs, step.lens, page, scale,
                                 causal, window)
    u = R.U[q.dtype]
    tol = u * (ref.abs() + mag) + 1e-4 * mag + 2.0 ** -25
    g = got[:T].double().cpu()
    assert torch.equal(g.isfinite(), ref.isfinite())
    bad = ((g - ref).abs() > tol) & ref.isfinite()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((g - ref).abs() / tol).nan_to_num().max()):.2f} x tolerance at {bad.nonzero()[0].tolist()}"
    gl = lse[:T].double().cpu()
    assert torch.equal(gl == -math.inf, rlse == -math.inf)
    fin = rlse.isfinite()
    assert bool(((gl - rlse).abs()[fin] <= 1e-4 + 1e-6 * rlse.abs()[fin]).all())
    assert bool((got[T:] == 7.0).all())
    return got, lse


# (qs, lens, page, H, Hk, D, dtype, cache, causal, window)
CASES = [
    ([1], [1], 16, 4, 1, 128, BF, BF, True, 0),
    ([1], [1000], 16, 32, 8, 128, BF, BF, True, 0),
    ([1, 1, 1, 1], [5, 64, 65, 1000], 16, 8, 2, 128, FP, FP, True, 0),
    ([1] * 37, [(i * 61) % 700 + 1 for i in range(37)], 32, 8, 8, 64, BF, BF, True, 0),
    ([1, 1, 1], [300, 1, 2049], 64, 28, 4, 128, BF, E4, True, 0),
    ([1, 1], [100, 517], 16, 16, 1, 64, FP, E4, True, 0),
    ([4, 4, 3], [4, 100, 800], 32, 16, 4, 64, FP, FP, True, 0),
    ([3, 1, 8], [130, 3, 700], 48, 6, 2, 128, BF, E4, True, 0),       # a page size that is no power of two
    ([1, 5], [900, 901], 16, 4, 2, 128, BF, BF, True, 100),            # window
    ([2, 40], [500, 333], 64, 3, 1, 128, BF, BF, True, 17),
    ([5, 1, 7], [5, 90, 300], 16, 4, 4, 64, FP, FP, False, 0),         # every key
    ([6, 9], [3, 0], 16, 4, 2, 128, BF, BF, True, 0),                  # tokens before position 0, no keys
    ([0, 2, 0], [50, 70, 0], 16, 4, 2, 64, BF, BF, True, 0),           # sequences without new tokens
    ([100], [100], 16, 8, 2, 128, BF, BF, True, 0),
    ([65, 333, 1, 128], [65, 700, 400, 129], 64, 8, 2, 128, BF, BF, True, 0),
    ([130, 31], [1000, 31], 128, 7, 1, 128, FP, FP, True, 0),
    ([200], [450], 16, 8, 8, 64, FP, FP, True, 64),
    ([77, 150], [400, 151], 16, 8, 2, 128, BF, E4, True, 0),
    ([90, 300], [90, 555], 32, 12, 4, 64, FP, E4, True, 130),
    ([120, 10], [260, 10], 16, 6, 2, 128, BF, BF, False, 0),
    ([257], [1300], 256, 4, 4, 128, BF, BF, True, 0),
    ([300, 2, 40], [299, 1, 500], 16, 24, 8, 128, BF, BF, True, 0),    # the first token sees nothing
]


def ident(c):
    return f"q{c[0][0]}x{len(c[0])}_len{max(c[1])}_p{c[2]}_h{c[3]}-{c[4]}_d{c[5]}_{NAMES[c[6]]}_{NAMES[c[7]]}" \
        + ("" if c[8] else "_full") + (f"_w{c[9]}" if c[9] else "")


def setup(c, seed=0, layout="NHD", pad=2):
    qs, lens, page, H, Hk, D, dtype, cdt, causal, window = c
    g = gen(seed + sum(lens) * 7 + sum(qs) + D)
    step, pages = R.make_step(g, qs, lens, page)
    cache = make_cache(g, pages, page, Hk, D, cdt, layout)
    if cdt == E4:  # values of magnitude 1 behind the scales
        for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            t.copy_((torch.randn(t.shape, generator=g).cuda() / s[:, None]).clamp(-448, 448).to(E4))
    # places that no sequence holds are NaN
    held = torch.zeros(pages, page, dtype=torch.bool)
    for b, L in enumerate(lens):
        i = torch.arange(L)
        held[step.table[b].cpu()[i // page].long(), i % page] = True
    for t in (cache.k, cache.v):
        if cdt == E4:
            t.view(torch.uint8)[~held.cuda()] = 0x7F
        else:
            t[~held.cuda()] = math.nan
    q = randn(g, sum(qs) + pad, H, D).to(dtype).cuda()
    return cache, step, q


PATHS = [1, 2]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("c", CASES, ids=ident)
def test_attention(c, path):
    cache, step, q = setup(c)
    check_attention(cache, step, q, c[2], c[5] ** -0.5, c[8], c[9], path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("c", [
    ([1], [9000], 32, 16, 1, 128, BF, BF, True, 0),
    ([1, 2], [3333, 5001], 64, 4, 1, 128, FP, FP, True, 0),    # units that begin inside a piece
    ([1], [2600], 16, 8, 1, 64, BF, E4, True, 0),
    ([3, 1, 0, 1], [4000, 70, 9, 12345], 64, 12, 2, 64, FP, FP, True, 0),
    ([1], [20000], 64, 5, 1, 128, BF, E4, True, 7000),
    ([2], [41000], 64, 2, 2, 64, BF, BF, True, 0),             # 600 pieces
], ids=ident)
def test_units_of_many_parts(c, path):
    """Long sequences alone on the GPU: tens to hundreds of parts per unit,
    joined in one step and in two; a second call finds the counts at zero."""
    cache, step, q = setup(c)
    o, lse = check_attention(cache, step, q, c[2], c[5] ** -0.5, c[8], c[9], path)
    for _ in range(3):
        o2, lse2 = paged_attention(q, cache, PagedBatch(step.cu_q, step.seq_lens, step.table, step.max_q),
                                   window=c[9], return_lse=True, path=path)
        n = sum(c[0])
        assert torch.equal(o2[:n], o[:n]) and torch.equal(lse2[:n], lse[:n])


@pytest.mark.parametrize("path", PATHS)
def test_attention_layouts_and_strides(path):
    """Heads before places in a page; queries out of a fused projection."""
    c = ([1, 20], [200, 90], 16, 8, 2, 128, BF, BF, True, 0)
    cache, step, q = setup(c, layout="HND", pad=0)
    fused = torch.empty(q.shape[0], 12, 128, dtype=BF, device="cuda")
    fused[:, 2:10] = q
    check_attention(cache, step, fused[:, 2:10], 16, 0.1, True, 0, path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype,cdt", [(BF, BF), (FP, FP), (BF, E4)], ids=["bf16", "fp16", "e4m3"])
def test_unseen_nonfinite_values_do_not_count(dtype, cdt, path):
    """An infinity or NaN in a key or value reaches the tokens that see it and
    no other, on the causal edge and at a window's start."""
    c = ([12, 150], [40, 400], 16, 4, 2, 64, dtype, cdt, True, 30)
    cache, step, q = setup(c, seed=3, pad=0)
    tab = step.table.cpu()

    def put(t, b, pos, ch, x):
        at = (int(tab[b, pos // 16]), pos % 16, 0, ch)
        if cdt == E4:
            t.view(torch.uint8)[at] = 0x7F
        else:
            t[at] = x

    put(cache.v, 0, 35, 3, math.nan)
    put(cache.v, 1, 330, 60, math.inf)
    put(cache.k, 1, 380, 5, math.nan)
    # a NaN score makes the whole row NaN; the reference's max would spread it too
    k, v = values(cache)
    got = paged_attention(q, cache, PagedBatch(step.cu_q, step.seq_lens, step.table, 150), scale=0.125,
                          window=30, path=path).double().cpu()
    clean_k, clean_v = torch.nan_to_num(k, nan=0.5), torch.nan_to_num(v, nan=0.5, posinf=0.5)
    ref, mag, _ = R.attention(q, clean_k, clean_v, tab, step.qs, step.lens, 16, 0.125, True, 30)
    tol = R.U[dtype] * (ref.abs() + mag) + 1e-4 * mag + 2.0 ** -25
    touched = torch.zeros(ref.shape, dtype=torch.bool)
    pos0, pos1 = torch.arange(28, 40), torch.arange(250, 400)
    touched[:12][(pos0 >= 35) & (pos0 < 65), :2, 3] = True
    touched[12:][(pos1 >= 330) & (pos1 < 360), :2, 60] = True
    touched[12:][(pos1 >= 380) & (pos1 < 410), :2] = True
    assert torch.equal(~got.isfinite(), touched)
    assert bool(((got - ref).abs() <= tol)[~touched].all())


@pytest.mark.parametrize("path", PATHS)
def test_attention_large_scores(path):
    """Scores of several hundred: the running maximum keeps the terms finite,
    and a later key that beats the earlier ones by far takes over."""
    c = ([1, 60], [700, 300], 16, 4, 2, 64, FP, FP, True, 0)
    cache, step, q = setup(c, seed=9, pad=0)
    k, v = values(cache)
    got = paged_attention(q, cache, PagedBatch(step.cu_q, step.seq_lens, step.table, 60), scale=20.0,
                          path=path).double().cpu()
    # fp32 scores of magnitude up to 20 * 60 are off by up to 64 * 2^-24 * 20 * 55
    ref, mag, _ = R.attention(q, k, v, step.table.cpu(), step.qs, step.lens, 16, 20.0, True, 0)
    tol = R.U[FP] * (ref.abs() + mag) + 2 * 64 * 2.0 ** -24 * 20 * 55 * mag + 2.0 ** -25
    assert bool(((got - ref).abs() <= tol).all())


@pytest.mark.parametrize("path", PATHS)
def test_attention_is_repeatable(path):
    c = ([1, 33, 4], [3000, 700, 900], 64, 8, 2, 128, BF, BF, True, 0)
    cache, step, q = setup(c)
    batch = PagedBatch(step.cu_q, step.seq_lens, step.table, 33)
    a = paged_attention(q, cache, batch, return_lse=True, path=path)
    cache.ws[4096:].fill_(0xFF)   # what scratch holds does not matter
    b = paged_attention(q, cache, batch, return_lse=True, path=path)
    assert torch.equal(a[0][:38], b[0][:38]) and torch.equal(a[1][:38], b[1][:38])


@pytest.mark.parametrize("path", PATHS)
def test_attention_reports_bad_pages(path):
    """Keys of an absent page do not count, and the status says so."""
    c = ([2, 1], [100, 80], 16, 4, 2, 64, BF, BF, True, 0)
    cache, step, q = setup(c, pad=0)
    step.table[0, 2] = 1 << 20
    step.table[1, 0] = -3
    got = paged_attention(q, cache, PagedBatch(step.cu_q, step.seq_lens, step.table, 2), path=path)
    assert cache.status() == 1
    cache.clear_status()
    # the same with the page's keys at a score of -inf: a cache without them
    k, v = values(cache)
    tab = step.table.cpu()
    ref = torch.zeros(3, 4, 64, dtype=torch.float64)
    for t, (b, P) in enumerate([(0, 98), (0, 99), (1, 79)]):
        i = torch.tensor([j for j in range(P + 1) if not (b == 0 and j // 16 == 2) and not (b == 1 and j < 16)])
        for h in range(4):
            kk, vv = (x[tab[b, i // 16].long(), i % 16, h // 2] for x in (k, v))
            ref[t, h] = torch.softmax(kk @ q[t, h].double().cpu() * 0.125, 0) @ vv
    assert float((got.double().cpu() - ref).abs().max()) < 2 * 2.0 ** -8 * 1.5 + 1e-3


def test_attention_reports_bad_batches():
    c = ([2, 3, 4], [100, 80, 60], 16, 4, 2, 64, BF, BF, True, 0)
    for path in PATHS:
        cache, step, q = setup(c, pad=0)
        want = paged_attention(q, cache, PagedBatch(step.cu_q, step.seq_lens, step.table, 4), path=path)
        cu = torch.tensor([0, 2, 1, 5], dtype=torch.int32, device="cuda")   # sequence 1 runs backwards
        out = torch.full_like(q, 7.0)
        paged_attention(q, cache, PagedBatch(cu, step.seq_lens, step.table, 4), path=path, out=out)
        assert cache.status() == 2
        assert torch.equal(out[0], want[0]) and bool((out[5:] == 7.0).all())
        cache.clear_status()
        lens = step.seq_lens.clone()
        lens[1] = 100000
        out = paged_attention(q, cache, PagedBatch(step.cu_q, lens, step.table, 4), path=path)
        assert cache.status() & 2
        assert torch.equal(out[:2], want[:2]) and torch.equal(out[5:], want[5:])


@pytest.mark.parametrize("path", PATHS)
def test_no_tokens_no_sequences(path):
    cache, step, q = setup(([2], [5], 16, 4, 2, 64, BF, BF, True, 0))
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    none = PagedBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), e, e.view(0, 0), 0)
    out = torch.full_like(q, 7.0)
    paged_attention(q, cache, none, out=out, path=path)
    assert bool((out == 7.0).all())
    assert paged_attention(q[:0], cache, PagedBatch(step.cu_q, step.seq_lens, step.table, 2),
                           path=path).shape == (0, 4, 64)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("cdt", [BF, E4], ids=["bf16", "e4m3"])
def test_offsets_past_32_bits(cdt, path):
    """Pages beyond 4 GiB of the cache (and beyond 2^32 elements in E4M3)."""
    page, hk, D = 64, 8, 128
    per = page * hk * D
    pages = (5 << 30) // per if cdt == E4 else (5 << 30) // per // 2
    k, v = [torch.zeros(pages, page, hk, D, dtype=cdt, device="cuda") for _ in range(2)]
    cache = PagedKVCache(k, v)
    lens, qs = [200, 150], [1, 40]
    table = torch.tensor([[pages - 1, 3, pages - 5, pages - 7], [pages - 2, pages - 9, 0, 1]],
                         dtype=torch.int32, device="cuda")
    g = gen(4)
    T = sum(lens)
    kn, vn = [(randn(g, T, hk, D) * 2).to(BF).cuda() for _ in range(2)]
    full = PagedBatch(torch.tensor([0, 200, 350], dtype=torch.int32, device="cuda"),
                      torch.tensor(lens, dtype=torch.int32, device="cuda"), table, 200)
    kv_append(cache, full, kn, vn)
    q = randn(g, sum(qs), 16, D).to(BF).cuda()
    step = PagedBatch(torch.tensor([0, 1, 41], dtype=torch.int32, device="cuda"), full.seq_lens, table, 40)
    got = paged_attention(q, cache, step, path=path).double().cpu()
    assert cache.status() == 0
    kk, vv = [x.to(cdt).float().cpu().double() for x in (kn, vn)]
    seq = [torch.arange(200), torch.arange(200, 350)]
    t = 0
    for b, n in enumerate(qs):
        for i in range(n):
            P = lens[b] - n + i
            ids = seq[b][:P + 1]
            for h in range(16):
                p = torch.softmax(kk[ids, h // 2] @ q[t, h].double().cpu() * D ** -0.5, 0)
                ref, mag = p @ vv[ids, h // 2], p @ vv[ids, h // 2].abs()
                assert bool(((got[t, h] - ref).abs() <= 2.0 ** -8 * (ref.abs() + mag) + 1e-4 * mag).all())
            t += 1


def test_step_in_a_graph_follows_device_lengths():
    """Append and attention captured once; lengths and pages change on the device."""
    page, H, Hk, D, B = 16, 8, 2, 128, 3
    g = gen(11)
    pages = 40
    cache = make_cache(g, pages, page, Hk, D, BF)
    perm = torch.randperm(pages, generator=g).to(torch.int32)[:36].view(B, 12).cuda()
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 30, 1], dtype=torch.int32, device="cuda")
    batch = PagedBatch(cu, lens, perm, 1)
    qkv = torch.empty(B, H + 2 * Hk, D, dtype=BF, device="cuda")
    q, k, v = qkv.split([H, Hk, Hk], 1)
    f = freqs(D)
    qkv.copy_(randn(g, *qkv.shape))

    def step():
        qr = kv_append(cache, batch, k, v, inv_freq=f, q=q)
        return paged_attention(qr, cache, batch)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in ([6, 31, 2], [100, 32, 190], [17, 64, 65]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        qkv.copy_(randn(g, *qkv.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())
        assert cache.status() == 0


def test_other_streams():
    """The calls run on the stream they are given, in its order."""
    c = ([1, 9], [700, 300], 16, 8, 2, 128, BF, BF, True, 0)
    cache, step, q = setup(c, pad=0)
    batch = PagedBatch(step.cu_q, step.seq_lens, step.table, 9)
    want = paged_attention(q, cache, batch)
    s = torch.cuda.Stream()
    buf = torch.zeros_like(q)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        buf.copy_(q)
        got = paged_attention(buf, cache, batch)
    assert got is not None
    s.synchronize()
    assert torch.equal(got, want)


def test_a_graph_outlives_a_larger_workspace():
    """A graph captured before the handle's workspace grew replays on the old one."""
    c = ([1, 1], [300, 90], 16, 4, 2, 64, BF, BF, True, 0)
    cache, step, q = setup(c, pad=0)
    batch = PagedBatch(step.cu_q, step.seq_lens, step.table, 1)
    want = paged_attention(q, cache, batch)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = paged_attention(q, cache, batch)
    small = cache.ws
    big = torch.zeros(20000, 4, 64, dtype=BF, device="cuda")  # padding rows: the workspace of a larger call
    paged_attention(big, cache, batch)
    assert cache.ws.numel() > small.numel()
    junk = torch.full((small.numel(),), 0xFF, dtype=torch.uint8, device="cuda")
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and bool((junk == 0xFF).all()) and cache.status() == 0


@pytest.mark.parametrize("q", [4, 5, 8, 9])
@pytest.mark.parametrize("dtype,cdt,D", [(BF, BF, 128), (BF, E4, 128), (FP, E4, 64)],
                         ids=["bf16_128", "e4m3_128", "e4m3_64"])
def test_both_sides_of_the_choice_of_kernel(q, dtype, cdt, D):
    """4 heads per kv head and 4 to 9 drafted tokens: 16 to 36 rows, where the
    choice between the two kernels changes."""
    c = ([q, q - 1, 1], [700, q, 65], 32, 8, 2, D, dtype, cdt, True, 0)
    cache, step, q_ = setup(c)
    check_attention(cache, step, q_, c[2], D ** -0.5, True, 0)
