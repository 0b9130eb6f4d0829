"""Append to and attention over an E4M3 cache with a scale per block and head.

Tolerances.  u is half a step of a type.
  scales: the fp32 chain of norm and rotation is off by less than 3e-6 of a
    row's magnitude, so the power of two is the 64-bit form's unless the block's
    largest value is that near to 448 times one, which the data here are not
    (checked).
  new bytes: one rounding of a value that is off by 3e-6 of its row; old bytes
    and values: a product by a power of two (or one fp32 product) and a
    rounding, as torch does it, equal bit for bit.
  attention: softmax terms are rounded to fp16 (u at most that of the output's
    type), the output once more; scores are fp32 sums of D products plus a
    logarithm of magnitude up to 40, off by less than 1e-4 for the data here
    (64 * 2^-24 * 10 for the logarithm's sum, D * 2^-24 * sum |q k| * scale)."""
import math

import pytest
import torch

import _attention_ref as A
import _speculate_ref as R
from trellis_quantized_moe_exl3_gb300 import PagedBatch, PagedKVCache, kv_append, paged_attention
from trellis_quantized_moe_exl3_gb300._lib import Exl3Error

pytestmark = pytest.mark.gpu

BF, FP, E4 = torch.bfloat16, torch.float16, R.E4M3


def gen(seed):
    return torch.Generator().manual_seed(seed)


def freqs(rot):
    return (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).cuda() if rot else None


def u8(t):
    return t.contiguous().view(torch.uint8)


def blank(pages, page, hk, D, layout="NHD"):
    shape = (pages, page, hk, D) if layout == "NHD" else (pages, hk, page, D)
    kv = [torch.zeros(shape, dtype=E4, device="cuda") for _ in range(2)]
    if layout != "NHD":
        kv = [t.permute(0, 2, 1, 3) for t in kv]
    return PagedKVCache(*kv, *[torch.zeros(pages, hk, device="cuda") for _ in range(2)])


def batch_of(step):
    return PagedBatch(step.cu_q, step.seq_lens, step.table, step.max_q)


# ------------------------------------------------------------ append
def expect(cache, before, step, page, k, v, exact_keys=False):
    """Checks both halves of a cache after an append of keys k (64 bits) and
    values v against its state before."""
    table = step.table.cpu()
    for name, new in (("k", k), ("v", v.double().cpu())):
        old_x, old_s = before[name]
        got_x, got_s = u8(getattr(cache, name)).cpu().view(old_x.shape), getattr(cache, name + "_scale").cpu()
        want_x, want_s = u8(old_x).clone().view(old_x.shape), old_s.clone()
        check = torch.zeros(old_x.shape[:3], dtype=torch.bool)
        at = 0
        for b, (n, L) in enumerate(zip(step.qs, step.lens)):
            p0 = L - n
            for blk in range(p0 // page, -(-L // page) if n else 0):
                lo, hi, pg = max(p0, blk * page), min(L, (blk + 1) * page), int(table[b, blk])
                rows = new[at + lo - p0:at + hi - p0]
                for h in range(rows.shape[1]):
                    x = rows[:, h]
                    top = float(x.abs().max())
                    old = max(float(old_s[pg, h]), R.LEAST) if lo > blk * page else 0.0
                    s = old if old and top <= 448 * old else R.scale_for(top)
                    # (no border between two scales as near as the fp32 chain is off)
                    if name == "k" and not exact_keys and top > 0:
                        assert abs(math.log2(top / 448) - round(math.log2(top / 448))) > 1e-5
                    want_s[pg, h] = s
                    if lo > blk * page and s != old:
                        o = old_x[pg, :lo - blk * page, h].float() * float(torch.tensor(old) / s)
                        want_x[pg, :lo - blk * page, h] = o.to(E4).view(torch.uint8)
                    places = slice(lo - blk * page, hi - blk * page)
                    if name == "v":  # (bit for bit)
                        y = (x.float() * (1.0 / torch.tensor(s))).clamp(-448, 448).to(E4)
                        want_x[pg, places, h] = y.view(torch.uint8)
                    else:
                        y = got_x[pg, places, h].view(E4).double()
                        z = x / s  # (another 2^-23 of it at most where s is no power of two)
                        err = (y - z.clamp(-448, 448)).abs()
                        tol = R.U[E4] * z.abs() + 2.0 ** -10 + (3e-6 + 2.0 ** -23) * z.abs().amax(-1, keepdim=True)
                        assert bool((err <= tol).all())
                        check[pg, places, h] = True
            at += n
        assert torch.equal(got_s, want_s)
        assert torch.equal(got_x[~check], want_x[~check])


@pytest.mark.parametrize("steps,page,H,Hk,D,rot,inter,dtype,layout", [
    # (new tokens of every sequence, step by step)
    ([[1]], 16, 4, 1, 128, 128, False, BF, "NHD"),
    ([[1, 1, 1]] * 20, 16, 8, 2, 128, 128, False, BF, "NHD"),
    ([[5, 0, 33, 1], [1, 1, 1, 1], [0, 3, 4, 2]], 32, 6, 2, 64, 32, True, FP, "HND"),
    ([[40, 3], [2, 1], [9, 90]], 48, 3, 3, 80, 48, False, FP, "HND"),
    ([[130, 70], [200, 1]], 128, 4, 2, 256, 64, True, BF, "NHD"),
    ([[700, 900, 1200], [4, 4, 4], [64, 3, 300]], 64, 8, 2, 128, 64, True, BF, "NHD"),
    ([[300], [500]], 512, 2, 1, 64, 0, False, BF, "NHD"),       # blocks of more rows than a team holds
    ([[4]], 16, 2, 2, 48, 16, False, FP, "NHD"),
])
def test_append_blocks(steps, page, H, Hk, D, rot, inter, dtype, layout):
    """Step after step: values grow, so that blocks do."""
    g = gen(D + page + sum(map(sum, steps)))
    total = [sum(x) for x in zip(*steps)]
    whole, pages = A.make_step(g, total, total, page)
    cache = blank(pages, page, Hk, D, layout)
    lens = [0] * len(total)
    for i, qs in enumerate(steps):
        lens = [a + n for a, n in zip(lens, qs)]
        cu = torch.tensor([0] + torch.tensor(qs).cumsum(0).tolist(), dtype=torch.int32).cuda()
        step = A.Step(cu, torch.tensor(lens, dtype=torch.int32).cuda(), whole.table, max(qs), qs, lens)
        T, pad = sum(qs), 2
        qkv = (torch.randn(T + pad, H + 2 * Hk, D, generator=g) * 1.3 ** i).to(dtype).cuda()
        q, k, v = qkv.split([H, Hk, Hk], 1)
        wq = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda()
        wk = ((1 + 0.2 * torch.randn(D, generator=g)) * 1.4 ** i).to(dtype).cuda()
        before = {x: (getattr(cache, x).cpu(), getattr(cache, x + "_scale").cpu()) for x in "kv"}
        q_out = torch.full((T + pad, H, D), 7.0, dtype=dtype, device="cuda")
        f = freqs(rot)
        kv_append(cache, batch_of(step), k, v, inv_freq=f, k_weight=wk, q=q, q_weight=wq, q_out=q_out,
                  interleaved=inter)
        assert cache.status() == 0
        pos = torch.cat([torch.arange(L - n, L) for n, L in zip(qs, lens)]).int()
        rq = A.norm_rope(q[:T], pos, f, wq, 1e-6, inter)
        tol = R.U[dtype] * rq.abs() + 3e-6 * rq.abs().amax(-1, keepdim=True) + (2.0 ** -25 if dtype == FP else 0)
        assert bool(((q_out[:T].double().cpu() - rq).abs() <= tol).all())
        assert bool((q_out[T:] == 7.0).all())
        expect(cache, before, step, page, A.norm_rope(k[:T], pos, f, wk, 1e-6, inter), v[:T])


def test_append_blocks_refuses_rows_off_16_bytes():
    """24 channels of 8 bits: rows that begin between two 16-byte boundaries."""
    cache = blank(3, 16, 2, 24)
    k = torch.zeros(4, 2, 24, dtype=FP, device="cuda")
    with pytest.raises(Exl3Error) as e:
        kv_append(cache, batch_of(one_step(None, [4], [4], 16, [[1]])), k, k)
    assert e.value.status == 1


def one_step(g, qs, lens, page, pages_of):
    cu = torch.tensor([0] + torch.tensor(qs).cumsum(0).tolist(), dtype=torch.int32).cuda()
    table = torch.tensor(pages_of, dtype=torch.int32).cuda()
    return A.Step(cu, torch.tensor(lens, dtype=torch.int32).cuda(), table, max(qs), qs, lens)


@pytest.mark.parametrize("old", [0.0, 1e-20, 0.013, 3.0, 2.0 ** 40])
def test_append_to_blocks_with_any_scale(old):
    """Scales of other programs' making: kept where they cover the new values,
    grown from where they do not."""
    g = gen(5)
    for magnitude in (0.0, 1e-3, 1.0, 300.0, 5e4):
        cache = blank(3, 16, 2, 64)
        for x in (cache.k, cache.v):
            x.copy_((torch.randn(x.shape, generator=g) * 60).to(E4))
        cache.k_scale.fill_(old)
        cache.v_scale.fill_(old)
        step = one_step(g, [3], [10], 16, [[1]])
        k, v = ((torch.randn(3, 2, 64, generator=g) * magnitude).to(BF).cuda() for _ in range(2))
        before = {x: (getattr(cache, x).cpu(), getattr(cache, x + "_scale").cpu()) for x in "kv"}
        kv_append(cache, batch_of(step), k, v)
        assert cache.status() == 0
        # (without norm and rotation keys are exact as values are)
        expect(cache, before, step, 16, k.double().cpu(), v, exact_keys=True)


def test_append_blocks_nonfinite_and_extreme_values():
    cache = blank(1, 16, 1, 16)
    v = torch.zeros(2, 1, 16, dtype=BF, device="cuda")
    v[0, 0, :5] = torch.tensor([math.nan, 1.0, -3.0, 448.0, 2.0 ** -12])
    step = one_step(None, [2], [2], 16, [[0]])
    kv_append(cache, batch_of(step), torch.zeros_like(v), v)
    got = cache.v[0, 0, 0].float().cpu()
    assert math.isnan(float(got[0])) and got[1:5].tolist() == [1.0, -3.0, 448.0, 0.0]
    assert float(cache.v_scale[0, 0]) == 1.0 and float(cache.k_scale[0, 0]) == 2.0 ** -40
    v[1, 0, 0], v[1, 0, 1], v[1, 0, 2] = math.inf, -math.inf, 3e38
    step = one_step(None, [1], [2], 16, [[0]])
    kv_append(cache, batch_of(step), torch.zeros_like(v)[1:], v[1:])
    assert float(cache.v_scale[0, 0]) == 2.0 ** 40
    assert cache.v[0, 1, 0, :3].float().tolist() == [448.0, -448.0, 448.0]
    assert math.isnan(float(cache.v[0, 0, 0, 0].float())) and cache.status() == 0


def test_append_blocks_reports():
    k = torch.ones(3, 1, 16, dtype=BF, device="cuda")

    def run(cu, lens, table, scale=0.0):
        cache = blank(4, 16, 1, 16)
        cache.k_scale.fill_(scale)
        b = PagedBatch(*[torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, lens, table)], 3)
        kv_append(cache, b, k, k)
        return cache.status(), int((cache.k.float() != 0).sum()) // 16, int((cache.v.float() != 0).sum()) // 16

    assert run([0, 3], [3], [[1, 2]]) == (0, 3, 3)
    assert run([0, 3], [18], [[1, 4]]) == (1, 1, 1)        # the second page does not exist
    assert run([0, 3], [18], [[-1, 3]]) == (1, 2, 2)
    assert run([0, 3], [2], [[1, 2]]) == (2, 2, 2)         # the first token stands before position 0
    assert run([0, 3], [40], [[1, 2]])[0] == 2             # longer than its table
    assert run([0, 4], [4], [[1, 2]]) == (2, 0, 0)         # past the rows
    for bad in (-1.0, math.nan, math.inf, 2.0 ** 41):
        assert run([0, 3], [3], [[1, 2]], bad) == (0, 3, 3)    # a block that begins anew
        assert run([0, 3], [18], [[1, 2]], bad) == (8, 2, 3)   # older tokens behind no scale
    assert run([0, 3, 3], [3, 0], [[1, 2], [0, 0]]) == (0, 3, 3)
    assert run([0, 0, 3], [0, 3], [[1, 2], [0, 0]]) == (0, 3, 3)


def test_append_blocks_in_one_go_or_token_by_token():
    """The same scales, and the same values but for those that left E4M3's
    normal range and were rounded again."""
    g = gen(8)
    T, page = 70, 32
    k, v = ((torch.randn(T, 2, 64, generator=g) * torch.rand(T, 1, 1, generator=g) * 9).to(BF).cuda()
            for _ in range(2))
    table = [[2, 0, 1]]
    all_at_once = blank(3, page, 2, 64)
    kv_append(all_at_once, batch_of(one_step(g, [T], [T], page, table)), k, v)
    slowly = blank(3, page, 2, 64)
    for t in range(T):
        kv_append(slowly, batch_of(one_step(g, [1], [t + 1], page, table)), k[t:t + 1], v[t:t + 1])
    for x in "kv":
        a, b = getattr(all_at_once, x), getattr(slowly, x)
        assert torch.equal(getattr(all_at_once, x + "_scale"), getattr(slowly, x + "_scale"))
        a, b = a.float(), b.float()
        assert torch.equal(a[a.abs() >= 2.0 ** -6], b[a.abs() >= 2.0 ** -6])
        assert float((a - b).abs().max()) <= 2.0 ** -9       # a step of the subnormal range


# ------------------------------------------------------------ attention
def setup(c, seed=0, layout="NHD", pad=2, spread=3.0):
    qs, lens, page, H, Hk, D, dtype, causal, window = c
    g = gen(seed + sum(lens) * 7 + sum(qs) + D)
    step, pages = A.make_step(g, qs, lens, page)
    cache = blank(pages, page, Hk, D, layout)
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        n = (torch.randn(x.shape, generator=g) * 100).clamp(-448, 448)
        x.copy_(n.to(E4))
        s.copy_(0.01 * 2 ** (spread * torch.randn(s.shape, generator=g).clamp(-2, 2)) if s is cache.v_scale
                else 0.01 * (0.3 + torch.rand(s.shape, generator=g)))
    # places that no sequence holds are NaN, and so are the scales of such blocks
    held = torch.zeros(pages, page, dtype=torch.bool)
    for b, L in enumerate(lens):
        i = torch.arange(L)
        held[step.table[b].cpu()[i // page].long(), i % page] = True
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x.view(torch.uint8)[~held.cuda()] = 0x7F
        s[~held.any(1).cuda()] = math.nan
    q = torch.randn(sum(qs) + pad, H, D, generator=g).to(dtype).cuda()
    return cache, step, q


def check(cache, step, q, c, path, absent=None, status=0):
    qs, lens, page, H, Hk, D, dtype, causal, window = c
    T, scale = sum(qs), D ** -0.5
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    got, lse = paged_attention(q, cache, batch_of(step), scale=scale, causal=causal, window=window, out=out,
                               return_lse=True, path=path)
    assert cache.status() == status
    cache.clear_status()
    k, v = R.values(cache.k, cache.k_scale), R.values(cache.v, cache.v_scale)
    ref, mag, rlse = R.attention(q[:T], k, v, step.table.cpu(), qs, lens, page, scale, causal, window, absent)
    tol = R.U[q.dtype] * (ref.abs() + mag) + 1e-4 * mag + 2.0 ** -25
    g = got[:T].double().cpu()
    # (what is past the output type's range rounds to an infinity, as near to its
    # end as the tolerance either may)
    top = torch.finfo(dtype).max
    far, edge = ref.abs() - tol > top * (1 + R.U[dtype]), ref.abs() + tol > top
    assert torch.equal(g[far], torch.sign(ref[far]) * math.inf)
    ref = torch.where(far | edge, math.inf, ref)
    g = torch.where(far | edge, math.inf, g)
    assert torch.equal(g.isfinite(), ref.isfinite())
    bad = ((g - ref).abs() > tol) & ref.isfinite()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((g - ref).abs() / tol).nan_to_num().max()):.2f} x tolerance at {bad.nonzero()[0].tolist()}"
    gl = lse[:T].double().cpu()
    assert torch.equal(gl == -math.inf, rlse == -math.inf)
    fin = rlse.isfinite()
    assert bool(((gl - rlse).abs()[fin] <= 1e-4 + 1e-6 * rlse.abs()[fin]).all())
    assert bool((got[T:] == 7.0).all())
    return got, lse


# (qs, lens, page, H, Hk, D, dtype, causal, window)
CASES = [
    ([1], [1], 16, 4, 1, 128, BF, True, 0),
    ([1], [1000], 16, 32, 8, 128, BF, True, 0),
    ([1, 1, 1, 1], [5, 64, 65, 1000], 16, 8, 2, 128, FP, True, 0),
    ([1] * 37, [(i * 61) % 700 + 1 for i in range(37)], 32, 8, 8, 64, BF, True, 0),
    ([1, 1], [100, 517], 16, 16, 1, 64, FP, True, 0),
    ([4, 4, 3], [4, 100, 800], 32, 16, 4, 64, FP, True, 0),
    ([3, 1, 8], [130, 3, 700], 48, 6, 2, 128, BF, True, 0),
    ([1, 5], [900, 901], 16, 4, 2, 128, BF, True, 100),
    ([2, 40], [500, 333], 64, 3, 1, 128, BF, True, 17),
    ([5, 1, 7], [5, 90, 300], 16, 4, 4, 64, FP, False, 0),
    ([6, 9], [3, 0], 16, 4, 2, 128, BF, True, 0),
    ([0, 2, 0], [50, 70, 0], 16, 4, 2, 64, BF, True, 0),
    ([65, 333, 1, 128], [65, 700, 400, 129], 64, 8, 2, 128, BF, True, 0),
    ([130, 31], [1000, 31], 128, 7, 1, 128, FP, True, 0),
    ([200], [450], 16, 8, 8, 64, FP, True, 64),
    ([77, 150], [400, 151], 16, 8, 2, 128, BF, True, 0),
    ([120, 10], [260, 10], 112, 6, 2, 128, BF, False, 0),
    ([257], [1300], 256, 4, 4, 128, BF, True, 0),
    ([300, 2, 40], [299, 1, 500], 16, 24, 8, 128, BF, True, 0),
    ([2], [9000], 64, 8, 1, 64, BF, True, 0),
    ([1], [20000], 64, 5, 1, 128, FP, True, 7000),
]


def ident(c):
    return f"q{c[0][0]}x{len(c[0])}_len{max(c[1])}_p{c[2]}_h{c[3]}-{c[4]}_d{c[5]}_{'bf16' if c[6] == BF else 'fp16'}" \
        + ("" if c[7] else "_full") + (f"_w{c[8]}" if c[8] else "")


PATHS = [1, 2]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("c", CASES, ids=ident)
def test_attention_blocks(c, path):
    cache, step, q = setup(c)
    check(cache, step, q, c, path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("c", [CASES[2], CASES[7], CASES[12], CASES[15]], ids=ident)
def test_attention_blocks_far_apart(c, path):
    """Value scales from 0 to 2^40 in the blocks of one sequence: each row's
    output is as exact as the blocks that make it up allow."""
    cache, step, q = setup(c, layout="HND")
    g = gen(11)
    s = cache.v_scale
    live = ~s.isnan()
    e = torch.randint(-40, 41, s.shape, generator=g).float().cuda()
    s[live] = torch.exp2(e)[live]
    s[live & (e < -35)] = 0.0
    cache.k_scale[live & (e == 7).cuda()] = 0.0
    check(cache, step, q, c, path)
    # one large block that a window or the end of the range hides from no one
    s[live] = 2.0 ** -30
    check(cache, step, q, c, path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("c", [CASES[2], CASES[6], CASES[12], CASES[14]], ids=ident)
def test_attention_blocks_without_a_scale(c, path):
    """A scale that is negative, not finite or too large: the block's keys of
    that head count as absent, whatever bytes it holds, and the status says so."""
    cache, step, q = setup(c)
    page, hk = c[2], c[4]
    absent = torch.zeros(cache.k.shape[0], hk, dtype=torch.bool)
    for i, (b, bad) in enumerate(((0, -1.0), (1, math.nan), (1, math.inf), (len(c[0]) - 1, 2.0 ** 41))):
        blocks = -(-c[1][b] // page) if b < len(c[0]) else 0
        if blocks < 2:
            continue
        # (with a window, a block that is seen)
        pg = int(step.table[b, blocks - 2 if c[8] else (i * 3 + 1) % (blocks - 1)])
        (cache.k_scale if i % 2 else cache.v_scale)[pg, i % hk] = bad
        cache.v.view(torch.uint8)[pg, 3, i % hk, 5] = 0x7F
        absent[pg, i % hk] = True
    assert bool(absent.any())
    # (a NaN value of a head that has its scale still counts where it is seen)
    check(cache, step, q, c, path, absent, status=8)


@pytest.mark.parametrize("path", PATHS)
def test_attention_blocks_all_without_a_scale(path):
    c = ([3], [40], 16, 4, 1, 64, BF, True, 0)
    cache, step, q = setup(c)
    cache.v_scale.fill_(-1.0)
    out, lse = paged_attention(q[:3], cache, batch_of(step), return_lse=True, path=path)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and cache.status() == 8


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("c", [CASES[2], CASES[12]], ids=ident)
def test_attention_blocks_unseen_values(c, path):
    """NaN keys and values reach the rows that see them and no others."""
    cache, step, q = setup(c)
    for b, L in enumerate(c[1]):
        at = L - 1
        pg = int(step.table[b, at // c[2]])
        cache.v.view(torch.uint8)[pg, at % c[2], 0, 3] = 0xFF
    check(cache, step, q, c, path)


@pytest.mark.parametrize("path", PATHS)
def test_attention_blocks_equal_scales_per_head(path):
    """With one scale everywhere the result is that of a scale per head, up to
    the terms' rounding."""
    c = ([3, 70], [300, 500], 32, 8, 2, 128, BF, True, 0)
    cache, step, q = setup(c)
    cache.k_scale.fill_(0.01)
    cache.v_scale.fill_(0.25)
    got, lse = check(cache, step, q, c, path)
    per_head = PagedKVCache(cache.k, cache.v, torch.full((2,), 0.01, device="cuda"),
                            torch.full((2,), 0.25, device="cuda"))
    want, lse2 = paged_attention(q, per_head, batch_of(step), return_lse=True, path=path)
    # (0.25 is a power of two: the terms are the same up to their last bits)
    d = (got[:73].float() - want[:73].float()).abs()
    assert float(d.max()) <= 2 * 2.0 ** -8 * float(want[:73].float().abs().max())
    assert float((lse[:73] - lse2[:73]).abs().max()) <= 1e-5


def test_attention_blocks_results_do_not_depend_on_timing():
    c = ([1, 2], [3333, 5001], 64, 4, 1, 128, BF, True, 0)
    cache, step, q = setup(c)
    want = paged_attention(q, cache, batch_of(step), return_lse=True)
    for _ in range(3):
        got = paged_attention(q, cache, batch_of(step), return_lse=True)
        assert all(torch.equal(a[:3], b[:3]) for a, b in zip(got, want))


# ------------------------------------------------------------ how a line is cut, streams, graphs
@pytest.mark.parametrize("qs,lens,H,Hk,D", [
    ([1] * 32, [(i * 97) % 1500 + 1 for i in range(32)], 8, 2, 128),     # as many as a warp cuts
    ([1] * 33, [(i * 97) % 1500 + 1 for i in range(33)], 8, 2, 128),     # one more
    ([0] * 31 + [1], [50] * 31 + [5000], 4, 1, 64),                      # one of them has new tokens
    ([1, 1, 1, 1], [1, 512, 513, 9000], 8, 8, 64),                       # whole units beside cut ones
    ([70, 3, 1], [90, 2000, 30000], 16, 2, 64),                          # several chunks of rows
    ([2, 2], [70000, 3], 2, 2, 128),                                     # parts joined in two steps
    ([1] * 20, [8000 - 390 * i for i in range(20)], 16, 8, 128),         # too long to be cut one by one
    ([300], [300], 8, 1, 64),                                            # more units than half the grid
])
def test_attention_blocks_cuts(qs, lens, H, Hk, D):
    c = (qs, lens, 64, H, Hk, D, BF, True, 0)
    cache, step, q = setup(c)
    first = check(cache, step, q, c, 1)
    for _ in range(2):  # the counters are back at zero, and the result is the same
        again = paged_attention(q, cache, batch_of(step), scale=D ** -0.5, return_lse=True, path=1)
        assert all(torch.equal(a[:sum(qs)], b[:sum(qs)]) for a, b in zip(first, again))


@pytest.mark.parametrize("path", PATHS)
def test_attention_blocks_without_a_scale_beside_nan(path):
    """A NaN that some rows see sends tiles through the careful way: blocks without
    a scale stay absent there too."""
    c = CASES[12]
    cache, step, q = setup(c)
    absent = torch.zeros(cache.k.shape[0], c[4], dtype=torch.bool)
    b, L = 1, c[1][1]                                   # 333 new tokens of 700
    nan_at, bad_blk = L - 100, (L - 150) // c[2]
    pg, bad_pg = int(step.table[b, nan_at // c[2]]), int(step.table[b, bad_blk])
    for h in range(c[4]):
        cache.v.view(torch.uint8)[pg, nan_at % c[2], h, 7] = 0x7F
        cache.v.view(torch.uint8)[bad_pg, 5, h, 9] = 0x7F
        cache.v_scale[bad_pg, h] = -2.0
        absent[bad_pg, h] = True
    check(cache, step, q, c, path, absent, status=8)


def test_block_scales_on_other_streams_and_in_graphs():
    """Append and attention on a stream of their own (stream= and a current one),
    and two captured graphs of one handle replayed in turn."""
    g = gen(21)
    qs, lens, page = [1, 5, 40], [30, 5, 333], 16
    step, pages = A.make_step(g, qs, lens, page)
    T = sum(qs)
    qkv, f = torch.randn(T, 12, 64, generator=g).to(BF).cuda(), freqs(64)

    def fresh():
        cache = blank(pages, page, 2, 64)
        for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            x.copy_((torch.randn(x.shape, generator=gen(5)) * 50).to(E4))
            s.fill_(2.0 ** -6)
        return cache

    def run(cache, stream=None):
        q = kv_append(cache, batch_of(step), qkv[:, 8:10], qkv[:, 10:], q=qkv[:, :8], inv_freq=f,
                      stream=stream)
        return paged_attention(q, cache, batch_of(step), stream=stream)

    cache = fresh()
    want = run(cache)
    state = [u8(cache.k), u8(cache.v), cache.k_scale.clone(), cache.v_scale.clone()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for how in ("stream=", "current"):
        cache = fresh()
        torch.cuda.synchronize()
        if how == "stream=":
            got = run(cache, side)
        else:
            with torch.cuda.stream(side):
                got = run(cache)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and cache.status() == 0
        for a, b in zip(state, [u8(cache.k), u8(cache.v), cache.k_scale, cache.v_scale]):
            assert torch.equal(a, b)
    cache = fresh()
    run(cache)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(cache)
        graphs.append((graph, out))
    for graph, out in graphs + graphs:
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert cache.status() == 0


@pytest.mark.parametrize("page,D", [(16, 128), (64, 64), (256, 128)])
def test_append_blocks_whatever_max_q_says(page, D):
    """max_q only picks how many lanes share a block: the bytes are the same."""
    g = gen(page)
    qs, lens = [40, 1, 300], [55, 70, 333]
    step, pages = A.make_step(g, qs, lens, page)
    k, v = (torch.randn(sum(qs), 2, D, generator=g).to(FP).cuda() for _ in range(2))
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(FP).cuda()
    want = None
    for hint in (300, 0, 1, 2, 9, 33, 1 << 20):
        cache = blank(pages, page, 2, D)
        kv_append(cache, PagedBatch(step.cu_q, step.seq_lens, step.table, hint), k, v, inv_freq=freqs(D),
                  k_weight=w)
        got = [u8(cache.k), u8(cache.v), cache.k_scale, cache.v_scale]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and cache.status() == 0
