"""The operators of a speculative serving step over a paged 8-bit cache, as they are measured.

  pages      a step's block table, slot map, positions and lengths from the sequences' lengths, pages
             taken from the pool's free list and given back, all on the GPU
  append     new tokens' keys (normed and rotated) and values to an 8-bit cache that has a scale for
             each block (page) and head, older tokens of a block requantised where its scale grows
  attention  attention of new tokens over that cache
  verify     drafted tokens accepted or replaced by the target's probabilities and given random numbers

A case is a dict of plain values.  ``run`` computes the plain form, or, where ``own`` is true, calls
the package.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
TOP = 448.0             # the largest E4M3 value
LEAST, MOST = -40, 40   # exponents of the least and the greatest block scale


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a small decode batch: latency is everything
        dict(name="pages_decode", op="pages", seqs=8, q=1, q_lo=1, ctx=4000, ctx_lo=17, page=64,
             max_seqs=32, max_pages=128),
        # a large batch of drafts over long contexts, small pages
        dict(name="pages_verify", op="pages", seqs=256, q=6, q_lo=1, ctx=32000, ctx_lo=300, page=16,
             max_seqs=300, max_pages=2048),
        # a decode batch: one token of each of 64 sequences
        dict(name="append_decode", op="append", seqs=64, q=1, q_lo=1, ctx=2000, ctx_lo=100,
             heads=32, kv_heads=8, dim=128, rot=128, inter=False, norm=True, dtype="bf16", page=64),
        # ragged prompts that continue earlier context
        dict(name="append_prompt", op="append", seqs=5, q=2047, q_lo=700, ctx=4000, ctx_lo=2048,
             heads=32, kv_heads=8, dim=128, rot=128, inter=False, norm=True, dtype="bf16", page=64),
        # one user, short context: the smallest call
        dict(name="decode_one", op="attention", seqs=1, q=1, q_lo=1, ctx=1000, ctx_lo=1000, heads=32,
             kv_heads=8, dim=128, dtype="bf16", page=16, window=0, lse=False),
        # a decode batch with ragged contexts
        dict(name="decode_batch", op="attention", seqs=64, q=1, q_lo=1, ctx=8000, ctx_lo=500, heads=32,
             kv_heads=8, dim=128, dtype="bf16", page=64, window=0, lse=False),
        # four drafted tokens checked at once
        dict(name="verify_4", op="attention", seqs=16, q=4, q_lo=4, ctx=6001, ctx_lo=1003, heads=32,
             kv_heads=8, dim=64, dtype="fp16", page=32, window=0, lse=True),
        # chunks of odd lengths
        dict(name="chunk_333", op="attention", seqs=6, q=333, q_lo=65, ctx=8191, ctx_lo=2000, heads=32,
             kv_heads=8, dim=128, dtype="bf16", page=16, window=0, lse=False),
        # a whole prompt
        dict(name="prompt_7168", op="attention", seqs=1, q=7168, q_lo=7168, ctx=7168, ctx_lo=7168,
             heads=32, kv_heads=8, dim=128, dtype="bf16", page=64, window=0, lse=True),
        # one user's four drafts
        dict(name="drafts_one", op="verify", seqs=1, drafts=4, drafts_lo=4, vocab=32000, dtype="fp32",
             given=True),
        # a batch with ragged drafts from a drafting model
        dict(name="drafts_batch", op="verify", seqs=64, drafts=5, drafts_lo=1, vocab=131072,
             dtype="fp32", given=True),
        # drafts looked up in the text (certain, so without probabilities), an odd vocabulary
        dict(name="drafts_lookup", op="verify", seqs=33, drafts=8, drafts_lo=0, vocab=50001,
             dtype="bf16", given=False),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "attention", "attention", "attention", "verify", "verify"])
    page = rng.choice([16, 32, 64, 128])
    if op == "pages":
        seqs = _between(rng, 1, 512)
        ctx, q = _between(rng, 1, 1000000 // seqs), _between(rng, 1, max(1, 16384 // seqs))
        return dict(op=op, seqs=seqs, q=q, q_lo=rng.choice([q, 0, max(1, q // 3)]), ctx=ctx,
                    ctx_lo=ctx // rng.choice([1, 2, 9]), page=page, max_seqs=seqs + rng.randrange(0, 99),
                    max_pages=-(-(ctx + q) // page) + rng.randrange(0, 70))
    if op == "verify":
        vocab = _between(rng, 64, 200000)
        seqs, drafts = _between(rng, 1, max(2, min(128, 8000000 // vocab))), rng.randrange(1, 10)
        return dict(op=op, seqs=seqs, drafts=drafts, drafts_lo=rng.choice([drafts, 0, drafts // 2]),
                    vocab=vocab, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    given=rng.random() < 0.7)
    heads, kv_heads = rng.choice([(32, 8), (32, 4), (16, 2), (24, 8), (8, 8), (28, 4), (40, 8)])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    seqs = _between(rng, 1, 64)
    if op == "append":
        q = _between(rng, 1, max(1, 8192 // seqs))
        ctx_lo = q + rng.randrange(0, 2000)
        return dict(op=op, seqs=seqs, q=q, q_lo=max(1, q // rng.choice([1, 3])), ctx_lo=ctx_lo,
                    ctx=ctx_lo + rng.randrange(0, 1000), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), inter=rng.random() < 0.5, norm=rng.random() < 0.8,
                    dtype=dtype, page=page)
    kind = rng.choice(["decode", "decode", "verify", "chunk", "prompt"])
    if kind == "decode":
        q, ctx = 1, _between(rng, 1, 250000 // seqs)
    elif kind == "verify":
        q, ctx = rng.randrange(2, 9), _between(rng, 16, 200000 // seqs)
    elif kind == "chunk":
        seqs = min(seqs, 8)
        q = _between(rng, 9, 1024)
        ctx = q + _between(rng, 1, 40000 // seqs)
    else:
        seqs = min(seqs, 4)
        q = ctx = _between(rng, 100, 7000 // seqs)
    ctx_lo = max(q, ctx // rng.choice([1, 2, 8]))
    return dict(op=op, seqs=seqs, q=q, q_lo=max(1, q // rng.choice([1, 2])), ctx=max(ctx, ctx_lo),
                ctx_lo=ctx_lo, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page,
                window=rng.choice([0, 0, 0, _between(rng, 16, 5000)]), lse=rng.random() < 0.5)


def _spread(n, most, least):
    """n whole numbers from least to most, in a mixed order."""
    return [most - int((b * 29 % n) / max(1, n - 1) * (most - least)) for b in range(n)]


def lengths(case):
    """The new tokens and the whole lengths (new tokens among them) of the sequences of a case."""
    q = _spread(case["seqs"], case["q"], case["q_lo"])
    ctx = _spread(case["seqs"], case["ctx"], case["ctx_lo"])
    return q, [max(c, k) for c, k in zip(ctx, q)]


# ------------------------------------------------------------------ what a program has in hand
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _prefix(v):
    return _ints([0] + torch.tensor(v).cumsum(0).tolist())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"pages": _prepare_pages, "verify": _prepare_verify}.get(case["op"], _prepare_cache)(case, g)


def _prepare_pages(case, g):
    """A pool in the middle of its life: shuffled pages, sequences in arbitrary rows."""
    s, page, rows, cols = dict(case), case["page"], case["max_seqs"], case["max_pages"]
    q = _spread(case["seqs"], case["q"], case["q_lo"])
    ctx = _spread(case["seqs"], case["ctx"], case["ctx_lo"])
    held = torch.zeros(rows, dtype=torch.int64, device="cuda")
    s["seqs"] = torch.randperm(rows, generator=g, device="cuda")[:len(q)].int()
    held[s["seqs"].long()] = _ints(ctx, torch.int64)
    s["q_lens"], s["rows"] = _ints(q), sum(q)
    need = (held + page - 1) // page
    used = int(need.sum())
    s["pages"] = used + sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, q)) + 5
    order = torch.randperm(s["pages"], generator=g, device="cuda").int()
    col = torch.arange(cols, device="cuda")
    at = (need.cumsum(0) - need)[:, None] + col
    s["table"] = torch.where(col < need[:, None], order[at.clamp(max=s["pages"] - 1)], -1).int()
    s["lens"] = held.int()
    s["free"] = torch.cat([order[used:], torch.full((used,), -1, dtype=torch.int32, device="cuda")])
    s["count"] = _ints([s["pages"] - used])
    if own:
        import trellis_quantized_moe_exl3_gb300 as moe
        pool = s["pool"] = moe.PagePool(s["pages"], page, rows, cols)
        for x in ("table", "lens", "free", "count"):
            getattr(pool, x).copy_(s[x])
    return s


def _prepare_verify(case, g):
    """Probabilities of a target and of a drafting model that is often right."""
    s, v, dt = dict(case), case["vocab"], DTYPES[case["dtype"]]
    d = _spread(case["seqs"], case["drafts"], case["drafts_lo"])
    n = sum(d)
    logits = torch.randn(n + len(d), v, generator=g, device="cuda") * 2.5
    # (one token stands out, as after a prompt that says what comes)
    more = 5 * torch.rand(len(logits), 1, generator=g, device="cuda")
    logits.scatter_add_(1, logits.argmax(-1, keepdim=True), more)
    s["p"] = logits.softmax(-1).to(dt)
    s["cu_draft"] = _prefix(d)
    # the target's row of every drafted token
    seq = torch.repeat_interleave(torch.arange(len(d), device="cuda"), _ints(d, torch.int64))
    row = torch.arange(n, device="cuda") + seq
    near = logits[row] if n else logits[:0]
    near = (near + torch.randn(n, v, generator=g, device="cuda")).softmax(-1).to(dt)
    s["q"] = near if case["given"] else None
    s["draft"] = torch.multinomial(near.float(), 1, generator=g)[:, 0].int() if n else _ints([])
    s["accept_u"] = torch.rand(n, generator=g, device="cuda")
    s["sample_u"] = torch.rand(len(d), generator=g, device="cuda")
    return s


def _prepare_cache(case, g):
    dt, d, page, hk = DTYPES[case["dtype"]], case["dim"], case["page"], case["kv_heads"]
    s = dict(case)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    q, ctx = lengths(case)
    t, most = sum(q), max(-(-c // page) for c in ctx)
    need = _ints([-(-c // page) for c in ctx], torch.int64)
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    col = torch.arange(most, device="cuda")
    at = (need.cumsum(0) - need)[:, None] + col
    s["block_table"] = torch.where(col < need[:, None], order[at.clamp(max=pages - 1)], -1).int()
    s["cu_q"], s["seq_lens"] = _prefix(q), _ints(ctx)
    s["max_q"], s["longest"] = max(q), most * page
    for x in "kv":
        c = torch.randn(pages, page, hk, d, generator=g, device="cuda")
        c *= 1 + 3 * (torch.rand(pages, 1, hk, 1, generator=g, device="cuda") < 0.1)
        top = c.abs().amax((1, 3))
        # (what other programs write has any scale, what append writes a power of two)
        scale = top / TOP if case["op"] == "attention" else _power_of_two(top)
        s[x + "_scale"] = scale
        s[x + "_cache"] = (c / scale[:, None, :, None]).clamp_(-TOP, TOP).to(E4M3)
    if case["op"] == "append":
        r = case["rot"]
        s["inv_freq"] = 500000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
        s["q_weight"] = (1 + normal(d, std=0.1)).to(dt) if case["norm"] else None
        s["k_weight"] = (1 + normal(d, std=0.1)).to(dt) if case["norm"] else None
        s["q"], s["k"], s["v"] = normal(t, case["heads"] + 2 * hk, d).split([case["heads"], hk, hk], 1)
    else:
        s["q"] = normal(t, case["heads"], d)
        s["scale"] = d ** -0.5
    if own:
        import trellis_quantized_moe_exl3_gb300 as moe
        s["cache"] = moe.PagedKVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["batch"] = moe.PagedBatch(s["cu_q"], s["seq_lens"], s["block_table"], max_q=s["max_q"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"pages": _pages, "append": _append, "attention": _attention, "verify": _verify}[s["op"]](s)


def _pages(s):
    """A step begun and taken back whole, as one that is cancelled: the pool is as before."""
    if own:
        pool = s["pool"]
        step = pool.extend(s["seqs"], s["q_lens"], max_q=s["q"], max_tokens=s["rows"])
        pool.trim(s["seqs"], s["q_lens"])
        return {"cu_q": step.cu_q, "seq_lens": step.seq_lens, "block_table": step.block_table,
                "positions": step.positions, "slots": step.slots, "table": pool.table,
                "lens": pool.lens, "free": pool.free, "count": pool.count}
    page, seqs, q = s["page"], s["seqs"].long(), s["q_lens"].long()
    old = s["lens"].long()[seqs]
    cu = torch.cat([q.new_zeros(1), q.cumsum(0)])
    have, want = (old + page - 1) // page, (old + q + page - 1) // page
    first = (want - have).cumsum(0) - (want - have)
    col = torch.arange(s["max_pages"], device="cuda")
    taken = s["count"] - 1 - first[:, None] - (col - have[:, None])
    new = s["free"][taken.clamp(0, s["pages"] - 1).long()]
    own_row = s["table"][seqs]
    step = torch.where(col < have[:, None], own_row, torch.where(col < want[:, None], new, -1)).int()
    t = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = old[seq] + t - cu[seq]
    slots = step[seq, pos // page].long() * page + pos % page
    # (everything that was taken goes back to where it was)
    return {"cu_q": cu.int(), "seq_lens": (old + q).int(), "block_table": step, "positions": pos.int(),
            "slots": slots, "table": s["table"].clone(), "lens": s["lens"].clone(),
            "free": s["free"].clone(), "count": s["count"].clone()}


def _power_of_two(top):
    """The least 2^e with top <= 448 * 2^e, e within the range of scales."""
    m, e = torch.frexp(top.clamp(min=TOP * 2.0 ** LEAST))
    e = torch.where(m <= TOP / 512, e - 9, e - 8).clamp(LEAST, MOST)
    return torch.ldexp(torch.ones_like(top), e)


def _append(s):
    if own:
        import trellis_quantized_moe_exl3_gb300 as moe
        q = moe.kv_append(s["cache"], s["batch"], s["k"], s["v"], inv_freq=s["inv_freq"],
                          k_weight=s["k_weight"], q=s["q"], q_weight=s["q_weight"], eps=EPS,
                          interleaved=s["inter"])
        return {"q": q, **{x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")}}
    page, table = s["page"], s["block_table"].long()
    seq, pos = _places(s)
    block, place = table[seq, pos // page], pos % page
    # blocks that hold older tokens, and how many of them
    cu, lens = s["cu_q"].long(), s["seq_lens"].long()
    start = lens - (cu[1:] - cu[:-1])
    older = table.gather(1, (start // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    older, count = older[start % page > 0], (start % page)[start % page > 0]
    k = _plain_norm_rope(s["k"], pos, s, s["k_weight"])
    for x, new in (("k", k), ("v", s["v"].float())):
        cache, scale = s[x + "_cache"].view(torch.uint8), s[x + "_scale"]
        top = torch.zeros_like(scale).scatter_reduce_(0, block[:, None].expand(new.shape[:2]),
                                                      new.abs().amax(-1), "amax")
        old = torch.zeros_like(scale)
        old[older] = scale[older]
        grown = torch.where((old > 0) & (top <= TOP * old), old, _power_of_two(top))
        held = cache[older]
        turned = held.view(E4M3).float() * (old / grown)[older][:, None, :, None]
        turned = turned.to(E4M3).view(torch.uint8)
        move = (torch.arange(page, device="cuda") < count[:, None])[:, :, None, None]
        cache[older] = torch.where(move, turned, held)
        scale[block] = grown[block]
        new = (new / grown[block][..., None]).clamp(-TOP, TOP)
        cache[block, place] = new.to(E4M3).view(torch.uint8)
    q = _plain_norm_rope(s["q"], pos, s, s["q_weight"]).to(s["q"].dtype)
    return {"q": q, **{x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")}}


def _attention(s):
    if own:
        import trellis_quantized_moe_exl3_gb300 as moe
        got = moe.paged_attention(s["q"], s["cache"], s["batch"], scale=s["scale"], causal=True,
                                  window=s["window"], return_lse=s["lse"])
        return {"out": got[0], "lse": got[1]} if s["lse"] else {"out": got}
    # padded to the longest sequence and the most new tokens
    q, (n, _), hk, d = s["q"], s["block_table"].shape, s["kv_heads"], s["dim"]
    seq, pos = _places(s)
    row = torch.arange(len(seq), device="cuda") - s["cu_q"].long()[seq]
    group, most = s["heads"] // hk, s["max_q"]
    padded = torch.zeros(n, most, hk, group, d, device="cuda")
    padded[seq, row] = q.float().view(-1, hk, group, d)
    at = torch.full((n, most), -1, device="cuda")
    at[seq, row] = pos
    keys = torch.arange(s["longest"], device="cuda")
    seen = (keys <= at[..., None]) & (keys < s["seq_lens"][:, None, None])
    if s["window"]:
        seen &= keys > at[..., None] - s["window"]
    pages = s["block_table"].long().clamp(min=0)
    held = (keys < s["seq_lens"][:, None])[:, None, :, None]
    k, v = ((s[x + "_cache"][pages].float() * s[x + "_scale"][pages][:, :, None, :, None])
            .flatten(1, 2).transpose(1, 2) for x in "kv")                 # [n, hk, keys, d]
    mine = padded.permute(0, 2, 1, 3, 4).flatten(2, 3)                    # [n, hk, most * group, d]
    score = (mine @ k.transpose(2, 3)).mul_(s["scale"]).view(n, hk, most, group, -1)
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = (score.flatten(2, 3) @ v.masked_fill(~held, 0.0)).view(n, hk, most, group, d)
    o = (o / total.clamp(min=1e-30)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [n, most, heads, d]
    out = o[seq, row].to(q.dtype)
    lse = (top + total.log())[..., 0].permute(0, 2, 1, 3).flatten(2, 3)[seq, row]
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}


def _verify(s):
    if own:
        import trellis_quantized_moe_exl3_gb300 as moe
        tokens, accepted, dropped = moe.verify_drafts(s["p"], s["draft"], s["cu_draft"], s["accept_u"],
                                                      s["sample_u"], q=s["q"])
        return {"tokens": tokens, "accepted": accepted, "dropped": dropped}
    p, q, cu, x = s["p"], s["q"], s["cu_draft"].long(), s["draft"].long()
    n, d = len(cu) - 1, cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), d, output_size=len(x))
    i = torch.arange(len(x), device="cuda")
    # (a product of two 24-bit values is exact in 64 bits)
    chance = q[i, x].double() if q is not None else 1.0
    kept = s["accept_u"].double() * chance < p[i + seq, x].double()
    accepted = d.clone().scatter_reduce_(0, seq, torch.where(kept, d[seq], i - cu[seq]), "amin")
    row = cu[:-1] + torch.arange(n, device="cuda") + accepted
    left = p[row].double()                                    # long sums and their borders: 64 bits
    if len(x):
        at = (cu[:-1] + accepted).clamp(max=len(x) - 1)
        again = (accepted < d)[:, None]
        if q is not None:
            rest = left - torch.where(again, q[at].double(), 0.0)
        else:
            rest = left.scatter(1, x[at][:, None], torch.where(again, 0.0, left.gather(1, x[at][:, None])))
        rest = rest.clamp(min=0.0)
        left = torch.where(rest.sum(-1, keepdim=True) > 0, rest, left)
    below = left.cumsum(-1)
    drawn = (below <= s["sample_u"].double()[:, None] * below[:, -1:]).sum(-1)
    tokens = torch.full((len(x) + n,), -1, dtype=torch.int32, device="cuda")
    tokens[i + seq] = torch.where(i - cu[seq] < accepted[seq], x, -1).int()
    tokens[row] = drawn.int()
    return {"tokens": tokens, "accepted": accepted.int(), "dropped": (d - accepted).int()}


def _places(s):
    """The sequence and the position of every new token."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    cu = s["cu_q"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, s["seq_lens"].long()[seq] - (cu[seq + 1] - t)


def _plain_norm_rope(x, positions, s, weight):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = positions.double()[:, None, None] * s["inv_freq"]  # far positions: 32 bits would lose the angle
    c, n, r = angle.cos().float(), angle.sin().float(), s["rot"]
    if s["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * c - b * n, a * n + b * c], -1)
    return torch.cat([turned, x[..., r:]], -1)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "pages":
        q = _spread(case["seqs"], case["q"], case["q_lo"])
        ctx = _spread(case["seqs"], case["ctx"], case["ctx_lo"])
        held = sum(-(-(c + n) // case["page"]) for c, n in zip(ctx, q))
        n = 4 * (held + case["seqs"] * case["max_pages"] + 7 * case["seqs"]) + 12 * sum(q)
        return {"bytes": n, "flops": n // 4}
    if case["op"] == "verify":
        d = _spread(case["seqs"], case["drafts"], case["drafts_lo"])
        size = 4 if case["dtype"] == "fp32" else 2
        # one row of each sequence is sampled from; one of the draft's where a draft was turned down
        rows = len(d) + (sum(n > 0 for n in d) if case["given"] else 0)
        return {"bytes": rows * case["vocab"] * size + 20 * sum(d) + 20 * len(d),
                "flops": 2 * rows * case["vocab"]}
    d, hq, hk = case["dim"], case["heads"], case["kv_heads"]
    q, ctx = lengths(case)
    blocks = [-(-c // case["page"]) - (c - n) // case["page"] for n, c in zip(q, ctx)]
    if case["op"] == "append":
        t = sum(q)
        return {"bytes": t * d * (4 * hq + 2 * hk * 3) + 4 * t + 16 * hk * sum(blocks),
                "flops": 8 * t * (hq + hk) * d + 4 * t * hk * d}
    keys = pairs = 0
    for n, c in zip(q, ctx):
        w = case["window"] or c
        keys += c - max(0, c - n - w + 1)
        full = max(0, min(n, c - w + 1)) if case["window"] else 0  # rows that see a whole window
        part = n - full                                            # rows that see every key up to their own
        pairs += full * w + (c - n + 1 + c - n + part) * part // 2
    bytes_ = keys * hk * d * 2 + keys // case["page"] * hk * 8 + 4 * sum(q) * hq * d
    return {"bytes": bytes_ + 4 * sum(q) * hq * case["lse"], "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"pages": _exact_pages, "verify": _exact_verify, "append": _exact_append,
            "attention": _exact_attention}[case["op"]](case, s)


def _exact_pages(case, s):
    page, table, lens = case["page"], s["table"].tolist(), s["lens"].tolist()
    stack = s["free"].tolist()[:int(s["count"])]
    cu, out, rows, at = [0], [], [], []
    for b, n in zip(s["seqs"].tolist(), s["q_lens"].tolist()):
        mine = [x for x in table[b] if x >= 0]
        while len(mine) * page < lens[b] + n:
            mine.append(stack.pop())
        for pos in range(lens[b], lens[b] + n):
            rows.append(pos)
            at.append(mine[pos // page] * page + pos % page)
        cu.append(cu[-1] + n)
        out.append((lens[b] + n, mine + [-1] * (case["max_pages"] - len(mine))))
    return {"cu_q": _ints(cu), "seq_lens": _ints([x for x, _ in out]),
            "block_table": _ints([x for _, x in out]), "positions": _ints(rows),
            "slots": _ints(at, torch.int64), "table": s["table"], "lens": s["lens"], "free": s["free"],
            "count": s["count"]}


def _exact_verify(case, s):
    cu, p, q = s["cu_draft"].tolist(), s["p"], s["q"]
    tokens, accepted = [], []
    for b in range(len(cu) - 1):
        d, a = cu[b + 1] - cu[b], 0
        rows = p[cu[b] + b:cu[b + 1] + b + 1].double()
        while a < d:
            x = int(s["draft"][cu[b] + a])
            have, said = float(rows[a, x]), float(q[cu[b] + a, x]) if q is not None else 1.0
            # u < have / said, with nothing over nothing as 0
            if have == 0 or (said > 0 and float(s["accept_u"][cu[b] + a]) >= have / said):
                break
            tokens.append(x)
            a += 1
        weight = rows[a]
        if a < d:
            minus = torch.zeros_like(weight)
            if q is not None:
                minus = q[cu[b] + a].double()
            else:
                x = int(s["draft"][cu[b] + a])
                minus[x] = weight[x]
            more = torch.relu(weight - minus)
            weight = more if bool(more.any()) else weight
        line = torch.cumsum(weight, 0)
        want = float(s["sample_u"][b]) * float(line[-1])
        tokens += [int(torch.searchsorted(line, want, right=True))] + [-1] * (d - a)
        accepted.append(a)
    d = [cu[b + 1] - cu[b] - a for b, a in enumerate(accepted)]
    return {"tokens": _ints(tokens), "accepted": _ints(accepted), "dropped": _ints(d)}


def _spans(case):
    q, ctx = lengths(case)
    at = 0
    for n, c in zip(q, ctx):
        yield at, at + n, c - n, c
        at += n


def _exact_append(case, s):
    """Scales exactly; values before their rounding to 8 bits, in units of their block's scale."""
    page, spans = case["page"], list(_spans(case))
    pos = torch.cat([torch.arange(a, b, dtype=torch.float64, device="cuda") for _, _, a, b in spans])
    res = {"q": _rotated(s, s["q"], pos, s["q_weight"])}
    for x, new in (("k", _rotated(s, s["k"], pos, s["k_weight"])), ("v", s["v"].double())):
        cache, scale = s[x + "_cache"].double(), s[x + "_scale"].double()
        for b, (i, j, p0, p1) in enumerate(spans):
            for blk in range(p0 // page, -(-p1 // page)):
                lo, hi = max(p0, blk * page), min(p1, (blk + 1) * page)
                at, mine = int(s["block_table"][b, blk]), new[i + lo - p0:i + hi - p0]
                old = scale[at].clone() if lo > blk * page else torch.zeros_like(scale[at])
                want = torch.ceil(torch.log2(mine.abs().amax((0, 2)) / TOP)).clamp(LEAST, MOST)
                grown = torch.maximum(old, torch.exp2(want))
                cache[at, :lo - blk * page] *= (old / grown)[:, None]
                cache[at, lo - blk * page:hi - blk * page] = mine / grown[:, None]
                scale[at] = grown
        res[x + "_cache"], res[x + "_scale"] = cache, scale
    return res


def _exact_attention(case, s):
    hk, group, page = case["kv_heads"], case["heads"] // case["kv_heads"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, (i, j, p0, p1) in enumerate(_spans(case)):
        p = torch.arange(p0, p1, device="cuda")[:, None]
        key = torch.arange(p1, device="cuda")
        at, place = s["block_table"][b].long()[key // page], key % page
        hidden = (key[None] > p) | ((key[None] <= p - case["window"]) if case["window"] else False)
        for h in range(hk):
            k, v = (s[x + "_cache"][at, place, h].double() * s[x + "_scale"][at, h].double()[:, None]
                    for x in "kv")
            for m in range(h * group, (h + 1) * group):
                z = torch.einsum("id,jd->ij", s["q"][i:j, m].double(), k) * s["scale"]
                z = z.masked_fill_(hidden, -math.inf)
                total = torch.logsumexp(z, -1)
                lse[i:j, m] = total
                out[i:j, m] = z.sub_(total[:, None]).exp_() @ v
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _rotated(s, x, positions, weight):
    x, r = x.double(), s["rot"]
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    i = torch.arange(r // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if s["inter"] else (i, i + r // 2)
    z = torch.complex(x[..., first], x[..., second])
    z = z * torch.polar(torch.ones_like(s["inv_freq"]), positions[:, None] * s["inv_freq"])[:, None]
    res = x.clone()
    res[..., first], res[..., second] = z.real, z.imag
    return res
