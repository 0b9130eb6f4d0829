"""The operators of attention over a paged key/value cache, as they are measured.

Three operators of the serving step that surrounds a mixture-of-experts layer:

  norm_rope  RMS norm of every query and key head and the position rotation, in one pass
  append     the same for new tokens, whose keys and values go to a paged cache on the way
  attention  attention of new tokens (one, a few, a chunk, a whole prompt) over that cache

A case is a dict of plain values.  ``run`` computes the plain form, or, where ``own`` is true, calls
the package.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one step of a small decode batch: launch latency is everything
        dict(name="norm_rope_decode", op="norm_rope", tokens=8, heads=32, kv_heads=8, dim=128,
             rot=128, inter=False, norm=True, dtype="bf16", pos=100000),
        # a prompt out of one fused projection, half of every head rotated, neighbouring pairs
        dict(name="norm_rope_prompt", op="norm_rope", tokens=7168, heads=32, kv_heads=8, dim=128,
             rot=64, inter=True, norm=True, dtype="bf16", pos=0),
        # a decode batch: one token of each of 64 sequences goes to an 8-bit cache
        dict(name="append_decode_e4m3", op="append", seqs=64, q=1, q_lo=1, ctx=2000, ctx_lo=100,
             heads=32, kv_heads=8, dim=128, rot=128, inter=False, norm=True, dtype="bf16",
             cache="e4m3", page=64),
        # ragged prompts that continue earlier context, 16-bit cache
        dict(name="append_prompt", op="append", seqs=5, q=2047, q_lo=700, ctx=4000, ctx_lo=2048,
             heads=32, kv_heads=8, dim=128, rot=128, inter=False, norm=True, dtype="bf16",
             cache="bf16", page=16),
        # one user, short context: the smallest call
        dict(name="decode_one", op="attention", seqs=1, q=1, q_lo=1, ctx=1000, ctx_lo=1000,
             heads=32, kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=16, window=0, lse=False),
        # a decode batch with ragged contexts
        dict(name="decode_batch", op="attention", seqs=64, q=1, q_lo=1, ctx=8000, ctx_lo=500,
             heads=32, kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=64, window=0, lse=False),
        # few sequences, long contexts, 8-bit cache: the work of one head is split over the GPU
        dict(name="decode_long_e4m3", op="attention", seqs=4, q=1, q_lo=1, ctx=131071, ctx_lo=90001,
             heads=32, kv_heads=4, dim=128, dtype="bf16", cache="e4m3", page=64, window=0, lse=True),
        # four drafted tokens checked at once
        dict(name="verify_4", op="attention", seqs=16, q=4, q_lo=4, ctx=6001, ctx_lo=1003,
             heads=32, kv_heads=8, dim=64, dtype="fp16", cache="fp16", page=32, window=0, lse=False),
        # a chunk of a long prompt
        dict(name="chunk_512", op="attention", seqs=2, q=512, q_lo=512, ctx=16384, ctx_lo=9000,
             heads=32, kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=64, window=0, lse=True),
        # chunks of odd lengths over an 8-bit cache
        dict(name="chunk_e4m3", op="attention", seqs=6, q=333, q_lo=65, ctx=8191, ctx_lo=2000,
             heads=32, kv_heads=8, dim=128, dtype="bf16", cache="e4m3", page=16, window=0, lse=False),
        # a whole prompt
        dict(name="prompt_7168", op="attention", seqs=1, q=7168, q_lo=7168, ctx=7168, ctx_lo=7168,
             heads=32, kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=64, window=0, lse=True),
        # two prompts of a layer that looks back over a window
        dict(name="prompt_window", op="attention", seqs=2, q=8192, q_lo=5000, ctx=8192, ctx_lo=5000,
             heads=32, kv_heads=8, dim=64, dtype="fp16", cache="fp16", page=64, window=1024, lse=False),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads, kv_heads = rng.choice([(32, 8), (32, 4), (16, 2), (24, 8), (8, 8), (28, 4), (40, 8)])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    op = rng.choice(["norm_rope", "append", "attention", "attention", "attention"])
    if op == "norm_rope":
        return dict(op=op, tokens=_between(rng, 1, 16384), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), inter=rng.random() < 0.5,
                    norm=rng.random() < 0.8, dtype=dtype, pos=rng.randrange(0, 1 << 20))
    cache = rng.choice([dtype, dtype, "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    seqs = _between(rng, 1, 64)
    if op == "append":
        q = _between(rng, 1, max(1, 16384 // seqs))
        ctx_lo = q + rng.randrange(0, 2000)
        return dict(op=op, seqs=seqs, q=q, q_lo=max(1, q // rng.choice([1, 3])), ctx_lo=ctx_lo,
                    ctx=ctx_lo + rng.randrange(0, 1000), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), inter=rng.random() < 0.5,
                    norm=rng.random() < 0.8, dtype=dtype, cache=cache, page=page)
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
    q_lo = max(1, q // rng.choice([1, 2]))
    ctx_lo = max(q, ctx // rng.choice([1, 2, 8]))
    return dict(op=op, seqs=seqs, q=q, q_lo=q_lo, ctx=max(ctx, ctx_lo), ctx_lo=ctx_lo, heads=heads,
                kv_heads=kv_heads, dim=dim, dtype=dtype, cache=cache, page=page,
                window=rng.choice([0, 0, 0, _between(rng, 16, 5000)]), lse=rng.random() < 0.5)


def lengths(case):
    """The new tokens and the whole lengths (new tokens among them) of the sequences of a case."""
    n = case["seqs"]
    at = [(b * 29 % n) / max(1, n - 1) for b in range(n)]
    q = [case["q"] - int(a * (case["q"] - case["q_lo"])) for a in at]
    ctx = [case["ctx"] - int(a * (case["ctx"] - case["ctx_lo"])) for a in at]
    return q, [max(c, k) for c, k in zip(ctx, q)]


# ------------------------------------------------------------------ what a program has in hand
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d = DTYPES[case["dtype"]], case["dim"]
    s = dict(case)

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device="cuda")

    if "rot" in case:
        r = case["rot"]
        s["inv_freq"] = 500000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
        s["q_weight"] = (1 + normal(d, std=0.1)).to(dt) if case["norm"] else None
        s["k_weight"] = (1 + normal(d, std=0.1)).to(dt) if case["norm"] else None
    if case["op"] == "norm_rope":
        t = case["tokens"]
        qkv = normal(t, case["heads"] + 2 * case["kv_heads"], d)
        s["q"], s["k"] = qkv[:, :case["heads"]], qkv[:, case["heads"]:case["heads"] + case["kv_heads"]]
        first = int(torch.randint(0, 1000, (1,), generator=g, device="cuda")) + case["pos"]
        s["positions"] = torch.arange(first, first + t, dtype=torch.int32, device="cuda")
        return s
    q, ctx = lengths(case)
    t, page, hk = sum(q), case["page"], case["kv_heads"]
    most = max(-(-c // page) for c in ctx)
    pages = sum(-(-c // page) for c in ctx) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.full((len(q), most), -1, dtype=torch.int32, device="cuda"), 0
    for b, c in enumerate(ctx):
        n = -(-c // page)
        table[b, :n] = order[at:at + n]
        at += n
    s["cu_q"] = ints([0] + torch.tensor(q).cumsum(0).tolist())
    s["seq_lens"], s["block_table"] = ints(ctx), table
    s["max_q"], s["max_len"], s["longest"] = max(q), max(ctx), most * page
    eight = case["cache"] == "e4m3"
    for x in ("k", "v"):
        scale = 0.01 + 0.01 * torch.rand(hk, generator=g, device="cuda") if eight else None
        c = torch.randn(pages, page, hk, d, generator=g, device="cuda")
        if eight:
            c.div_(scale[:, None]).clamp_(-E4M3_MAX, E4M3_MAX)
        s[x + "_cache"], s[x + "_scale"] = c.to(DTYPES[case["cache"]]), scale
    if case["op"] == "append":
        qkv = normal(t, case["heads"] + 2 * hk, d)
        s["q"], s["k"], s["v"] = qkv.split([case["heads"], hk, hk], dim=1)
    else:
        s["q"] = normal(t, case["heads"], d)
        s["scale"] = d ** -0.5
    if own:
        import trellis_quantized_moe_exl3_gb300 as moe
        s["cache_handle"] = moe.PagedKVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["batch"] = moe.PagedBatch(s["cu_q"], s["seq_lens"], s["block_table"], max_q=s["max_q"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"norm_rope": _norm_rope, "append": _append, "attention": _attention}[s["op"]](s)


def _norm_rope(s):
    if own:
        import trellis_quantized_moe_exl3_gb300 as moe
        q, k = moe.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
                                k_weight=s["k_weight"], eps=EPS, interleaved=s["inter"])
        return {"q": q, "k": k}
    return {x: _plain_norm_rope(s[x], s["positions"], s, s[x + "_weight"]).to(s[x].dtype) for x in "qk"}


def _append(s):
    if own:
        import trellis_quantized_moe_exl3_gb300 as moe
        q = moe.kv_append(s["cache_handle"], s["batch"], s["k"], s["v"], inv_freq=s["inv_freq"],
                          k_weight=s["k_weight"], q=s["q"], q_weight=s["q_weight"], eps=EPS,
                          interleaved=s["inter"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    seq, pos = _places(s)
    page = s["block_table"][seq, pos // s["page"]].long()
    k = _plain_norm_rope(s["k"], pos, s, s["k_weight"])
    for x, new in (("k", k), ("v", s["v"].float())):
        cache = s[x + "_cache"]
        if s[x + "_scale"] is not None:
            new = (new / s[x + "_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype).view(torch.uint8)
            cache = cache.view(torch.uint8)
        cache[page, pos % s["page"]] = new.to(cache.dtype)
    q = _plain_norm_rope(s["q"], pos, s, s["q_weight"]).to(s["q"].dtype)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attention(s):
    if own:
        import trellis_quantized_moe_exl3_gb300 as moe
        got = moe.paged_attention(s["q"], s["cache_handle"], s["batch"], scale=s["scale"], causal=True,
                                  window=s["window"], return_lse=s["lse"])
        return {"out": got[0], "lse": got[1]} if s["lse"] else {"out": got}
    return _plain_attention(s)


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


def _plain_attention(s):
    """Padded to the longest sequence and the most new tokens; one key/value head at a time."""
    q, (n, _), hk, d = s["q"], s["block_table"].shape, s["kv_heads"], s["dim"]
    seq, pos = _places(s)
    row = torch.arange(len(seq), device="cuda") - s["cu_q"].long()[seq]
    group, most = s["heads"] // hk, s["max_q"]
    padded = torch.zeros(n, most, s["heads"], d, device="cuda")
    padded[seq, row] = q.float()
    at = torch.full((n, most), -1, device="cuda")
    at[seq, row] = pos
    keys = torch.arange(s["longest"], device="cuda")
    seen = (keys <= at[..., None]) & (keys < s["seq_lens"][:, None, None])
    if s["window"]:
        seen &= keys > at[..., None] - s["window"]
    pages = s["block_table"].long().clamp(min=0)
    held = (keys < s["seq_lens"][:, None])[..., None]
    out = torch.empty(len(seq), s["heads"], d, dtype=q.dtype, device="cuda")
    lse = torch.empty(len(seq), s["heads"], device="cuda")
    for h in range(hk):
        k, v = (s[x + "_cache"][:, :, h].float()[pages].flatten(1, 2) for x in "kv")
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"][h], v * s["v_scale"][h]
        mine = padded[:, :, h * group:(h + 1) * group].flatten(1, 2)
        score = (mine @ k.transpose(1, 2) * s["scale"]).view(n, most, group, -1)
        score.masked_fill_(~seen[:, :, None], -math.inf)
        top = score.amax(-1, keepdim=True).clamp(min=-1e30)
        score = score.sub_(top).exp_()
        total = score.sum(-1, keepdim=True)
        o = (score.flatten(1, 2) @ torch.where(held, v, 0.0)).view(n, most, group, d)
        o = o / total.clamp(min=1e-30)
        out[:, h * group:(h + 1) * group] = o[seq, row].to(q.dtype)
        lse[:, h * group:(h + 1) * group] = (top + total.log())[seq, row, :, 0]
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    d, hq, hk = case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "norm_rope":
        n = case["tokens"] * (hq + hk) * d
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 8 * n}
    q, ctx = lengths(case)
    size = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        t = sum(q)
        return {"bytes": t * d * (4 * hq + 2 * hk * (2 + size)) + 4 * t, "flops": 8 * t * (hq + hk) * d}
    keys = pairs = 0
    for n, c in zip(q, ctx):
        w = case["window"] or c
        first = max(0, c - n - w + 1)
        keys += c - first
        full = max(0, min(n, c - w + 1))           # rows that see a whole window (or all)
        full = min(full, n) if case["window"] else 0
        part = n - full                            # rows that see every key up to their own
        pairs += full * w + sum((c - n + 1, c - n + part)) * part // 2
    bytes_ = keys * hk * d * 2 * size + 4 * sum(q) * hq * d + 4 * sum(q) * hq * case["lse"]
    return {"bytes": bytes_, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "norm_rope":
        return {x: _rotated(s, s[x], s["positions"].double(), s[x + "_weight"]) for x in "qk"}
    q, ctx = lengths(case)
    spans, at = [], 0
    for n, c in zip(q, ctx):
        spans.append((at, at + n, c - n, c))
        at += n
    if case["op"] == "append":
        pos = torch.cat([torch.arange(a, b, dtype=torch.float64, device="cuda") for _, _, a, b in spans])
        res = {"q": _rotated(s, s["q"], pos, s["q_weight"])}
        for x, new in (("k", _rotated(s, s["k"], pos, s["k_weight"])), ("v", s["v"].double())):
            cache = s[x + "_cache"].double()
            if s[x + "_scale"] is not None:
                new = new / s[x + "_scale"].double()[:, None]
            for b, (i, j, p0, p1) in enumerate(spans):
                flat = _slots(s, b, p1)[p0:]
                cache.view(-1, case["kv_heads"], case["dim"])[flat] = new[i:j].clamp(-E4M3_MAX, E4M3_MAX) \
                    if s[x + "_scale"] is not None else new[i:j]
            res[x + "_cache"] = cache
        return res
    hk, group = case["kv_heads"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, (i, j, p0, p1) in enumerate(spans):
        slots = _slots(s, b, p1)
        p = torch.arange(p0, p1, device="cuda")[:, None]
        key = torch.arange(p1, device="cuda")[None]
        hidden = (key > p) | ((key <= p - case["window"]) if case["window"] else False)
        for h in range(hk):
            k, v = (s[x + "_cache"].view(-1, hk, case["dim"])[:, h][slots].double() for x in "kv")
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for m in range(h * group, (h + 1) * group):
                z = torch.einsum("id,jd->ij", s["q"][i:j, m].double(), k) * s["scale"]
                z = z.masked_fill_(hidden, -math.inf)
                total = torch.logsumexp(z, -1)
                lse[i:j, m] = total
                out[i:j, m] = z.sub_(total[:, None]).exp_() @ v
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _slots(s, b, length):
    """Where the positions 0 .. length-1 of sequence b are held, counted over all pages."""
    p = torch.arange(length, device="cuda")
    return s["block_table"][b].long()[p // s["page"]] * s["page"] + p % s["page"]


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
