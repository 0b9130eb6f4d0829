"""Plain 64-bit forms of the attention operators, and seeded step data.

The references follow the formulas of include/exl3.h with float64 torch
operations on the CPU, one sequence and head at a time."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

E4M3 = torch.float8_e4m3fn
# Half a step of each type's rounding, relative to the value.
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, E4M3: 2.0 ** -4}


def rotate(x, positions, inv_freq, interleaved):
    """x [..., T, H, D] float64, positions [T]."""
    if inv_freq is None:
        return x
    r = 2 * len(inv_freq)
    # a float64 product of a position below 2^31 and a frequency of at most 1
    # is off by at most 2^-53 * 2^31 radians
    ang = positions.double()[:, None] * inv_freq.double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, a * s + b * c
    return y


def norm_rope(x, positions, inv_freq, weight, eps, interleaved):
    x = x.double().cpu()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double().cpu()
    return rotate(x, positions.cpu(), inv_freq.cpu() if inv_freq is not None else None, interleaved)


@dataclass
class Step:
    cu_q: torch.Tensor
    seq_lens: torch.Tensor
    table: torch.Tensor
    max_q: int
    qs: list
    lens: list


def make_step(g, qs, lens, page, spare=3, pad=0):
    """Device tensors of a step over shuffled pages; unused table entries are
    out of range on purpose."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(qs), max(need + [1]) + 1), 1 << 30, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = torch.tensor([0] + torch.tensor(qs).cumsum(0).tolist(), dtype=torch.int32)
    return Step(cu.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), max(qs),
                qs, lens), pages


def attention(q, k, v, table, qs, lens, page, scale, causal, window):
    """q [T, H, D]; k, v [pages, page, Hk, D] float64 values (CPU).  Returns
    out, sum of p |v| (what rounding errors of p are measured against) and lse."""
    q = q.double().cpu()
    T, H, D = q.shape
    hk = k.shape[2]
    grp = H // hk
    out, mag = torch.zeros(T, H, D, dtype=torch.float64), torch.zeros(T, H, D, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    t0 = 0
    for b, (n, L) in enumerate(zip(qs, lens)):
        if n and L:
            ids = table[b, torch.arange(L) // page].long()
            kk, vv = k[ids, torch.arange(L) % page], v[ids, torch.arange(L) % page]
            pos = torch.arange(L - n, L)[:, None]
            key = torch.arange(L)[None]
            seen = (key <= pos) if causal else torch.ones(n, L, dtype=torch.bool)
            if window:
                seen = seen & (key > pos - window)
            for h in range(H):
                s = q[t0:t0 + n, h] @ kk[:, h // grp].T * scale
                s = torch.where(seen, s, -math.inf)
                m = s.amax(-1, keepdim=True)
                ok = m.isfinite()[:, 0]
                p = torch.where(seen, (s - torch.where(m.isfinite(), m, 0.0)).exp(), 0.0)
                l = p.sum(-1, keepdim=True)
                p = p / torch.where(l > 0, l, 1.0)
                # a key that is not seen does not count, whatever its value
                vh = vv[:, h // grp]
                if vh.isfinite().all():
                    out[t0:t0 + n, h] = p @ vh
                    mag[t0:t0 + n, h] = p @ vh.abs()
                else:
                    prod = torch.where(seen[..., None], p[..., None] * vh, 0.0)
                    out[t0:t0 + n, h] = prod.sum(1)
                    mag[t0:t0 + n, h] = prod.abs().sum(1)
                lse[t0:t0 + n, h] = torch.where(ok, m[:, 0] + l[:, 0].log(), -math.inf)
        t0 += n
    return out, mag, lse
