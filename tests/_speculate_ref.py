"""Plain forms of the speculative step's operators, and seeded data: a pool of
pages as Python lists, drafts decided in whole numbers, attention over a cache
with block scales in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, E4M3: 2.0 ** -4}
LEAST, MOST = 2.0 ** -40, 2.0 ** 40


# ------------------------------------------------------------ pages
class Pool:
    def __init__(self, pages, page, rows, cols):
        self.P, self.rows_n, self.cols = page, rows, cols
        self.held = [[] for _ in range(rows)]
        self.lens = [0] * rows
        self.free = list(range(pages - 1, -1, -1))
        self.status = 0

    def extend(self, seqs, q_lens, max_tokens):
        start = len(self.free)
        stack, asked, cu, lens, table = list(self.free), 0, [0], [], []
        pos, slots = [-1] * max_tokens, [-1] * max_tokens
        for i, (s, n) in enumerate(zip(seqs, q_lens)):
            ok = 0 <= s < self.rows_n and s not in seqs[:i] and n >= 0
            if not ok:
                self.status |= 1
            n = max(n, 0)
            old = self.lens[s] if ok else 0
            if ok and old + n > min(self.cols * self.P, 1 << 30):
                ok, self.status = False, self.status | 4
            need = -(-(old + n) // self.P) - -(-old // self.P) if ok else 0
            asked += need
            q0 = cu[-1]
            if ok and n and q0 + n > max_tokens:
                ok, self.status = False, self.status | 4
            if ok and need and asked > start:
                ok, self.status = False, self.status | 2
            self_q1 = min(q0 + n, max_tokens) if q0 + n <= max_tokens else max_tokens
            row = []
            if ok:
                for _ in range(need):
                    self.held[s].append(stack.pop())
                self.lens[s] += n
                row = self.held[s]
                for j in range(n):
                    p = old + j
                    pos[q0 + j] = p
                    slots[q0 + j] = row[p // self.P] * self.P + p % self.P
            cu.append(self_q1)
            lens.append(self.lens[s] if ok else 0)
            table.append(row + [-1] * (self.cols - len(row)))
        self.free = stack
        return cu, lens, table, pos, slots

    def trim(self, seqs, drop=None):
        back = []
        for i, s in enumerate(seqs):
            if not 0 <= s < self.rows_n or s in seqs[:i]:
                self.status |= 1
                continue
            n = self.lens[s] if drop is None else drop[i]
            if not 0 <= n <= self.lens[s]:
                self.status |= 1
                n = min(max(n, 0), self.lens[s])
            self.lens[s] -= n
            keep = -(-self.lens[s] // self.P)
            back += self.held[s][keep:]
            self.held[s] = self.held[s][:keep]
        self.free += back[::-1]

    def state(self):
        return ([r + [-1] * (self.cols - len(r)) for r in self.held], self.lens, self.free)


# ------------------------------------------------------------ verification
def fixed(x):
    """Probabilities rounded to units of 2^-46 (exact up to it: a product by a power of two)."""
    x = x.double().cpu().numpy()
    x = np.where(x > 0, np.minimum(x, 1.0), 0.0)
    return np.rint(x * 2.0 ** 46).astype(np.uint64)


def verify(p, draft, cu, accept_u, sample_u, q):
    tokens, accepted, dropped = [], [], []
    for b in range(len(cu) - 1):
        c, d, a = cu[b], cu[b + 1] - cu[b], 0
        while a < d:
            x = int(draft[c + a])
            if not 0 <= x < p.shape[1]:
                break
            # 24 bits times 24 bits: exact
            said = float(q[c + a, x]) if q is not None else 1.0
            if not float(accept_u[c + a]) * said < float(p[c + b + a, x]):
                break
            a += 1
        w = fixed(p[c + b + a])
        if a < d:
            if q is not None:
                m = fixed(q[c + a])
                rest = np.where(w > m, w - m, np.uint64(0))
            else:
                rest = w.copy()
                if 0 <= int(draft[c + a]) < len(rest):
                    rest[int(draft[c + a])] = 0
            w = rest if rest.any() else w
        line = np.cumsum(w, dtype=np.uint64)
        total = int(line[-1])
        want = int(float(sample_u[b]) * 2.0 ** 64) * total >> 64
        t = int(np.searchsorted(line, np.uint64(want), side="right")) if total else -1
        tokens += [int(draft[c + j]) for j in range(a)] + [t] + [-1] * (d - a)
        accepted.append(a)
        dropped.append(d - a)
    return tokens, accepted, dropped


# ------------------------------------------------------------ block scales
def scale_for(top):
    """The least power of two, 2^-40 .. 2^40, with top <= 448 * it (float64)."""
    m, e = math.frexp(max(top, 448 * LEAST))
    return min(2.0 ** (e - 9 if m <= 0.875 else e - 8), MOST)


def values(x, scale):
    """A block-scaled cache [pages, page, heads, dim] as float64 on the CPU."""
    s = scale.double().cpu().clamp(min=LEAST)
    return x.float().cpu().double() * s[:, None, :, None]


def attention(q, k, v, table, qs, lens, page, scale, causal, window, absent=None):
    """q [T, H, D]; k, v [pages, page, Hk, D] float64; absent [pages, Hk]: blocks
    whose keys do not count.  out, sum of p |v| and lse."""
    q = q.double().cpu()
    T, H, D = q.shape
    hk = k.shape[2]
    out, mag = torch.zeros(T, H, D, dtype=torch.float64), torch.zeros(T, H, D, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    t0 = 0
    for b, (n, L) in enumerate(zip(qs, lens)):
        if n and L:
            ids = table[b, torch.arange(L) // page].long()
            place = torch.arange(L) % page
            pos, key = torch.arange(L - n, L)[:, None], torch.arange(L)[None]
            seen0 = (key <= pos) if causal else torch.ones(n, L, dtype=torch.bool)
            if window:
                seen0 = seen0 & (key > pos - window)
            for h in range(H):
                g = h // (H // hk)
                seen = seen0 if absent is None else seen0 & ~absent[ids, g][None]
                s = torch.where(seen, q[t0:t0 + n, h] @ k[ids, place, g].T * scale, -math.inf)
                m = s.amax(-1, keepdim=True)
                w = torch.where(seen, (s - torch.where(m.isfinite(), m, 0.0)).exp(), 0.0)
                l = w.sum(-1, keepdim=True)
                w = w / torch.where(l > 0, l, 1.0)
                # what is not seen does not count, whatever it is
                used = seen.any(0)
                vh = torch.where(used[:, None], v[ids, place, g], 0.0)
                if vh.isfinite().all():
                    out[t0:t0 + n, h], mag[t0:t0 + n, h] = w @ vh, w @ vh.abs()
                else:
                    x = torch.where(seen[..., None], w[..., None] * vh, 0.0)
                    out[t0:t0 + n, h], mag[t0:t0 + n, h] = x.sum(1), x.abs().sum(1)
                lse[t0:t0 + n, h] = torch.where(m.isfinite()[:, 0], m[:, 0] + l[:, 0].log(), -math.inf)
        t0 += n
    return out, mag, lse
