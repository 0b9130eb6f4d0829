"""One decoder layer: attention over a paged cache, then the coded MoE layer.

    block = DecoderBlock(moe, router, w_qkv, w_out, heads, kv_heads, top_k=8, inv_freq=f,
                         q_norm=wq, k_norm=wk)
    y = block(x, cache, batch)        # x [tokens, hidden], new tokens of every sequence

The new tokens may be prompts, chunks of prompts, drafted tokens and single
tokens of different sequences at once.  The dense projections are plain
library products; everything else is the library's kernels.
"""
from __future__ import annotations

import torch

from .api import Layer, rmsnorm
from .attention import PagedBatch, PagedKVCache, kv_append, paged_attention


class DecoderBlock:
    """moe: the coded layer; router [hidden, experts], w_qkv [hidden, (heads +
    2 kv_heads) * head_dim], w_out [heads * head_dim, hidden], all of the
    activations' type; q_norm, k_norm [head_dim] or None; inv_freq as in
    qk_norm_rope, or None."""

    def __init__(self, moe: Layer, router, w_qkv, w_out, heads: int, kv_heads: int, top_k: int,
                 inv_freq=None, q_norm=None, k_norm=None, eps: float = 1e-6,
                 interleaved: bool = False, window: int = 0):
        self.moe, self.router, self.w_qkv, self.w_out = moe, router, w_qkv, w_out
        self.heads, self.kv_heads, self.top_k = heads, kv_heads, top_k
        self.head_dim = w_out.shape[0] // heads
        if w_qkv.shape[1] != (heads + 2 * kv_heads) * self.head_dim:
            raise ValueError(f"w_qkv has {w_qkv.shape[1]} columns, expected "
                             f"{(heads + 2 * kv_heads) * self.head_dim}")
        self.inv_freq, self.q_norm, self.k_norm = inv_freq, q_norm, k_norm
        self.eps, self.interleaved, self.window = eps, interleaved, window

    def attend(self, x, cache: PagedKVCache, batch: PagedBatch):
        """x + attention(norm(x)); appends the new tokens to the cache."""
        T = x.shape[0]
        qkv = (rmsnorm(x, self.eps) @ self.w_qkv).view(T, -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        q = kv_append(cache, batch, k, v, inv_freq=self.inv_freq, k_weight=self.k_norm, q=q,
                      q_weight=self.q_norm, eps=self.eps, interleaved=self.interleaved)
        a = paged_attention(q, cache, batch, window=self.window)
        return torch.addmm(x, a.view(T, -1), self.w_out)

    def __call__(self, x, cache: PagedKVCache, batch: PagedBatch):
        x = self.attend(x, cache, batch)
        h = rmsnorm(x, self.eps)
        return self.moe.forward(h, (h @ self.router).float(), self.top_k, residual=x)
