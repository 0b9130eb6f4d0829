"""Attention over a paged key/value cache: Python API over the C ABI.

    cache = PagedKVCache(k, v)                              # [pages, page_size, kv_heads, dim]
    batch = PagedBatch(cu_q, seq_lens, block_table, max_q)  # the step's sequences
    q = kv_append(cache, batch, k_new, v_new, inv_freq=f, k_weight=wk, q=q_new, q_weight=wq)
    out = paged_attention(q, cache, batch)                  # [tokens, heads, dim]

``qk_norm_rope`` is the norm and rotation alone, for keys that go to no cache.
PyTorch supplies device memory and streams only; every call is one or a few
kernels of the library on the current stream (or on stream=, which the inputs
must then be ready on), allocates nothing but its outputs, and can be captured
in a CUDA graph.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct

import torch

from . import _lib
from ._lib import check
from .api import device_status

_ACT = {torch.float16: _lib.EXL3_F16, torch.bfloat16: _lib.EXL3_BF16}
_CODES = {torch.float16: _lib.EXL3_F16, torch.bfloat16: _lib.EXL3_BF16,
          torch.float8_e4m3fn: _lib.EXL3_E4M3}


# exl3_heads and exl3_rope as C lays them out.  Single-token calls last a few
# microseconds on the GPU, so the call's own cost counts: the argument structs
# are packed bytes, the stream is asked for by its raw handle.
_HEADS = struct.Struct("@QQQiqqqq")
_ROPE = struct.Struct("@Qii")
assert _HEADS.size == ctypes.sizeof(_lib.Heads) and _ROPE.size == ctypes.sizeof(_lib.Rope)
_current_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing


def _stream(stream, t):
    return _current_stream(t.get_device()) if stream is None else stream.cuda_stream


def _on(stream):
    """Makes stream, where there is one, torch's current stream."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    """An uninitialised contiguous tensor that the launch stream may write at
    once, for use on the current stream later."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _cuda(t, name, dtype):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype if isinstance(dtype, torch.dtype) else t.dtype not in dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _dense(t, name, dtype, shape):
    _cuda(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class PagedKVCache:
    """A paged cache: k and v [pages, page_size, kv_heads, head_dim], fp16, bf16
    or float8_e4m3fn, channels contiguous, the other strides free but alike (a
    permuted view of [pages, kv_heads, page_size, head_dim] works).  k_scale,
    v_scale: fp32 [kv_heads], E4M3 only; a stored x stands for x * scale (0 and
    negative scales are fine).
    page_size is a multiple of 16.  The tensors must stay alive as long as the
    handle.  `status()` is the sticky device status of all calls on the handle
    (it synchronises).

    The handle keeps a workspace per stream (`ws` is the current stream's), so
    calls on different streams may overlap.  A captured call uses that of the
    stream it is captured on; torch.cuda.graph's own capture stream gets one
    that another stream leaves to it for good, so run a step (or call
    `workspace()`) once before its capture, which raises a RuntimeError where
    none is large enough.  Replays of a handle's graphs must not overlap one
    another, nor calls on the stream they were captured on, unless ws= keeps
    them apart."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _cuda(k, "k", _CODES)
        _cuda(v, "v", k.dtype)
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride():
            raise ValueError("k and v must be [pages, page_size, kv_heads, head_dim] with the "
                             "same shape and strides")
        if k.numel() and k.stride(3) != 1 and k.shape[3] > 1:
            raise ValueError("the channels of k and v must be contiguous")
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                _dense(t, n, torch.float32, (k.shape[2],))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kv_heads, self.head_dim, self.dtype = k.shape[2], k.shape[3], k.dtype
        d = _lib.KVCache()
        d.k, d.v, d.dtype = k.data_ptr(), v.data_ptr(), _CODES[k.dtype]
        d.num_pages, d.page_size, d.kv_heads, d.head_dim = k.shape
        d.page_stride, d.token_stride, d.head_stride = _strides(k)
        d.k_scale = k_scale.data_ptr() if k_scale is not None else None
        d.v_scale = v_scale.data_ptr() if v_scale is not None else None
        self._d, self._ref = d, ctypes.byref(d)
        self._spaces = {}  # raw stream -> the workspace of its calls
        self._all = []     # every one so far: a graph may hold an outgrown one
        self._spaces[_current_stream(k.get_device())] = self._space(_lib.EXL3_ATTENTION_HEAD_BYTES)

    def _space(self, n):
        if n == _lib.EXL3_ATTENTION_HEAD_BYTES:
            ws = torch.zeros(n, dtype=torch.uint8, device=self.k.device)
        else:
            ws = torch.empty(n, dtype=torch.uint8, device=self.k.device)
            ws[:_lib.EXL3_ATTENTION_HEAD_BYTES].zero_()
        self._all.append(_Space(ws))
        return self._all[-1]

    def _room(self, stream, raw, size):
        """The workspace of a call of size (tokens, heads, num_seqs), or of one
        that needs the status word only (None), on a stream."""
        w = self._spaces.get(raw)
        n = _lib.EXL3_ATTENTION_HEAD_BYTES if size is None else self.workspace_size(*size)
        if w is None or w.bytes < n:
            with _on(stream):
                if _capturing():
                    w = self._take(n)
                else:
                    # 1 MiB over: each 256 rows more take tens of bytes more
                    w = self._space(n if size is None else n + (1 << 20))
            self._spaces[raw] = w
        w.fits = size
        return w

    def _take(self, n):
        """A workspace for a capture: no other stream's from now on, unless
        only those that graphs have taken are large enough."""
        fit = [(not w.graph, w.bytes, r) for r, w in self._spaces.items() if w.bytes >= n]
        if not fit:
            raise RuntimeError(f"no workspace of {n} bytes to capture this call with: run it once, or "
                               "call workspace() for its size, before the capture")
        free, _, raw = max(fit)
        w = self._spaces.pop(raw) if free else self._spaces[raw]
        w.graph = True
        return w

    @property
    def ws(self) -> torch.Tensor:
        return (self._spaces.get(_current_stream(self.k.get_device())) or self._all[-1]).ws

    def status(self, stream=None) -> int:
        """The status bits set so far (0: fine); see exl3.h."""
        torch.cuda.synchronize(self.k.device)
        bits = 0
        for w in self._all:
            bits |= device_status(w.ws, stream)
        return bits

    def clear_status(self):
        wait = (lambda d: None) if _capturing() else torch.cuda.synchronize
        wait(self.k.device)  # (the calls of every stream before and after)
        for w in self._all:
            w.ws[:4].zero_()
        wait(self.k.device)

    def workspace_size(self, tokens: int, heads: int, num_seqs: int) -> int:
        return int(_lib.lib().exl3_paged_attention_workspace_size(
            tokens, heads, self.kv_heads, self.head_dim, num_seqs))

    def workspace(self, tokens: int, heads: int, num_seqs: int) -> torch.Tensor:
        """The current stream's workspace, grown to hold a call of this size."""
        return self._room(None, _current_stream(self.k.get_device()), (tokens, heads, num_seqs)).ws


class _Space:
    """A workspace: graph: a capture has taken it; fits: the size of call it was
    last found to fit."""
    __slots__ = ("ws", "ptr", "bytes", "graph", "fits")

    def __init__(self, ws):
        self.ws, self.ptr, self.bytes, self.graph, self.fits = ws, ws.data_ptr(), ws.numel(), False, None


class PagedBatch:
    """The sequences of one step.  Sequence b has the new tokens cu_q[b] ..
    cu_q[b+1]-1 and seq_lens[b] tokens in all, the new ones last, so new token
    i of n stands at position seq_lens[b] - n + i; position p is in place
    p % page_size of page block_table[b, p // page_size].  int32 CUDA tensors
    [B + 1], [B], [B, max_pages]; their values may change between calls (they
    are read on the device).  max_q: the most new tokens of a sequence, a hint
    that picks the kernel."""

    def __init__(self, cu_q, seq_lens, block_table, max_q: int):
        n = seq_lens.shape[0]
        _dense(cu_q, "cu_q", torch.int32, (n + 1,))
        _dense(seq_lens, "seq_lens", torch.int32, (n,))
        _cuda(block_table, "block_table", torch.int32)
        if block_table.dim() != 2 or block_table.shape[0] != n or \
                (block_table.shape[1] > 1 and block_table.stride(1) != 1):
            raise ValueError("block_table must be [sequences, pages] with contiguous rows")
        self.cu_q, self.seq_lens, self.block_table = cu_q, seq_lens, block_table
        self.num_seqs, self.max_q = n, int(max_q)
        d = _lib.KVBatch()
        d.num_seqs, d.max_q, d.max_pages = n, self.max_q, block_table.shape[1]
        d.table_stride = block_table.stride(0)
        d.cu_q, d.seq_lens = cu_q.data_ptr(), seq_lens.data_ptr()
        d.block_table = block_table.data_ptr()
        self._d, self._ref = d, ctypes.byref(d)


def _strides(t):
    """All strides but the last, 0 where a dimension of one leaves them open."""
    return [0 if n == 1 else s for n, s in zip(t.shape[:-1], t.stride()[:-1])]


def _act(x, name, dim):
    """Checks a [tokens, heads, dim] tensor; its shape and the strides of a
    token and a head."""
    shape, stride = x.shape, x.stride()
    if x.dtype not in _ACT or not x.is_cuda:
        _cuda(x, name, _ACT)
    if len(shape) != 3 or shape[2] != dim or (stride[2] != 1 and x.numel()):
        raise ValueError(f"{name} must be [tokens, heads, {dim}] with contiguous channels")
    T, H, _ = shape
    return T, H, 0 if T == 1 else stride[0], 0 if H == 1 else stride[1]


def _like(x, stream):
    """An uninitialised contiguous tensor of x's shape."""
    if stream is None and x.is_contiguous():
        return torch.empty_like(x)
    return _empty(x.shape, x.dtype, x.device, stream)


def _weight(w, name, dtype, dim):
    if w is None:
        return 0
    if w.dtype != dtype or w.shape != (dim,) or not w.is_cuda or not w.is_contiguous():
        _dense(w, name, dtype, (dim,))
    return w.data_ptr()


def _out(out, x, T, H, dim, name, stream):
    """(out, exl3_heads' out pointer and strides): a new tensor, or the given
    one checked."""
    if out is None:
        out = _like(x, stream)
        return out, out.data_ptr(), H * dim, dim
    if out.dtype != x.dtype or out.shape != x.shape:
        raise ValueError(f"{name} must be {tuple(x.shape)} {x.dtype}")
    _, _, ts, hs = _act(out, name, dim)
    return out, out.data_ptr(), ts, hs


def _positions(positions, T):
    if positions is None:
        return None
    if positions.dtype != torch.int32 or positions.shape != (T,) or not positions.is_cuda or \
            not positions.is_contiguous():
        _dense(positions, "positions", torch.int32, (T,))
    return positions.data_ptr()


def _rope(inv_freq, interleaved):
    if inv_freq is None:
        return None
    if inv_freq.dtype != torch.float64 or not inv_freq.is_cuda:
        _cuda(inv_freq, "inv_freq", torch.float64)
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous [rotary_dim / 2] tensor")
    return _ROPE.pack(inv_freq.data_ptr(), 2 * inv_freq.shape[0], 1 if interleaved else 0)


def qk_norm_rope(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None,
                 eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """(q, k) with every head vector RMS normed (where there is a weight) and
    rotated by its token's position (where there is an inv_freq).

    q [tokens, heads, dim] and k [tokens, kv_heads, dim] (or None), fp16 or
    bf16, any strides that are multiples of 8 elements; positions int32
    [tokens]; inv_freq float64 [rotary_dim / 2], radians per position of pair
    (i, i + rotary_dim/2) of the first rotary_dim channels, or (2i, 2i + 1)
    when interleaved.  q_out and k_out may be q and k."""
    dim = q.shape[-1]
    T, H, ts, hs = _act(q, "q", dim)
    dtype = q.dtype
    q_out, p, ots, ohs = _out(q_out, q, T, H, dim, "q_out", stream)
    hq = _HEADS.pack(q.data_ptr(), p, _weight(q_weight, "q_weight", dtype, dim), H, ts, hs, ots, ohs)
    hk = None
    if k is not None:
        Tk, Hk, ts, hs = _act(k, "k", dim)
        if Tk != T or k.dtype != dtype:
            raise ValueError("q and k must have the same dtype and tokens")
        k_out, p, ots, ohs = _out(k_out, k, T, Hk, dim, "k_out", stream)
        hk = _HEADS.pack(k.data_ptr(), p, _weight(k_weight, "k_weight", dtype, dim), Hk, ts, hs, ots,
                         ohs)
    check(_lib.lib().exl3_qk_norm_rope(hq, hk, _ACT[dtype], T, dim, _positions(positions, T),
                                       _rope(inv_freq, interleaved), eps, _stream(stream, q)),
          "exl3_qk_norm_rope")
    return q_out, k_out


def kv_append(cache: PagedKVCache, batch: PagedBatch, k, v, inv_freq=None, k_weight=None, q=None,
              q_weight=None, q_out=None, positions=None, eps: float = 1e-6,
              interleaved: bool = False, stream=None):
    """Writes the new tokens' keys (normed and rotated as by qk_norm_rope) and
    values to the cache; with q, returns the normed and rotated queries, from
    the same launch.  positions: those of the rotation (default: the positions
    in the sequence).  A value past the E4M3 range saturates."""
    dim, dtype = cache.head_dim, k.dtype
    T, H, ts, hs = _act(k, "k", dim)
    Tv, Hv, tv, hv = _act(v, "v", dim)
    if v.dtype != dtype or Tv != T or H != cache.kv_heads or Hv != H:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] of one dtype")
    pk = _HEADS.pack(k.data_ptr(), 0, _weight(k_weight, "k_weight", dtype, dim), H, ts, hs, 0, 0)
    pv = _HEADS.pack(v.data_ptr(), 0, 0, H, tv, hv, 0, 0)
    pq = None
    if q is not None:
        Tq, Hq, ts, hs = _act(q, "q", dim)
        if Tq != T or q.dtype != dtype:
            raise ValueError("q and k must have the same dtype and tokens")
        q_out, p, ots, ohs = _out(q_out, q, T, Hq, dim, "q_out", stream)
        pq = _HEADS.pack(q.data_ptr(), p, _weight(q_weight, "q_weight", dtype, dim), Hq, ts, hs, ots,
                         ohs)
    raw = _stream(stream, k)
    check(_lib.lib().exl3_kv_append(cache._ref, batch._ref, pq, pk, pv, _ACT[dtype], T,
                                    _rope(inv_freq, interleaved), _positions(positions, T), eps,
                                    (cache._spaces.get(raw) or cache._room(stream, raw, None)).ptr, raw),
          "exl3_kv_append")
    return q_out


def paged_attention(q, cache: PagedKVCache, batch: PagedBatch, scale=None, causal: bool = True,
                    window: int = 0, out=None, return_lse: bool = False, path: int = 0, ws=None,
                    stream=None):
    """Attention of the new tokens q [tokens, heads, head_dim] over the cache,
    which already holds them.  A token at position P sees the positions p <= P
    of its sequence (all of them when causal is false), and p > P - window when
    window > 0.  scale defaults to head_dim ** -0.5.  Returns out [tokens,
    heads, head_dim], or (out, lse fp32 [tokens, heads]) with return_lse; a
    token that sees nothing gets out 0 and lse -inf.

    ws: a workspace of the caller's instead of the handle's, uint8, of at least
    cache.workspace_size(tokens, heads, sequences) bytes, whose first 4096
    (exl3.h: EXL3_ATTENTION_HEAD_BYTES) were zeroed before its first call.  It
    serves one call at a time, and holds the status of its own calls
    (device_status(ws))."""
    if not q.is_cuda:
        _cuda(q, "q", _ACT)
    dim = cache.head_dim
    T, heads, ts, hs = _act(q, "q", dim)
    raw = _stream(stream, q)
    if ws is None:
        w, size = cache._spaces.get(raw), (T, heads, batch.num_seqs)
        if w is None or w.fits != size:
            w = cache._room(stream, raw, size)
        ws_ptr, ws_bytes = w.ptr, w.bytes
    else:
        _dense(ws, "ws", torch.uint8, ws.shape)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel()
    if out is None:
        out = _like(q, stream)
    else:
        _dense(out, "out", q.dtype, (T, heads, dim))
    lse = _empty((T, heads), torch.float32, q.device, stream) if return_lse else None
    check(_lib.lib().exl3_paged_attention(
        cache._ref, batch._ref, q.data_ptr(), ts, hs, _ACT[q.dtype], T, heads,
        dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, out.data_ptr(),
        None if lse is None else lse.data_ptr(), path, ws_ptr, ws_bytes, raw), "exl3_paged_attention")
    return (out, lse) if return_lse else out
