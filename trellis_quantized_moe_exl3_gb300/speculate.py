"""Speculative decoding around the paged cache: Python API over the C ABI.

    pool = PagePool(num_pages, page_size, max_seqs, max_pages)   # pages of the cache, on the GPU
    step = pool.extend(seqs, q_lens, max_q, max_tokens)          # a PagedBatch with its pages
    q = kv_append(cache, step, ...); out = paged_attention(q, cache, step)
    tokens, accepted, dropped = verify_drafts(p, draft, cu_draft, accept_u, sample_u, q=q_probs,
                                              step=step)
    pool.trim(seqs, dropped)                                     # refused drafts leave the cache

Nothing of it is read on the host, so a whole step can be captured in a CUDA
graph.  Every call is one or two kernels on the current stream (or on stream=,
which the inputs must then be ready on, and which keeps their memory until it
is done).
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import device_status
from .attention import PagedBatch, _capturing, _Lent


class PagedStep(PagedBatch):
    """A step as PagePool.extend lays it out: a PagedBatch (cu_q, seq_lens,
    block_table) with positions [max_tokens] int32 and slots [max_tokens] int64
    (page * page_size + place) of its new tokens, -1 in rows that are none's.
    cu_q, seq_lens and positions share an allocation: one that is kept, or saved,
    keeps the others (clone it)."""

    def __init__(self, device, pages, max_q, cu_q, seq_lens, block_table, positions, slots, batch):
        self.cu_q, self.seq_lens, self.block_table = cu_q, seq_lens, block_table
        self.positions, self.slots = positions, slots
        self.num_seqs, self.max_q, self._device, self._pages = len(seq_lens), max_q, device, pages
        self._at = self._ref = batch  # exl3_kv_batch, its bytes


class PagePool(_Lent):
    """The pages of a cache and the sequences that hold them, on the GPU: `table`
    [max_seqs, max_pages], `lens` [max_seqs], `free` [num_pages] and `count` [1],
    int32.  A sequence is a row of the table; free[0 .. count - 1] are the free
    pages, taken from the end.  Between calls a program may write these tensors
    (a restored state); `status()` is the sticky device status (exl3.h; it
    synchronises).  A pool's calls follow one another: it serves one stream at a
    time."""

    def __init__(self, num_pages: int, page_size: int, max_seqs: int, max_pages: int, device=None):
        if num_pages < 0 or max_seqs < 1 or max_pages < 1:
            raise ValueError("a pool has pages, rows and columns")
        device = torch.device("cuda") if device is None else torch.device(device)
        if device.type != "cuda":
            raise ValueError("a pool lives on a CUDA device")

        def full(x, *shape):
            return torch.full(shape, x, dtype=torch.int32, device=device)

        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self.max_seqs, self.max_pages = int(max_seqs), int(max_pages)
        self.table, self.lens = full(-1, max_seqs, max_pages), full(0, max_seqs)
        self.free = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.count = full(num_pages, 1)
        n = _lib.lib().exl3_pages_workspace_size(self.max_seqs, self.max_seqs)
        if n == 0:
            raise ValueError(f"max_seqs {max_seqs} is out of range")
        self.ws = torch.zeros(n, dtype=torch.uint8, device=device)
        d = _lib.PagePool()
        d.num_pages, d.page_size, d.max_seqs, d.max_pages = num_pages, page_size, max_seqs, max_pages
        d.table, d.lens = self.table.data_ptr(), self.lens.data_ptr()
        d.free, d.count = self.free.data_ptr() or None, self.count.data_ptr()
        self._d, self._at = d, ctypes.addressof(d)
        self._ws, self._ws_bytes, self._device = self.ws.data_ptr(), n, self.ws.get_device()
        if not _capturing():  # calls on other streams find it made
            torch.cuda.current_stream(device).synchronize()
        self._native = _lib.native()

    def _tensors(self):
        return self.table, self.lens, self.free, self.count, self.ws

    def extend(self, seqs, q_lens, max_q: int, max_tokens: int, stream=None) -> PagedStep:
        """Begins a step: row seqs[i] of the pool gets q_lens[i] new tokens and the
        pages for them (int32 [sequences]).  max_tokens: rows of the step's token
        tensors, at least the sum of q_lens; max_q: as PagedBatch's.  A sequence
        for which there are no pages left keeps its rows, but has length 0 in the
        step and stays as it was in the pool (give the step to verify_drafts, or to
        trim, so that it stays so; kv_append's status reports its tokens)."""
        self._lend(stream)
        return PagedStep(self._device, (self.page_size, self.num_pages), max_q, *self._native.pages_extend(
            self._at, self._ws, self._ws_bytes, seqs, q_lens, max_tokens, max_q, stream, self._device))

    def trim(self, seqs, drop=None, stream=None, step=None):
        """Takes the last drop[i] tokens (None: all) of row seqs[i] off and gives
        back the pages that hold nothing any more.  step: the step of the same
        seqs that these tokens are of (extend's); rows that it did not serve got
        none, and are left alone.  Without it a drop of tokens that never came
        takes older ones."""
        self._lend(stream)
        self._native.pages_trim(self._at, self._ws, self._ws_bytes, seqs, drop, stream, self._device,
                                None if step is None else step.seq_lens)

    def status(self, stream=None) -> int:
        """The status bits set so far (0: fine); see exl3.h."""
        torch.cuda.synchronize(self.ws.device)
        return device_status(self.ws, stream)

    def clear_status(self):
        wait = (lambda d: None) if _capturing() else torch.cuda.synchronize
        wait(self.ws.device)
        self.ws[:4].zero_()
        wait(self.ws.device)


def verify_drafts(p, draft, cu_draft, accept_u, sample_u, q=None, stream=None, step=None):
    """Which drafted tokens stand, and the token after them.

    Sequence b has the drafts draft[cu_draft[b] .. cu_draft[b+1] - 1] (int32;
    cu_draft int32 [sequences + 1], read on the device).  p [drafts + sequences,
    vocab]: the target's probabilities, fp32, fp16 or bf16, one row more per
    sequence than drafts: row cu_draft[b] + b + j is that of the token after j
    drafts.  q [drafts, vocab]: the probabilities that the drafts were drawn from
    (None: they are certain).  accept_u [drafts], sample_u [sequences]: fp32
    random numbers in [0, 1).

    Draft x is accepted, after all before it, if accept_u * q(x) < p(x).  After
    the first refusal a token is drawn from max(p - q, 0), after the last draft
    from p: the first whose cumulative weight is above sample_u of the total.
    The first is decided exactly; weights are rounded to units of 2^-46 (a token
    below 2^-47 is never drawn) and summed without a further rounding, whatever
    the size of the vocabulary.  NaN and what is negative count as 0, what is
    above 1 as 1; a row may sum to less than 2^16.  Where p - q leaves nothing, p
    itself counts; a row of p without weight gives -1 for the token.

    Returns int32 (tokens [drafts + sequences], accepted [sequences], dropped
    [sequences]): from place cu_draft[b] + b on, the accepted drafts, the drawn
    token, then -1; accepted drafts, and the others (what PagePool.trim takes).
    Places of no sequence hold -1, those of one whose cu_draft does not ascend too.
    They share an allocation: one that is kept, or saved, keeps the others.

    step: the step (PagePool.extend's) that p was computed for.  A sequence that
    it did not serve, for want of pages, has seen nothing: it gets tokens -1, and
    0 of both counts, so that trim takes nothing off its row."""
    return _lib.native().verify_drafts(p, draft, cu_draft, accept_u, sample_u, q, stream,
                                       None if step is None else step.seq_lens)
