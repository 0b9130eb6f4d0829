"""One decoder layer served: ragged prompts in chunks, then single tokens from a CUDA graph.

    python examples/serve_block.py [--experts 32] [--seqs 8] [--prompt 700] [--steps 64] [--e4m3]
                                   [--blocks] [--drafts 4]

The cache's pages come from a pool on the GPU.  --e4m3: an 8-bit cache with a
scale per head, --blocks: with one per page and head.  --drafts N: then steps of
N drafted tokens each, verified and taken back where they are refused, from a
graph as well.  Synthetic weights; prints the tokens per second of every phase
and the layer's device status."""
import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from trellis_quantized_moe_exl3_gb300 import (DecoderBlock, Layer, PagedKVCache, PagePool,  # noqa: E402
                                               synth, verify_drafts)


def build_block(spec, heads, kv_heads, dim, top_k, seed=0):
    """A block with random dense weights around a coded layer of synthetic codes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = spec.hidden

    def w(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * shape[0] ** -0.5).bfloat16()

    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()  # noqa: E731
    sides = [synth.side_vectors(spec, p) for p in range(3)]
    moe = Layer([dev(synth.layer_codes(spec, p)) for p in range(3)],
                [dev(s[0]).view(torch.float16) for s in sides],
                [dev(s[1]).view(torch.float16) for s in sides], spec.K)
    norm = lambda: (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).bfloat16()  # noqa: E731
    inv_freq = 500000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    return DecoderBlock(moe, w(H, spec.num_experts), w(H, (heads + 2 * kv_heads) * dim),
                        w(heads * dim, H), heads, kv_heads, top_k, inv_freq, norm(), norm())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--chunk", type=int, default=256)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--e4m3", action="store_true", help="8-bit cache, a scale per head")
    ap.add_argument("--blocks", action="store_true", help="8-bit cache, a scale per page and head")
    ap.add_argument("--drafts", type=int, default=0, help="drafted tokens per step of a last phase")
    a = ap.parse_args()
    heads, kv_heads, dim, page = 32, 8, 128, 64
    spec = synth.LayerSpec(seed=2, num_experts=a.experts)
    block = build_block(spec, heads, kv_heads, dim, top_k=min(8, a.experts))
    prompts = [max(1, a.prompt - 37 * b) for b in range(a.seqs)]
    # (a token per step, then a token and its drafts at most)
    per = -(-(max(prompts) + (a.steps + 8) * (2 + a.drafts if a.drafts else 1)) // page)
    pages = a.seqs * per
    eight = a.e4m3 or a.blocks
    kv = [torch.zeros(pages, page, kv_heads, dim, device="cuda",
                      dtype=torch.float8_e4m3fn if eight else torch.bfloat16) for _ in range(2)]
    scale = [torch.zeros(pages, kv_heads, device="cuda") if a.blocks else
             torch.full((kv_heads,), 0.05, device="cuda") if eight else None for _ in range(2)]
    cache, pool = PagedKVCache(*kv, *scale), PagePool(pages, page, a.seqs, per)
    seqs = torch.arange(a.seqs, dtype=torch.int32, device="cuda")

    def extend(new):
        return pool.extend(seqs, torch.tensor(new, dtype=torch.int32, device="cuda"), max(new), sum(new))

    # prompts, a chunk of each sequence at a time
    done, t0, out = [0] * a.seqs, time.perf_counter(), None
    while any(d < p for d, p in zip(done, prompts)):
        new = [min(a.chunk, p - d) for d, p in zip(done, prompts)]
        done = [d + n for d, n in zip(done, new)]
        x = torch.randn(sum(new), spec.hidden, device="cuda").bfloat16()
        out = block(x, cache, extend(new))
    torch.cuda.synchronize()
    print(f"prompts: {sum(prompts)} tokens, {sum(prompts) / (time.perf_counter() - t0):.0f} tokens/s "
          f"(first calls included), output norm {float(out.float().norm()):.3e}")

    # single tokens: one captured step that takes its pages from the pool
    one = torch.ones(a.seqs, dtype=torch.int32, device="cuda")
    x = torch.randn(a.seqs, spec.hidden, device="cuda").bfloat16()
    y, dt = timed(lambda: block(x, cache, pool.extend(seqs, one, 1, a.seqs)), a.steps)
    print(f"decode: {a.steps} steps of {a.seqs} sequences, {dt / a.steps * 1e6:.1f} us per step, "
          f"{a.steps * a.seqs / dt:.0f} tokens/s, lengths now {pool.lens.tolist()}, "
          f"output norm {float(y.float().norm()):.3e}")
    if a.drafts:
        speculate(block, cache, pool, seqs, spec.hidden, a.drafts, a.steps)
    print("device status", cache.status() | pool.status())


def timed(step, steps):
    """The last result of a step that is captured and replayed, and the seconds taken."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    return y, time.perf_counter() - t0


def speculate(block, cache, pool, seqs, hidden, drafts, steps, vocab=1000):
    """Steps of a token and its drafts: pages, the block, the target's probabilities,
    verification, and refused drafts out of the cache again.  The drafting model
    here says that every token is as likely as any other."""
    n, rows = len(seqs), drafts + 1
    embed = torch.randn(vocab, hidden, device="cuda").bfloat16()
    head = (torch.randn(hidden, vocab, device="cuda") * hidden ** -0.5).bfloat16()
    q_lens = torch.full((n,), rows, dtype=torch.int32, device="cuda")
    cu_draft = torch.arange(0, n * drafts + 1, drafts, dtype=torch.int32, device="cuda")
    q = torch.full((n * drafts, vocab), 1.0 / vocab, device="cuda")
    last = torch.zeros(n, dtype=torch.int64, device="cuda")
    made = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step():
        draft = torch.randint(0, vocab, (n, drafts), device="cuda")
        x = embed[torch.cat([last[:, None], draft], 1).flatten()]
        at = pool.extend(seqs, q_lens, rows, n * rows)
        y = block(x, cache, at).float()
        p = ((y / y.norm(dim=-1, keepdim=True)) @ head.float()).softmax(-1)
        tokens, accepted, dropped = verify_drafts(
            p, draft.int().flatten(), cu_draft, torch.rand(n * drafts, device="cuda"),
            torch.rand(n, device="cuda"), q=q, step=at)
        pool.trim(seqs, dropped)
        last.copy_(tokens.view(n, rows).gather(1, accepted.long()[:, None])[:, 0])
        made.add_((accepted + 1).sum())
        return accepted

    made.zero_()
    accepted, dt = timed(step, steps)
    made = int(made)
    print(f"drafts: {steps} steps of {n} x {drafts}, {dt / steps * 1e6:.1f} us per step, "
          f"{made / (steps + 1):.1f} tokens per step, lengths now {pool.lens.tolist()}, "
          f"last token {int(last[0])}")


if __name__ == "__main__":
    main()
