"""One decoder layer served: ragged prompts in chunks, then single tokens from a CUDA graph.

    python examples/serve_block.py [--experts 32] [--seqs 8] [--prompt 700] [--steps 64] [--e4m3]

Synthetic weights; prints the tokens per second of both phases and the layer's
device status."""
import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from trellis_quantized_moe_exl3_gb300 import DecoderBlock, Layer, PagedBatch, PagedKVCache, synth  # noqa: E402


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
    ap.add_argument("--e4m3", action="store_true", help="8-bit cache")
    a = ap.parse_args()
    heads, kv_heads, dim, page = 32, 8, 128, 64
    spec = synth.LayerSpec(seed=2, num_experts=a.experts)
    block = build_block(spec, heads, kv_heads, dim, top_k=min(8, a.experts))
    prompts = [max(1, a.prompt - 37 * b) for b in range(a.seqs)]
    per = -(-(max(prompts) + a.steps + 8) // page)
    table = torch.randperm(a.seqs * per, device="cuda").int().view(a.seqs, per)
    kv = [torch.zeros(a.seqs * per, page, kv_heads, dim, device="cuda",
                      dtype=torch.float8_e4m3fn if a.e4m3 else torch.bfloat16) for _ in range(2)]
    scale = [torch.full((kv_heads,), 0.05, device="cuda") if a.e4m3 else None for _ in range(2)]
    cache = PagedKVCache(*kv, *scale)

    def batch_of(new, total):
        cu = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
        return PagedBatch(cu, torch.tensor(total, dtype=torch.int32, device="cuda"), table, max(new))

    # prompts, a chunk of each sequence at a time
    done, t0, out = [0] * a.seqs, time.perf_counter(), None
    while any(d < p for d, p in zip(done, prompts)):
        new = [min(a.chunk, p - d) for d, p in zip(done, prompts)]
        done = [d + n for d, n in zip(done, new)]
        x = torch.randn(sum(new), spec.hidden, device="cuda").bfloat16()
        out = block(x, cache, batch_of(new, done))
    torch.cuda.synchronize()
    print(f"prompts: {sum(prompts)} tokens, {sum(prompts) / (time.perf_counter() - t0):.0f} tokens/s "
          f"(first calls included), output norm {float(out.float().norm()):.3e}")

    # single tokens: one captured step whose lengths advance on the device
    batch = batch_of([1] * a.seqs, done)
    x = torch.randn(a.seqs, spec.hidden, device="cuda").bfloat16()

    def step():
        batch.seq_lens.add_(1)
        return block(x, cache, batch)

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
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    print(f"decode: {a.steps} steps of {a.seqs} sequences, {dt / a.steps * 1e6:.1f} us per step, "
          f"{a.steps * a.seqs / dt:.0f} tokens/s, lengths now {batch.seq_lens.tolist()}, "
          f"output norm {float(y.float().norm()):.3e}")
    print("device status", cache.status())


if __name__ == "__main__":
    main()
