"""Long sequences over block scales: however a line is cut, it is cut over the whole
GPU, and units of many parts are joined in two steps."""
import statistics

import pytest
import torch

import test_gpu_block_scales as T
from trellis_quantized_moe_exl3_gb300 import PagedBatch, PagedKVCache, paged_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qs,lens,H,Hk,D", [
    ([1], [120000], 4, 1, 64),                                # alone: more parts than one join takes
    ([2, 1, 4], [70000, 300, 4], 4, 2, 128),                  # beside short ones, cut as one line
    ([1] + [0] * 20, [50000] + [40] * 20, 2, 1, 64),          # beside sequences without new tokens
    ([1] + [1] * 32, [60000] + [9] * 32, 2, 1, 64),           # more sequences than a warp cuts
    ([3] + [0] * 39, [40000] + [0] * 39, 8, 1, 128),
])
def test_attention_blocks_joined_in_two_steps(qs, lens, H, Hk, D):
    c = (qs, lens, 64, H, Hk, D, T.BF, True, 0)
    cache, step, q = T.setup(c)
    first = T.check(cache, step, q, c, 1)
    for _ in range(2):  # the counters are back at zero, and the result is the same
        again = paged_attention(q, cache, T.batch_of(step), scale=D ** -0.5, return_lse=True, path=1)
        assert all(torch.equal(a[:sum(qs)], b[:sum(qs)]) for a, b in zip(first, again))


@pytest.mark.parametrize("D", [64, 128])
def test_one_long_sequence_uses_the_whole_gpu(D):
    """One sequence of 250000 keys and one kv head takes about as long alone as beside 32
    empty ones, which go by an equal cut (measured: 29 us at 64 channels and 33 at 128;
    cut into the parts of one join, on 24 or 40 CTAs, 82 and 66)."""
    keys, page = 250000, 64
    n = -(-keys // page)
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = [torch.randn(n, page, 1, D, generator=g, device="cuda").mul_(60).to(torch.float8_e4m3fn)
          for _ in range(2)]
    cache = PagedKVCache(*kv, *[torch.full((n, 1), 0.01, device="cuda") for _ in range(2)])
    x = torch.randn(1, 4, D, generator=g, device="cuda").to(T.BF)
    table = torch.arange(n, dtype=torch.int32, device="cuda").expand(33, n).contiguous()
    batches = [PagedBatch(torch.tensor([0] + [1] * m, dtype=torch.int32, device="cuda"),
                          torch.tensor([keys] + [0] * (m - 1), dtype=torch.int32, device="cuda"),
                          table[:m], 1) for m in (1, 33)]
    out = [torch.empty_like(x) for _ in range(2)]
    times = [[], []]
    for k in range(30):  # in turn
        for i in range(2):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda._sleep(100000)  # (the call is queued before its turn comes)
            a.record()
            paged_attention(x, cache, batches[i], out=out[i], path=1)
            b.record()
            torch.cuda.synchronize()
            times[i].append(a.elapsed_time(b))
    alone, beside = (statistics.median(t[5:]) for t in times)
    assert alone < 1.5 * beside, (alone, beside)
    assert float((out[0].float() - out[1].float()).abs().max()) <= 2.0 ** -7 * float(out[1].float().abs().max())
