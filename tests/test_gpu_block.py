"""A decoder layer: attention operators and the coded MoE layer together.

The same tokens, given to the block as one prompt, in chunks and one by one,
go through different kernels (tensor-core tiles, few rows); each must agree
with the block computed in 64 bits from the same bf16 weights."""
import os
import sys

import numpy as np
import pytest
import torch

import _attention_ref as R
from _helpers import FRO_REL, MAX_REL, HostLayer, act_to_f64
from trellis_quantized_moe_exl3_gb300 import DecoderBlock, PagedBatch, PagedKVCache, rmsnorm, synth

pytestmark = pytest.mark.gpu


def weights(seed, H, heads, kv, dim, E):
    g = torch.Generator().manual_seed(seed)
    w = lambda *s: (torch.randn(*s, generator=g) * s[0] ** -0.5).bfloat16().cuda()  # noqa: E731
    n = lambda: (1 + 0.2 * torch.randn(dim, generator=g)).bfloat16().cuda()  # noqa: E731
    return w(H, E), w(H, (heads + 2 * kv) * dim), w(heads * dim, H), n(), n()


def attend_ref(x, w_qkv, w_out, qn, kn, f, heads, kv, dim):
    """x + attention(norm(x)) of one sequence in float64 (x: [T, H] bf16)."""
    x = x.double().cpu()
    T = x.shape[0]
    h = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    h = h.bfloat16().double()  # the norm's output is stored in bf16
    qkv = (h @ w_qkv.double().cpu()).bfloat16().double().view(T, -1, dim)
    q, k, v = qkv.split([heads, kv, kv], 1)
    pos = torch.arange(T)
    q = R.norm_rope(q, pos, f, qn, 1e-6, False).bfloat16()
    k = R.norm_rope(k, pos, f, kn, 1e-6, False).bfloat16()
    table = torch.arange(-(-T // 16)).view(1, -1)
    pad = table.shape[1] * 16 - T
    page = lambda t: torch.cat([t.double(), torch.zeros(pad, kv, dim, dtype=torch.float64)]).view(-1, 16, kv, dim)  # noqa: E731
    out, _, _ = R.attention(q, page(k), page(v.bfloat16()), table, [T], [T], 16, dim ** -0.5, True, 0)
    return x + out.bfloat16().double().reshape(T, -1) @ w_out.double().cpu()


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (6, 2, 64)])
def test_block_as_prompt_chunks_and_tokens(heads, kv, dim):
    spec = synth.LayerSpec(seed=11, num_experts=8, hidden=256, inter=128)
    host = HostLayer(spec)
    moe = host.device()
    router, w_qkv, w_out, qn, kn = weights(3, 256, heads, kv, dim, 8)
    f = (500000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)).cuda()
    block = DecoderBlock(moe, router, w_qkv, w_out, heads, kv, top_k=2, inv_freq=f, q_norm=qn, k_norm=kn)
    T = 75
    x = torch.from_numpy(synth.activations(5, T, 256, "bf16").view(np.int16)).cuda().view(torch.bfloat16)
    want = attend_ref(x, w_qkv, w_out, qn, kn, f, heads, kv, dim)

    def run(cuts, method):
        kvc = [torch.zeros(6, 16, kv, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cache = PagedKVCache(*kvc)
        table = torch.tensor([[4, 1, 0, 5, 3]], dtype=torch.int32, device="cuda")
        out, at = [], 0
        for n in cuts:
            b = PagedBatch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                           torch.tensor([at + n], dtype=torch.int32, device="cuda"), table, n)
            out.append(method(x[at:at + n], cache, b))
            at += n
        assert at == T and cache.status() == 0
        return torch.cat(out)

    ol = host.oracle()
    for cuts in ([T], [40, 1, 34], [1] * T):
        a = run(cuts, block.attend)
        # bf16 steps on the way: projection, rotation, softmax terms, output,
        # sum; each moves a value by half a step of its own size, a few of them
        # in the same direction at most
        err = (a.double().cpu() - want).abs()
        assert float(err.max()) <= 6 * 2.0 ** -8 * float(want.abs().max()), (cuts, float(err.max()))
        assert float(err.norm() / want.norm()) <= 2 * 2.0 ** -8
        y = run(cuts, block)
        # the MoE half against the oracle, from the same attention output
        h = rmsnorm(a, 1e-6)
        lg, at = [], 0
        for n in cuts:  # (a product of another shape may round otherwise)
            lg.append((h[at:at + n] @ router).float())
            at += n
        lg = torch.cat(lg)
        ref = ol.forward(h.cpu().view(torch.int16).numpy().view(np.uint16), True, lg.cpu().numpy(), 2)
        d = act_to_f64(y) - (ref + act_to_f64(a))
        assert np.abs(d).max() <= MAX_REL * np.abs(ref).max()
        assert np.linalg.norm(d) <= FRO_REL * np.linalg.norm(ref) * 2


def test_block_checks_shapes():
    w = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        DecoderBlock(None, None, w, torch.zeros(64, 8), 2, 1, 2)


def test_example_runs(capsys, monkeypatch):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import serve_block
    finally:
        sys.path.pop(0)
    monkeypatch.setattr(sys, "argv", ["serve_block.py", "--experts", "4", "--seqs", "3", "--prompt", "150",
                                      "--chunk", "64", "--steps", "5", "--e4m3"])
    serve_block.main()
    text = capsys.readouterr().out
    assert "lengths now [156, 119, 82]" in text and "device status 0" in text
