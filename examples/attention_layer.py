"""A decoder layer of full attention with a mixture-of-experts block, on the
library's operators: packed prompts first, then single tokens of all sequences in
a CUDA graph over a 4-bit cache.

    residual stream h, layer input x
    (codes, scales, h) = add_rmsnorm_fp8(x, w1, h)      residual add, norm, e4m3 rows
    qkv = matmul_fp8(codes, scales, W_qkv)              one projection for q, k and v
    (q, k) = qk_norm_rope(q, k, positions)              slices of qkv
    kv_cache_write(cache, k, v, pages, starts)
    o = attention_prefill(q, k, v)                      a prompt, or
    o = attention_decode(q, cache, pages, lengths)      a token of each sequence
    y = matmul_fp8(quantize_fp8(o), W_o)                output projection
    (n, h) = add_rmsnorm(y, w2, h)
    x = MoE(n)                                          the next layer's x

Run it on a GB300: python examples/attention_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_mixture_experts_gemm_gb300 as moe  # noqa: E402
from sparse_mixture_experts_gemm_gb300 import synth  # noqa: E402

BF16, F64, I32 = torch.bfloat16, torch.float64, torch.int32
PAGE = 64  # tokens of a page


class AttentionLayer:
    """Random weights of one layer; e4m3 projections with a scale per output
    channel, quantised once.  A cache of its own."""

    def __init__(self, seed, d, Hq, Hk, D, rot, E, F, top_k, max_tokens, pages, device):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g) * std).to(BF16).to(device)

        self.Hq, self.Hk, self.D = Hq, Hk, D
        self.w1, self.w2 = ((1 + 0.1 * normal(d)).to(BF16) for _ in range(2))
        self.wq, self.wk = ((1 + 0.1 * normal(D)).to(BF16) for _ in range(2))
        self.freq = (10000.0 ** (-torch.arange(rot // 2, dtype=F64) * 2 / rot)).to(device)
        self.Wqkv = moe.quantize_fp8(normal((Hq + 2 * Hk) * D, d, std=d ** -0.5))
        self.Wo = moe.quantize_fp8(normal(d, Hq * D, std=(Hq * D) ** -0.5))
        self.cache = moe.kv_cache(pages, Hk, D, device)
        self.moe = moe.MoELayer(synth.layer_weights(seed + 1, d, F, E, 1, "bf16", device), top_k, max_tokens)

    def project(self, x, h, positions):
        """(q, k, v, h) of rows x"""
        codes, scales, h = moe.add_rmsnorm_fp8(x, self.w1, h)
        qkv = moe.matmul_fp8(codes, scales, *self.Wqkv).unflatten(-1, (-1, self.D))
        q, k, v = qkv.split((self.Hq, self.Hk, self.Hk), 1)
        q, k = moe.qk_norm_rope(q, k, self.wq, self.wk, positions, self.freq)
        return q, k, v, h

    def finish(self, o, h):
        """(x, h) of the next layer"""
        y = moe.matmul_fp8(*moe.quantize_fp8(o.reshape(len(o), -1)), *self.Wo)
        n, h = moe.add_rmsnorm(y, self.w2, h)
        return self.moe.forward(n), h

    def prefill(self, x, h, positions, offsets, pages):
        """Rows of packed sequences, from their first positions on."""
        q, k, v, h = self.project(x, h, positions)
        moe.kv_cache_write(self.cache, k, v, pages, offsets=offsets)
        return self.finish(moe.attention_prefill(q, k, v, offsets), h)

    def decode(self, x, h, lengths, pages):
        """A row per sequence, behind lengths[i] tokens: (x, h, q, o)"""
        q, k, v, h = self.project(x, h, lengths)
        moe.kv_cache_write(self.cache, k.unsqueeze(1), v.unsqueeze(1), pages, lengths)
        o = moe.attention_decode(q, self.cache, pages, lengths + 1)
        return *self.finish(o, h), q, o


def run(lens=(37, 0, 130, 5), new=6, layers=2, device="cuda", seed=0):
    """Prompts of these lengths, then `new` tokens of each sequence; returns the
    greatest relative difference between the last layer's attention in decoding
    and over the cache read back, and the last hidden rows."""
    d, Hq, Hk, D, rot, E, F, top_k = 512, 16, 2, 256, 64, 16, 256, 4
    n, total = len(lens), sum(lens)
    width = (max(lens) + new + PAGE - 1) // PAGE
    net = [AttentionLayer(seed + 10 * i, d, Hq, Hk, D, rot, E, F, top_k, total + n, n * width, device)
           for i in range(layers)]
    g = torch.Generator().manual_seed(seed + 5)
    prompt = torch.randn(total, d, generator=g).to(BF16).to(device)
    tokens = torch.randn(new, n, d, generator=g).to(BF16).to(device)
    offsets = torch.tensor([0, *lens], device=device).cumsum(0).to(I32)
    positions = torch.cat([torch.arange(length) for length in lens]).to(I32).to(device)
    pages = torch.randperm(n * width, generator=g).to(I32).view(n, width).to(device)

    x, h = prompt, torch.zeros_like(prompt)
    for layer in net:
        x, h = layer.prefill(x, h, positions, offsets, pages)

    # decoding: one step captured in a graph and replayed
    step_in = torch.zeros(n, d, dtype=BF16, device=device)
    lengths = torch.tensor(lens, dtype=I32, device=device)

    def step():
        x, h = step_in, torch.zeros_like(step_in)
        for layer in net:
            x, h, q, o = layer.decode(x, h, lengths, pages)
        lengths.add_(1)
        return x + h, q, o

    side = torch.cuda.Stream(device)
    side.wait_stream(torch.cuda.current_stream(device))
    with torch.cuda.stream(side):
        step()  # (first calls are not captured; the token's place is written again below)
    torch.cuda.current_stream(device).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        last, q, o = step()
    lengths.copy_(torch.tensor(lens, dtype=I32))
    queries, outputs = [], []
    for t in tokens:
        step_in.copy_(t)
        graph.replay()
        queries.append(q.clone())
        outputs.append(o.clone())

    # the last layer's new tokens again, over what the cache holds
    ends = [length + new for length in lens]
    k_offsets = torch.tensor([0, *ends], device=device).cumsum(0).to(I32)
    k, v = moe.kv_cache_read(net[-1].cache, pages, k_offsets, sum(ends))
    q_offsets = torch.arange(0, n * new + 1, new, dtype=I32, device=device)
    again = moe.attention_prefill(torch.stack(queries, 1).flatten(0, 1), k, v, q_offsets, k_offsets).float()
    made = torch.stack(outputs, 1).flatten(0, 1).float()
    diff = (made - again).norm(dim=-1) / again.norm(dim=-1)
    torch.cuda.synchronize(device)
    for layer in net:
        assert layer.moe.status()[0] == moe.MOE_OK
        layer.moe.close()
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK
    return diff.max().item(), last


if __name__ == "__main__":
    moe.build()
    diff, last = run()
    print(f"{last.shape[0]} sequences decoded; attention over the cache against attention over its values read back: "
          f"{diff:.2e} (rms of a head's row, relative)")
