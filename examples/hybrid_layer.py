"""A decoder layer of a linear-attention model with mixture-of-experts blocks,
on the library's operators: packed prompts first, then single tokens of all
sequences in a CUDA graph.

    residual stream h, layer input x
    (codes, scales, h) = add_rmsnorm_fp8(x, w1, h)    residual add, norm, e4m3 rows
    qkv = matmul_fp8(codes, scales, W_qkv)            one projection for q, k and v
    o, S = gdn_decay_scan(q, k, v, decay, S)          slices of qkv; the state S is kept
    y = matmul_fp8(quantize_fp8(o), W_o)              output projection
    (n, h) = add_rmsnorm(y, w2, h)
    x = MoE(n)                                        the next layer's x

Run it on a GB300: python examples/hybrid_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_mixture_experts_gemm_gb300 as moe  # noqa: E402
from sparse_mixture_experts_gemm_gb300 import synth  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class HybridLayer:
    """Random weights of one layer; e4m3 projections with a scale per output
    channel, quantised once."""

    def __init__(self, seed, d, Hk, Hv, dk, dv, E, F, top_k, max_tokens, device):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g) * std).to(BF16).to(device)

        self.Hk, self.Hv, self.dk, self.dv = Hk, Hv, dk, dv
        self.w1 = (1 + 0.1 * normal(d)).to(BF16)
        self.w2 = (1 + 0.1 * normal(d)).to(BF16)
        self.Wqkv = moe.quantize_fp8(normal(2 * Hk * dk + Hv * dv, d, std=d ** -0.5))
        self.Wo = moe.quantize_fp8(normal(d, Hv * dv, std=(Hv * dv) ** -0.5))
        self.decay = (1 - torch.exp2(-5 - torch.arange(Hv, dtype=F32) % 8)).to(device)
        self.moe = moe.MoELayer(synth.layer_weights(seed + 1, d, F, E, 1, "bf16", device), top_k, max_tokens)

    def mixer(self, x, h, state, offsets=None, state_out=None):
        """Rows x of packed sequences (offsets), or of one token per sequence:
        (y, h, state)."""
        a, b = self.Hk * self.dk, 2 * self.Hk * self.dk
        codes, scales, h = moe.add_rmsnorm_fp8(x, self.w1, h)
        qkv = moe.matmul_fp8(codes, scales, *self.Wqkv)
        if offsets is None:
            qkv = qkv.unsqueeze(1)  # [n][1][..]: n sequences of one token
        q = qkv[..., :a].unflatten(-1, (self.Hk, self.dk))
        k = qkv[..., a:b].unflatten(-1, (self.Hk, self.dk))
        v = qkv[..., b:].unflatten(-1, (self.Hv, self.dv))
        o, state = moe.gdn_decay_scan(q, k, v, self.decay, state, offsets, state_out=state_out)
        y = moe.matmul_fp8(*moe.quantize_fp8(o.view(len(x), -1)), *self.Wo)
        return y, h, state

    def forward(self, x, h, state, offsets=None, state_out=None):
        """(x, h, state) of the next layer"""
        y, h, state = self.mixer(x, h, state, offsets, state_out)
        n, h = moe.add_rmsnorm(y, self.w2, h)
        return self.moe.forward(n), h, state


def run(lens=(37, 0, 130, 5), new=6, layers=2, device="cuda", seed=0):
    """Prompts of these lengths, then `new` tokens of each sequence; returns the
    greatest relative difference between the first layer's mixer in decoding
    and one pass over the whole sequences, and the last hidden rows."""
    d, Hk, Hv, dk, dv, E, F, top_k = 512, 2, 4, 128, 128, 16, 256, 4
    n, total = len(lens), sum(lens)
    net = [HybridLayer(seed + 10 * i, d, Hk, Hv, dk, dv, E, F, top_k, total + n, device) for i in range(layers)]
    g = torch.Generator().manual_seed(seed + 5)
    prompt = torch.randn(total, d, generator=g).to(BF16).to(device)
    tokens = torch.randn(new, n, d, generator=g).to(BF16).to(device)
    offsets = torch.tensor([0, *lens], device=device).cumsum(0).to(torch.int32)
    states = [torch.zeros(n, Hv, dv, dk, dtype=F32, device=device) for _ in net]

    # the prompts; each layer's states are updated in place
    x, h = prompt, torch.zeros_like(prompt)
    for layer, s in zip(net, states):
        x, h, _ = layer.forward(x, h, s, offsets, state_out=s)
    after_prompt = [s.clone() for s in states]

    # decoding: one step captured in a graph and replayed
    step_in = torch.zeros(n, d, dtype=BF16, device=device)

    def step():
        x, h, first = step_in, torch.zeros_like(step_in), None
        for layer, s in zip(net, states):
            y, h, _ = layer.mixer(x, h, s, state_out=s)
            first = y if first is None else first
            norm, h = moe.add_rmsnorm(y, layer.w2, h)
            x = layer.moe.forward(norm)
        return first, x + h

    side = torch.cuda.Stream(device)
    side.wait_stream(torch.cuda.current_stream(device))
    with torch.cuda.stream(side):
        step()  # (first calls are not captured)
    torch.cuda.current_stream(device).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first, last = step()
    for s, kept in zip(states, after_prompt):
        s.copy_(kept)
    mixed = []
    for t in tokens:
        step_in.copy_(t)
        graph.replay()
        mixed.append(first.clone())

    # the first layer's mixer again, in one pass over prompt and new tokens
    parts, lo = [], 0
    for i, length in enumerate(lens):
        parts += [prompt[lo:lo + length], tokens[:, i]]
        lo += length
    whole = torch.cat(parts)
    ends = torch.tensor([0, *(length + new for length in lens)], device=device).cumsum(0).to(torch.int32)
    y, _, state = net[0].mixer(whole, torch.zeros_like(whole), None, ends)
    rows = torch.stack([y[int(e) - new:int(e)] for e in ends[1:]], 1).float()
    diff = (torch.stack(mixed).float() - rows).norm(dim=-1) / rows.norm(dim=-1)
    sdiff = (states[0] - state).abs().amax() / state.abs().amax()
    torch.cuda.synchronize(device)
    for layer in net:
        assert layer.moe.status()[0] == moe.MOE_OK
        layer.moe.close()
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK
    return diff.max().item(), sdiff.item(), last


if __name__ == "__main__":
    moe.build()
    diff, sdiff, last = run()
    print(f"{last.shape[0]} sequences decoded; decoding against one pass: mixer outputs {diff:.2e} "
          f"(rms of a row, relative), states {sdiff:.2e}")
