"""One decoder layer's decode step on NVFP4 weights and an NVFP4 key/value cache, in one CUDA graph.

    x -> norm (E4M3) -> q, k, v projection -> append -> attention -> output projection
      -> residual addition + norm (BF16 and E4M3) -> shared expert (SwiGLU, E4M3 in)
      -> + routed experts (NVFP4RoutedMoE, from the BF16 norm) -> residual addition

Every product, norm and attention is a call of this library; torch allocates, computes the router's
logits and top-k, and captures the graph. Position encodings are left to the caller. Run it
(`python examples/decode_layer.py`) for the time of a step of a 2048-wide layer.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_routed_moe_sort_gb300 as moe  # noqa: E402


class DecodeLayer:
    """Weights of one layer (random here) and the buffers of a batch of single new tokens."""

    def __init__(self, batch, hidden=2048, heads=16, kv_heads=4, head_dim=128, experts=128, top_k=10, inter=512,
                 shared_inter=512, pages=256, page_size=64, max_pages=32, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, device=device, generator=gen)

        def matrix(n, k):
            return (normal(n, k) / k ** 0.5).bfloat16()

        self.heads, self.kv_heads, self.head_dim, self.top_k = heads, kv_heads, head_dim, top_k
        rows = heads + 2 * kv_heads
        # kept in BF16 beside their encoded forms for whoever wants to compare; a server would drop them
        self.w = {"qkv": matrix(rows * head_dim, hidden), "out": matrix(hidden, heads * head_dim),
                  "shared_in": matrix(2 * shared_inter, hidden), "shared_out": matrix(hidden, shared_inter),
                  "router": matrix(experts, hidden), "norm1": (1 + 0.1 * normal(hidden)).bfloat16(),
                  "norm2": (1 + 0.1 * normal(hidden)).bfloat16(),
                  "w1": (normal(experts, 2 * inter, hidden) / hidden ** 0.5).bfloat16(),
                  "w2": (normal(experts, hidden, inter) / inter ** 0.5).bfloat16()}
        self.qkv = moe.NVFP4Linear.from_bf16(self.w["qkv"])
        self.out = moe.NVFP4Linear.from_bf16(self.w["out"])
        self.shared_in = moe.NVFP4Linear.from_bf16(self.w["shared_in"], "swiglu")
        self.shared_out = moe.NVFP4Linear.from_bf16(self.w["shared_out"])
        self.routed = moe.NVFP4RoutedMoE(*moe.quantize_weights(self.w["w1"]), *moe.quantize_weights(self.w["w2"]),
                                         activation="swiglu", num_experts=experts)
        self.cache = moe.NVFP4KVCache.allocate(pages, page_size, kv_heads, head_dim, device)
        # what a step reads: refill in place between replays
        self.x = torch.zeros(batch, hidden, dtype=torch.bfloat16, device=device)        # the residual stream
        self.page_table = torch.zeros(batch, max_pages, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=device)            # new tokens included
        self.slots = torch.full((batch,), -1, dtype=torch.int64, device=device)         # of the new tokens
        self.graph = self.result = None

    def step(self) -> torch.Tensor:
        """The residual stream after the layer, [batch, hidden] bf16; x itself is left as it is."""
        B = self.x.shape[0]
        _, _, x8, scale = moe.add_rms_norm(self.x, self.w["norm1"], fp8="group")
        qkv = self.qkv(x8, scale).view(B, -1, self.head_dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        self.cache.append(k, v, self.slots)
        o, _ = self.cache.attend(q.unsqueeze(1), self.page_table, self.seq_lens)
        o = self.out(o.view(B, -1))
        y, h, y8, scale = moe.add_rms_norm(o, self.w["norm2"], residual=self.x, fp8="group")
        weights, ids = torch.softmax(y.float() @ self.w["router"].float().T, -1).topk(self.top_k)
        weights = weights / weights.sum(-1, keepdim=True)
        ffn = self.shared_out(self.shared_in(y8, scale))
        self.routed.forward(y, ids.int(), weights, do_finalize=2, out=ffn)  # adds the routed experts
        return h + ffn

    def capture(self) -> torch.cuda.CUDAGraph:
        """Captures a step; replay() then leaves its output in ``result``."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.result = self.step()
        return self.graph


def main():
    batch, steps, page = 8, 50, 64
    layer = DecodeLayer(batch)
    layer.x.copy_(torch.randn(layer.x.shape, device="cuda"))
    layer.page_table.copy_(torch.randperm(256, device="cuda").view(batch, 32).int())
    graph = layer.capture()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    place = torch.arange(batch, device="cuda")
    times = []
    for t in range(steps):  # each sequence grows by one token a step
        layer.seq_lens.fill_(t + 1)
        layer.slots.copy_(layer.page_table[place, t // page].long() * page + t % page)
        begin.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end) * 1e3)
        layer.x.copy_(layer.result / layer.result.float().square().mean(-1, keepdim=True).sqrt())
    status = int(layer.cache.dev_status[0])
    print(f"{batch} sequences, {steps} steps: {sorted(times)[steps // 2]:.1f} us a step, device status {status}")


if __name__ == "__main__":
    main()
