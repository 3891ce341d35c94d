"""One decoder layer of a serving step: attention over a paged 8-bit cache, then the MoE FFN.

    python examples/attention_step.py [--requests 8] [--context 1500] [--new 1] [--steps 4] [--hidden 1024]

Per step: block tables and slots from the requests' lengths.  Per layer: the input projection (E4M3, a scale for each
block of 128), the append of the new keys and values, attention, the output projection, the MoE layer.  Norms, rotary
embedding and residual sums, which a model has around these, are left out; weights and states are random.  A step is
captured in a CUDA graph once and replayed with the lengths on the device.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_scaled_fp4_moe_gb300 import attn, inputs, moe  # noqa: E402


class Layer:
    """Weights of one layer and the buffers of steps of up to T new tokens of B requests."""

    def __init__(self, B, T, hidden, blocks, width, q_heads=16, kv_heads=4, dim=64, block_size=32, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        dev = dict(device="cuda")

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen, **dev) * std).to(torch.bfloat16)

        self.B, self.T, self.q_heads, self.kv_heads, self.dim, self.block_size = B, T, q_heads, kv_heads, dim, block_size
        self.cache = attn.KVCache.empty(blocks, kv_heads, dim, block_size)
        self.w_in = attn.FP8Weight.from_dense(normal((q_heads + 2 * kv_heads) * dim, hidden, std=hidden ** -0.5))
        self.w_out = attn.FP8Weight.from_dense(normal(hidden, q_heads * dim, std=(q_heads * dim) ** -0.5))
        cfg = inputs.MoEConfig("step", T=T, H=hidden, E=8, top_k=2, I=512)
        self.bank = moe.MXFP4Bank.from_host(inputs.make_bank(cfg), cfg.E, cfg.has_shared)
        self.router = torch.from_numpy(inputs.make_router(cfg)[0]).cuda()
        i32 = dict(dtype=torch.int32, **dev)
        self.ctx, self.new = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.free, self.free_head, self.free_next = torch.arange(blocks, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
        self.table, self.kv_lens, self.q_offsets = torch.zeros(B, width, **i32), torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
        self.slots, self.positions = torch.zeros(T, dtype=torch.int64, **dev), torch.zeros(T, **i32)
        self.x = normal(T, hidden)
        self.qkv = torch.empty(T, q_heads + 2 * kv_heads, dim, dtype=torch.bfloat16, **dev)
        self.heads = torch.zeros(T, q_heads, dim, dtype=torch.bfloat16, **dev)     # rows without a token stay zero
        self.mixed, self.y = torch.empty_like(self.x), torch.empty_like(self.x)
        self.ws = attn.alloc_workspace(T, B, q_heads, self.cache, (self.w_in, self.w_out))
        self.moe_ws = moe.alloc_workspace(T, self.bank, cfg.top_k)
        self.top_k = cfg.top_k

    def step(self):
        """Everything on the current stream; lengths, tables and the free list's head on the device."""
        q, k = self.q_heads, self.q_heads + self.kv_heads
        attn.moe_kv_build_tables(self.ctx, self.new, self.block_size, self.free, self.free_head, self.table, self.kv_lens, self.q_offsets,
                                 self.slots, self.positions, self.free_next, self.ws)
        attn.moe_linear_fp8(self.x, self.w_in, self.qkv.view(self.T, -1), self.ws)
        attn.moe_kv_append(self.qkv[:, q:k], self.qkv[:, k:], self.slots, self.cache, self.ws)
        attn.moe_kv_attention(self.qkv[:, :q], self.cache, self.table, self.q_offsets, self.kv_lens, self.dim ** -0.5, self.heads, None,
                              self.ws)
        attn.moe_linear_fp8(self.heads.view(self.T, -1), self.w_out, self.mixed, self.ws)
        moe.moe_layer_forward(self.mixed, self.router, None, self.top_k, self.bank, 1.0, self.y, ws=self.moe_ws)
        self.ctx.add_(self.new)                            # the step's tokens are in the cache now
        self.free_head.copy_(self.free_next)

    def check(self):
        for ws in (self.ws, self.moe_ws):
            st = moe.moe_check_device_status(ws)
            if st != moe.MOE_OK:
                raise moe.MoEError(st, "step")


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--context", type=int, default=1500)
    ap.add_argument("--new", type=int, default=1, help="new tokens of each request and step")
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=1024)
    a = ap.parse_args(argv)
    B, size = a.requests, 32
    width = -(-(a.context + a.new * a.steps) // size)
    layer = Layer(B, max(B * a.new, 1), a.hidden, B * width, width, block_size=size)

    # prompts: a chunk at a time through the same calls, on buffers of the chunk's size
    gen = torch.Generator(device="cuda").manual_seed(1)
    done, chunk = 0, max(1, 2048 // B)
    while done < a.context:
        n = min(chunk, a.context - done)
        layer.new.fill_(n)
        slots, positions = torch.empty(B * n, dtype=torch.int64, device="cuda"), torch.empty(B * n, dtype=torch.int32, device="cuda")
        attn.moe_kv_build_tables(layer.ctx, layer.new, size, layer.free, layer.free_head, layer.table, layer.kv_lens, layer.q_offsets, slots,
                                 positions, layer.free_next, layer.ws)
        kv = torch.randn(B * n, 2 * layer.kv_heads, layer.dim, generator=gen, device="cuda").to(torch.bfloat16)
        attn.moe_kv_append(kv[:, :layer.kv_heads], kv[:, layer.kv_heads:], slots, layer.cache, layer.ws)
        layer.ctx.add_(layer.new)
        layer.free_head.copy_(layer.free_next)
        done += n
    layer.new.fill_(a.new)
    ctx, head = layer.ctx.clone(), layer.free_head.clone()
    layer.step()                                           # first step outside the graph
    layer.check()
    layer.ctx.copy_(ctx)
    layer.free_head.copy_(head)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.steps):
        graph.replay()
    stop.record()
    torch.cuda.synchronize()
    layer.check()
    out = dict(us_per_step=start.elapsed_time(stop) * 1e3 / a.steps, context=layer.ctx.tolist(), finite=bool(torch.isfinite(layer.y.float()).all()))
    print(f"{B} requests, {a.context} + {a.steps} x {a.new} tokens: {out['us_per_step']:.1f} us a step, outputs finite: {out['finite']}")
    return out


if __name__ == "__main__":
    main()
