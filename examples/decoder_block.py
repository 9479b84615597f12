#!/usr/bin/env python3
"""A decoder block on the library's calls. Its attention half (Attention): norm, projection, rotary positions, paged cache;

    h  [T, H]   residual stream           ->  n = norm(h)            (fp4moe_add_rmsnorm)
    n                                      ->  q, k, v                (MxLinear, one product)
    lengths of the step's sequences        ->  pages, slots           (PagedKvCache.plan: once a step, for all layers)
    q, k, v                                ->  q turned, k and v into their pages, o = attention (append, attend)

and its feed-forward half (DecoderBlock): output projection, residual norm, MoE layer.

    o  [T, Ha]  attention output          ->  r = o Wo^T             (MxLinear: 4-bit activations and weights)
    h  [T, H]   residual stream           ->  h += r, n = norm(h)    (fp4moe_add_rmsnorm: n in bf16 and in block FP8)
    n                                      ->  y = experts(n)         (router and routed experts read the bf16 n, the
                                                                      shared expert its FP8 copy)

y is left to be added to the stream by the next norm. Every step is one call on one stream without host
synchronisation, so a step can be captured into a CUDA graph after it has run once; the graph of a decode step serves
every later step, since the lengths advance on the device.

    python examples/decoder_block.py            # DeepSeek-V4-Flash's sizes, 64 tokens: eager and graph times
    python examples/decoder_block.py --tiny     # a few experts, hidden 256
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synthgen as sg  # noqa: E402
from block_scaled_fp4_top_gb300 import _lib, api  # noqa: E402
from synthgen import gpu as sgpu  # noqa: E402


class DecoderBlock:
    """Output projection, residual norm and MoE layer of one block, for at most max_tokens rows."""

    def __init__(self, wo: torch.Tensor, gamma: torch.Tensor, moe: api.MoELayer, fmt: int = _lib.W_MXFP4,
                 eps: float = 1e-6):
        T, H = moe.cfg.max_tokens, moe.cfg.hidden
        self.proj = api.MxLinear(wo, T, fmt)
        self.gamma, self.eps, self.moe = gamma, eps, moe
        bf16 = dict(dtype=torch.bfloat16, device=wo.device)
        self.r, self.n, self.y = (torch.empty(T, H, **bf16) for _ in range(3))
        self.codes = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=wo.device)
        self.scales = torch.empty(H // 128, T, dtype=torch.float32, device=wo.device)

    def forward(self, o: torch.Tensor, h: torch.Tensor, stream=None) -> torch.Tensor:
        """h [T, H] is updated in place; the experts' output y [T, H] is returned (a view of the block's buffer)."""
        T = o.shape[0]
        r, n, y, codes = self.r[:T], self.n[:T], self.y[:T], self.codes[:T]
        self.proj.forward(o, r, stream)
        fp8 = self.moe.shared is not None
        api.fp4moe_add_rmsnorm(r, h, self.gamma, self.eps, h, n, codes if fp8 else None, self.scales if fp8 else None,
                               stream)
        self.moe.forward(n, y, stream=stream, x_fp8=(codes, self.scales) if fp8 else None)
        return y

    def read_error(self) -> int:
        return self.proj.read_error() | self.moe.read_error()


class Attention:
    """The attention half of one block, for steps of at most max_rows rows over a PagedKvCache."""

    def __init__(self, wqkv: torch.Tensor, gamma: torch.Tensor, heads: int, cache: api.PagedKvCache, max_rows: int,
                 layer: int = 0, fmt: int = _lib.W_MXFP4, eps: float = 1e-6, base: float = 10000.0):
        D = cache.k[0].shape[3]
        self.heads, self.kv_heads, self.cache, self.layer = heads, cache.k[0].shape[2], cache, layer
        self.proj, self.gamma, self.eps = api.MxLinear(wqkv, max_rows, fmt), gamma, eps
        self.inv_freq, self.scale = api.rope_inv_freq(D, base, device=wqkv.device), D ** -0.5
        bf16 = dict(dtype=torch.bfloat16, device=wqkv.device)
        self.n = torch.empty(max_rows, wqkv.shape[1], **bf16)
        self.qkv = torch.empty(max_rows, heads + 2 * self.kv_heads, D, **bf16)
        self.o = torch.empty(max_rows, heads, D, **bf16)

    def forward(self, h: torch.Tensor, stream=None) -> torch.Tensor:
        """o [T, heads * D] (a view of the layer's buffer) of the step's rows h [T, H], which the cache's plan placed."""
        T, H, K = h.shape[0], self.heads, self.kv_heads
        n, qkv, o = self.n[:T], self.qkv[:T], self.o[:T]
        api.fp4moe_add_rmsnorm(h, None, self.gamma, self.eps, None, n, stream=stream)
        self.proj.forward(n, qkv.flatten(1), stream)
        q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        self.cache.append(q, k, v, self.inv_freq, q, layer=self.layer, stream=stream)
        self.cache.attend(q, self.scale, o, layer=self.layer, stream=stream)
        return o.flatten(1)

    def read_error(self) -> int:
        return self.proj.read_error() | self.cache.read_error()


def make_attention(wl: sg.Workload, heads: int, kv_heads: int, head_dim: int, cache: api.PagedKvCache, max_rows: int,
                   layer: int = 0, seed: int = 3):
    """An attention half of the workload's hidden size with synthetic weights."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    wqkv = torch.randn((heads + 2 * kv_heads) * head_dim, wl.H, device="cuda", generator=gen) * wl.H ** -0.5
    gamma = (1 + 0.1 * torch.randn(wl.H, device="cuda", generator=gen)).to(torch.bfloat16)
    return Attention(wqkv, gamma, heads, cache, max_rows, layer)


def make_block(wl: sg.Workload, attn_width: int, fmt: int = _lib.W_MXFP4, chunk: int = 16, seed: int = 1):
    """A block of the workload's sizes with synthetic weights, its MoE layer calibrated on a warm-up batch."""
    cfg = api.config(wl.H, wl.I, wl.E, wl.k, wl.T, wl.swiglu_limit, shared_inter=wl.shared_I)
    moe = api.MoELayer(cfg)
    for e0 in range(0, wl.E, chunk):
        n = min(chunk, wl.E - e0)
        moe.quantize_weights(1, e0, sgpu.expert_w1(wl, e0, n))
        moe.quantize_weights(2, e0, sgpu.expert_w2(wl, e0, n))
    if wl.shared_I:
        moe.quantize_shared_weights(1, sgpu.shared_w1(wl))
        moe.quantize_shared_weights(2, sgpu.shared_w2(wl))
    moe.set_router(sgpu.router(wl))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    wo = torch.randn(wl.H, attn_width, device="cuda", generator=gen) * attn_width ** -0.5
    gamma = (1 + 0.1 * torch.randn(wl.H, device="cuda", generator=gen)).to(torch.bfloat16)
    block = DecoderBlock(wo, gamma, moe, fmt)
    o, h = inputs(wl, attn_width, seed + 1)
    block.proj.calibrate(o)
    n = torch.empty_like(h)
    block.proj.forward(o, block.r[:wl.T])
    api.fp4moe_add_rmsnorm(block.r[:wl.T], h, gamma, block.eps, h, n)
    moe.calibrate(n)
    return block, wo


def inputs(wl: sg.Workload, attn_width: int, seed: int):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    o = torch.randn(wl.T, attn_width, device="cuda", generator=gen).to(torch.bfloat16)
    h = torch.randn(wl.T, wl.H, device="cuda", generator=gen).to(torch.bfloat16)
    return o, h


def _time(fn, reps: int) -> float:
    for _ in range(3):
        fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(reps):
        fn()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) * 1e3 / reps


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tiny", action="store_true")
    ap.add_argument("--nvfp4", action="store_true", help="the projection in NVFP4 instead of MXFP4")
    args = ap.parse_args()
    wl = sg.TINY_SHARED if args.tiny else sg.DSV4_DECODE_SHARED
    block, _ = make_block(wl, wl.H, _lib.W_NVFP4 if args.nvfp4 else _lib.W_MXFP4)
    o, h = inputs(wl, wl.H, 7)
    h0 = h.clone()
    y = block.forward(o, h).clone()
    torch.cuda.synchronize()
    print(f"{wl.name}: T={wl.T} H={wl.H}, |h| {h.float().abs().mean():.3f}, |y| {y.float().abs().mean():.3f}, "
          f"error word {block.read_error():#x}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg = block.forward(o, h)
    h.copy_(h0)
    graph.replay()
    torch.cuda.synchronize()
    print("graph replay equals eager:", torch.equal(y, yg))
    print(f"eager {_time(lambda: block.forward(o, h), 200):.1f} us, graph {_time(graph.replay, 200):.1f} us a step")
    decode(wl, block, 64 if args.tiny else 4096)


def decode(wl: sg.Workload, block: DecoderBlock, prompt: int, steps: int = 50):
    """The whole block: one prompt for each of T sequences, in chunks of a sequence, then decode steps by a graph."""
    T, D = wl.T, 64 if wl.H < 1024 else 128
    heads, kv_heads = wl.H // D, max(1, wl.H // D // 4)
    rows = max(prompt, T)
    cache = api.PagedKvCache(T * ((prompt + steps) // 64 + 2), 64, kv_heads, D, T, prompt + 4 * steps, rows)
    attn = make_attention(wl, heads, kv_heads, D, cache, rows)
    gen = torch.Generator(device="cuda").manual_seed(9)
    new = torch.zeros(T, dtype=torch.int32, device="cuda")
    for b in range(T):  # (the experts of the block are sized for T rows, so prompts run through its attention half)
        new.zero_()
        new[b] = prompt - b % 7
        cache.plan(new, rows=prompt - b % 7)
        attn.forward(torch.randn(prompt - b % 7, wl.H, device="cuda", generator=gen).to(torch.bfloat16))
    new.fill_(1)
    h = torch.randn(T, wl.H, device="cuda", generator=gen).to(torch.bfloat16)

    def step():
        cache.plan(new, rows=T)
        return block.forward(attn.forward(h), h)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    print(f"decode over {prompt} cached tokens, {heads} heads of {D} on {kv_heads}: {_time(graph.replay, steps - 5):.1f} us a "
          f"step, error word {attn.read_error() | block.read_error():#x}, {int(cache.kv_len[0])} tokens of sequence 0")


if __name__ == "__main__":
    main()
