#!/usr/bin/env python3
"""The feed-forward half of a decoder block on the library's calls: output projection, residual norm, MoE layer.

    o  [T, Ha]  attention output          ->  r = o Wo^T             (MxLinear: 4-bit activations and weights)
    h  [T, H]   residual stream           ->  h += r, n = norm(h)    (fp4moe_add_rmsnorm: n in bf16 and in block FP8)
    n                                      ->  y = experts(n)         (router and routed experts read the bf16 n, the
                                                                      shared expert its FP8 copy)

y is left to be added to the stream by the next norm. Every step is one call on one stream without host
synchronisation, so a step can be captured into a CUDA graph after it has run once.

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


if __name__ == "__main__":
    main()
