"""GPU: the MoE layer fed by the residual norm, and the whole example block (projection, norm, experts).

* moe_shared_expert_fp8 on the codes that moe_shared_expert itself makes of x: the same bits, with any scale stride;
* moe_shared_expert_fp8 on the norm's codes against the FP8 definition in fp64;
* moe_forward_shared_fp8 against moe_forward_shared on the same x, and the block against its steps in fp64;
* the block in a CUDA graph, replayed on new inputs, equals eager.
"""
import os
import sys

import numpy as np
import pytest

import synthgen as sg
from dense_ref import MX, NV, e4m3_half_step, quantize, rms_norm, values
from helpers import ROOT, bits_to_torch, ensure_built, float_parity, make_layer, torch_to_bits
from oracle import codecs, fp8block, moe
from test_gpu_shared_expert import gpu_o_shared, gpu_shared_weights, layer_with_shared, shared_cfg

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def own_codes(cfg, ws, wl, T):
    """The activation codes and scales that moe_shared_expert left in its workspace ([tcap][H], [H / 128][tcap])."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    cfg0 = shared_cfg(wl, cfg.max_tokens, shared_inter=0)
    base, tcap = api.workspace_bytes(cfg0), (cfg.max_tokens + 127) // 128 * 128
    off = base + (tcap * cfg.hidden + 255) // 256 * 256
    codes = ws[base:base + T * cfg.hidden].view(T, cfg.hidden)
    scales = ws[off:off + 4 * tcap * (cfg.hidden // 128)].view(torch.float32).view(-1, tcap)
    return codes.clone(), scales.clone()


@pytest.mark.parametrize("T,stride", [(1, 1), (7, 7), (130, 130), (200, 200), (200, 213)])
def test_shared_expert_fp8_equals_its_own_quantisation(T, stride):
    import torch
    from block_scaled_fp4_top_gb300 import api
    wl = sg.TINY_SHARED
    cfg = shared_cfg(wl, wl.T)
    se = gpu_shared_weights(cfg, sg.shared_w1_f32(wl), sg.shared_w2_f32(wl))
    x = sg.activations_bf16(wl, sg.EVAL_SEED)[:T]
    want, ws = gpu_o_shared(cfg, se, x)
    codes, scales = own_codes(cfg, ws, wl, T)
    sc = torch.full((wl.H // 128, stride), float("nan"), device="cuda")
    sc[:, :T] = scales[:, :T]
    ws2 = torch.zeros(api.workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    o = torch.full((T, wl.H), float("nan"), device="cuda")
    api.moe_shared_expert_fp8(cfg, T, codes, sc, se, o, ws2)
    torch.cuda.synchronize()
    assert api.fp4moe_read_error(ws2) == 0
    assert (o.cpu().numpy().astype(np.float64) == want).all()


def test_shared_expert_on_fresh_weights_right_behind_their_quantisation():
    """The FP8 call has no kernel of its own between the caller's last one and the GEMM that streams the weights."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    wl = sg.TINY_SHARED
    cfg = shared_cfg(wl, wl.T)
    w1, w2 = torch.from_numpy(sg.shared_w1_f32(wl)).cuda(), torch.from_numpy(sg.shared_w2_f32(wl)).cuda()
    se = gpu_shared_weights(cfg, None, None, w1, w2)
    _, ws = gpu_o_shared(cfg, se, sg.activations_bf16(wl, sg.EVAL_SEED))
    codes, scales = own_codes(cfg, ws, wl, wl.T)
    outs = []
    for _ in range(3):
        o = torch.empty(wl.T, wl.H, device="cuda")
        api.moe_shared_expert_fp8(cfg, wl.T, codes, scales, se, o, ws)
        torch.cuda.synchronize()
        outs.append(o)
    for _ in range(20):
        for t in (se.w1, se.w2):
            t.zero_()
        o = torch.empty(wl.T, wl.H, device="cuda")
        torch.cuda.synchronize()
        api.fp4moe_shared_quantize_weights(cfg, 1, w1, se.w1, se.w1_scales)
        api.fp4moe_shared_quantize_weights(cfg, 2, w2, se.w2, se.w2_scales)
        api.moe_shared_expert_fp8(cfg, wl.T, codes, scales, se, o, ws)
        torch.cuda.synchronize()
        assert torch.equal(o, outs[0])


def test_shared_expert_on_the_norms_codes():
    import torch
    from block_scaled_fp4_top_gb300 import api
    wl = sg.TINY_SHARED
    T, H = wl.T, wl.H
    cfg = shared_cfg(wl, T)
    w1, w2 = sg.shared_w1_f32(wl), sg.shared_w2_f32(wl)
    se = gpu_shared_weights(cfg, w1, w2)
    x = bits_to_torch(sg.activations_bf16(wl, sg.EVAL_SEED))
    gen = torch.Generator(device="cuda").manual_seed(5)
    gamma = (1 + 0.1 * torch.randn(H, device="cuda", generator=gen)).to(torch.bfloat16)
    n = torch.empty_like(x)
    codes, scales = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(H // 128, T, device="cuda")
    api.fp4moe_add_rmsnorm(x, None, gamma, 1e-6, None, n, codes, scales)
    ws = torch.zeros(api.workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    o = torch.empty(T, H, device="cuda")
    api.moe_shared_expert_fp8(cfg, T, codes, scales, se, o, ws)
    torch.cuda.synchronize()
    assert api.fp4moe_read_error(ws) == 0
    q = fp8block.quantize_shared(w1, w2)
    xt = codecs.E4M3_TABLE[codes.cpu().numpy()] * np.repeat(scales.cpu().numpy().T.astype(np.float64), 128, axis=1)
    gu = xt @ fp8block.dequantize_blocks(q.w1_q, q.w1_s).T
    hh = moe.swiglu(gu[:, :wl.shared_I], gu[:, wl.shared_I:], wl.swiglu_limit)
    hq, hs = fp8block.quantize_groups(hh.astype(np.float32))
    w2f = fp8block.dequantize_blocks(q.w2_q, q.w2_s)
    ref = fp8block.dequantize_groups(hq, hs) @ w2f.T
    got = o.cpu().numpy().astype(np.float64)
    # fp32 sums of either GEMM; and h's requantisation, where a sum a few ulps off lands on the other side of an E4M3
    # tie: a whole step of one feature, rare enough (an ulp against a step of 2^-3) that two of a token bound it
    step = 2 * e4m3_half_step(codecs.E4M3_TABLE[hq]) * np.repeat(hs.astype(np.float64), 128, axis=1)
    flip = (step[:, None, :] * np.abs(w2f)[None]).max(axis=2)
    bar = 1e-3 * np.sqrt((ref ** 2).mean()) + 2 * flip
    assert (np.abs(got - ref) <= bar).all() and np.linalg.norm(got - ref) <= 1e-2 * np.linalg.norm(ref)


def test_forward_shared_fp8_equals_forward_shared():
    import torch
    from block_scaled_fp4_top_gb300 import api
    wl = sg.TINY_SHARED
    layer = layer_with_shared(wl, wl.T)
    layer.calibrate(bits_to_torch(sg.activations_bf16(wl, sg.WARMUP_SEED)))
    x = bits_to_torch(sg.activations_bf16(wl, sg.EVAL_SEED))
    want, got = torch.empty_like(x), torch.empty_like(x)
    layer.forward(x, want)
    torch.cuda.synchronize()
    codes, scales = own_codes(layer.cfg, layer.ws, wl, wl.T)
    ids = torch.empty(wl.T * wl.k, dtype=torch.int32, device="cuda")
    layer.forward(x, got, ids, x_fp8=(codes, scales))
    torch.cuda.synchronize()
    assert layer.read_error() == 0
    assert torch.equal(want, got) and int(ids.min()) >= 0
    plain = make_layer(sg.TINY, sg.TINY.T)
    with pytest.raises(api.Fp4MoeError):
        plain.forward(x[:4], got[:4], x_fp8=(codes[:4], scales))
    with pytest.raises(api.Fp4MoeError):
        layer.forward(x, got, x_fp8=(codes[:4], scales))


@pytest.mark.parametrize("fmt", [MX, NV])
def test_block_against_its_steps(fmt):
    import torch
    from decoder_block import inputs, make_block
    wl = sg.TINY_SHARED
    Ka = 416                                                       # an attention width of its own
    block, wo = make_block(wl, Ka, fmt)
    o, h = inputs(wl, Ka, 11)
    h0 = h.clone()
    y = block.forward(o, h)
    torch.cuda.synchronize()
    assert block.read_error() == 0
    gx = 1.0 if fmt == MX else block.proj.gx.item()
    gw = 1.0 if fmt == MX else block.proj.gw.item()
    qa, qw = quantize(fmt, o.float().cpu().numpy(), gx), quantize(fmt, wo.cpu().numpy(), gw)
    r = values(fmt, *qa, Ka) @ values(fmt, *qw, Ka).T / (np.float64(np.float32(gx)) * np.float64(np.float32(gw)))
    got_r = block.r[:wl.T].float().cpu().numpy().astype(np.float64)
    assert (np.abs(got_r - r) <= np.abs(r) * (2.0 ** -8 + 2.0 ** -20) + 1e-5 * np.abs(r).max()).all()
    assert torch.equal(h, (block.r[:wl.T].float() + h0.float()).to(torch.bfloat16))
    n = rms_norm(h.float().cpu().numpy().astype(np.float64), block.gamma.float().cpu().numpy().astype(np.float64), block.eps)
    got_n = block.n[:wl.T].float().cpu().numpy().astype(np.float64)
    assert (np.abs(got_n - n) <= np.abs(n) * (2.0 ** -8 + 2.0 ** -20)).all()
    # the FP8 copy: half a step of E4M3 under the group's scale; and the experts on exactly these inputs
    sc = np.repeat(block.scales.cpu().numpy().T.astype(np.float64), 128, axis=1)
    amax = np.abs(n.reshape(wl.T, -1, 128)).max(2).repeat(128, 1)
    assert (np.abs(sc - amax / 448) <= amax / 448 * 2.0 ** -18).all()
    v = codecs.E4M3_TABLE[block.codes.view(torch.uint8).cpu().numpy()]
    assert (np.abs(v - n / sc) <= e4m3_half_step(n / sc) * (1 + 2.0 ** -10) + np.abs(n / sc) * 2.0 ** -18).all()
    want = torch.empty_like(y)
    block.moe.forward(block.n[:wl.T].contiguous(), want, x_fp8=(block.codes, block.scales))
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_block_in_a_graph_and_with_fewer_tokens():
    import torch
    from decoder_block import inputs, make_block
    wl = sg.TINY_SHARED
    block, _ = make_block(wl, wl.H)
    o, h = inputs(wl, wl.H, 21)
    block.forward(o, h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg = block.forward(o, h)
    for seed in (31, 32):
        o2, h2 = inputs(wl, wl.H, seed)
        o.copy_(o2)
        h.copy_(h2)
        graph.replay()
        torch.cuda.synchronize()
        got = (h.clone(), yg.clone())
        y = block.forward(o2, h2)
        torch.cuda.synchronize()
        assert torch.equal(got[0], h2) and torch.equal(got[1], y)
    # the first 5 rows alone: rows do not depend on one another before the experts, and a token's expert row is its own
    o3, h3 = (t[:5].clone() for t in inputs(wl, wl.H, 32))
    y3 = block.forward(o3, h3)
    torch.cuda.synchronize()
    assert torch.equal(h3, got[0][:5])
    assert torch.equal(y3, got[1][:5])
    assert block.read_error() == 0


def test_example_runs():
    import subprocess
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_block.py"), "--tiny"], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "graph replay equals eager: True" in r.stdout and "error word 0x0" in r.stdout


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype,out_dtype", [("bfloat16", "bfloat16"), ("float16", "float32"), ("float32", "float16")])
def test_linear_is_its_two_calls(fmt, dtype, out_dtype):
    import torch
    from block_scaled_fp4_top_gb300 import api
    N, K, most = 200, 300, 130
    gen = torch.Generator("cuda").manual_seed(5)
    w = torch.randn(N, K, generator=gen, device="cuda")
    lin = api.MxLinear(w, most, fmt)
    x = torch.randn(most, K, generator=gen, device="cuda").to(getattr(torch, dtype))
    lin.calibrate(x)
    for T in (1, 129, 64, 0, most):
        out = torch.full((T, N), 7.0, dtype=getattr(torch, out_dtype), device="cuda")
        lin.forward(x[:T], out)
        codes = torch.empty(T * api.mx_row_bytes(K), dtype=torch.uint8, device="cuda")
        sf = torch.empty(api.mx_sf_bytes(fmt, T, K), dtype=torch.uint8, device="cuda")
        ref = torch.empty_like(out)
        api.fp4moe_mx_quantize(fmt, x[:T], lin.gx, codes, sf)
        api.fp4moe_mx_gemm(fmt, K, codes, sf, lin.w_codes, lin.w_sf, lin.alpha, ref, lin.err)
        assert torch.equal(out, ref), T
    assert lin.read_error() == 0


def test_linear_refusals():
    import torch
    from block_scaled_fp4_top_gb300 import api
    lin = api.MxLinear(torch.randn(64, 96, device="cuda"), 8, MX)
    ok = lambda t, n: torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    for x, out in ((ok(9, 96), ok(9, 64)), (ok(4, 95), ok(4, 64)), (ok(4, 96), ok(4, 63)), (ok(4, 96), ok(5, 64)),
                   (ok(4, 96).cpu(), ok(4, 64)), (ok(4, 96), ok(4, 64).cpu()), (ok(4, 192)[:, ::2], ok(4, 64)),
                   (ok(4, 96).double(), ok(4, 64)), (ok(4, 96)[0], ok(4, 64))):
        with pytest.raises(api.Fp4MoeError):
            lin.forward(x, out)


def test_linear_in_nvfp4_needs_an_activation_scale():
    """Without one, small blocks' scales would underflow and large ones saturate without a word."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    w, x = torch.randn(64, 96, device="cuda"), torch.randn(4, 96, device="cuda").to(torch.bfloat16)
    lin, out = api.MxLinear(w, 8, NV), torch.full((4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(api.Fp4MoeError, match="scale"):
        lin.forward(x, out)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    lin.calibrate(x)
    lin.forward(x, out)
    gs = lin.gx.item()
    other, again = api.MxLinear(w, 8, NV), torch.empty_like(out)
    other.set_activation_scale(gs)
    other.forward(x, again)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and lin.read_error() == 0 and other.read_error() == 0
    with pytest.raises(api.Fp4MoeError, match="global scale"):
        api.MxLinear(w, 8, MX).set_activation_scale(1.0)
    api.MxLinear(w, 8, MX).forward(x, out)
