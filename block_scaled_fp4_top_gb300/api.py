"""Python binding of the fp4moe C ABI: torch tensors in, C calls out.

Each function has the name of its C entry point and only marshals arguments:
it takes the device pointers of contiguous CUDA tensors and the current
stream, calls the library and raises Fp4MoeError on a non-OK status. All the
layer's arithmetic runs in the CUDA kernels of libfp4moe.so.

``MoELayer`` is a convenience owner of the buffers (allocated through torch)
for one configuration. It also runs the load-time prep: weight quantisation,
calibration and alpha tables. ``MxLinear`` is the same for a projection with
microscaled 4-bit weights, ``PagedKvCache`` for a key-value cache and the
attention over it.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import Config


class Fp4MoeError(RuntimeError):
    pass


def config(hidden: int, inter: int, num_experts: int, top_k: int, max_tokens: int, swiglu_limit: float,
           inter_logical: int = 0, w_format: int = _lib.W_NVFP4, ep_first: int = 0, ep_count: int = 0,
           shared_inter: int = 0) -> Config:
    """Layer configuration. ep_count > 0 makes the layer hold experts [ep_first, ep_first + ep_count) only;
    shared_inter > 0 gives it a block-FP8 shared expert of that (kernel-local) intermediate width."""
    return Config(hidden, inter, inter_logical or inter, num_experts, top_k, max_tokens, swiglu_limit, w_format,
                  ep_first, ep_count, shared_inter)


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda or not t.is_contiguous():
        raise Fp4MoeError("tensors must be contiguous CUDA tensors")
    return t.data_ptr()


# torch's own calls behind torch.cuda.current_stream(), absent from a build without CUDA
_raw_stream, _device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))


def _current_device():
    try:
        return _device()
    except (RuntimeError, TypeError):  # no driver, or a build without CUDA: no tensor is there
        return -2


def _s(stream):
    # the raw handle of the current stream, without building a torch.cuda.Stream (0.2 against 3 us a call)
    if stream is None:
        return _raw_stream(_device())
    return stream.cuda_stream


def _check(rc: int, what: str):
    if rc != _lib.OK:
        name = _lib.load().fp4moe_status_string(rc).decode()
        raise Fp4MoeError(f"{what}: {name}")


def capacity_rows(cfg: Config, T: int) -> int:
    return _lib.load().fp4moe_capacity_rows(ctypes.byref(cfg), T)


def workspace_bytes(cfg: Config) -> int:
    return _lib.load().fp4moe_workspace_bytes(ctypes.byref(cfg))


def weight_bytes(cfg: Config):
    v = [ctypes.c_size_t() for _ in range(4)]
    _check(_lib.load().fp4moe_weight_bytes(ctypes.byref(cfg), *[ctypes.byref(x) for x in v]), "fp4moe_weight_bytes")
    return tuple(x.value for x in v)


def moe_route(cfg, T, x, router_w, router_bias, logits_out, topk_ids, topk_w, counts, offsets, padded_offsets,
              slot_of_pair, pair_of_row, ws, stream=None):
    _check(_lib.load().moe_route(ctypes.byref(cfg), T, _p(x), _p(router_w), _p(router_bias), _p(logits_out),
                                 _p(topk_ids), _p(topk_w), _p(counts), _p(offsets), _p(padded_offsets),
                                 _p(slot_of_pair), _p(pair_of_row), _p(ws), _s(stream)), "moe_route")


def moe_route_noalloc(cfg, T, x, router_w, router_bias, logits_out, topk_ids, topk_w, counts, offsets,
                      padded_offsets, slot_of_pair, pair_of_row, err=None, stream=None):
    """moe_route without a workspace: for callers that must not allocate device
    memory. The library's own fixed scratch stands in for the workspace, so
    calls on one device must not overlap (see include/fp4moe.h)."""
    _check(_lib.load().moe_route_noalloc(ctypes.byref(cfg), T, _p(x), _p(router_w), _p(router_bias),
                                         _p(logits_out), _p(topk_ids), _p(topk_w), _p(counts), _p(offsets),
                                         _p(padded_offsets), _p(slot_of_pair), _p(pair_of_row), _p(err),
                                         _s(stream)), "moe_route_noalloc")


def moe_quantize_scatter(cfg, T, x, gs1, slot_of_pair, a1_fp4, a1_sf, ws, stream=None):
    _check(_lib.load().moe_quantize_scatter(ctypes.byref(cfg), T, _p(x), _p(gs1), _p(slot_of_pair), _p(a1_fp4),
                                            _p(a1_sf), _p(ws), _s(stream)), "moe_quantize_scatter")


def moe_grouped_gemm_w1_swiglu(cfg, T, a1_fp4, a1_sf, padded_offsets, pair_of_row, w1_fp4, w1_sf, alpha1, gs2,
                               a2_fp4, a2_sf, ws, stream=None):
    _check(_lib.load().moe_grouped_gemm_w1_swiglu(ctypes.byref(cfg), T, _p(a1_fp4), _p(a1_sf), _p(padded_offsets),
                                                  _p(pair_of_row), _p(w1_fp4), _p(w1_sf), _p(alpha1), _p(gs2),
                                                  _p(a2_fp4), _p(a2_sf), _p(ws), _s(stream)),
           "moe_grouped_gemm_w1_swiglu")


def moe_grouped_gemm_w2(cfg, T, a2_fp4, a2_sf, padded_offsets, pair_of_row, w2_fp4, w2_sf, alpha2, o_pairs, ws,
                        stream=None):
    _check(_lib.load().moe_grouped_gemm_w2(ctypes.byref(cfg), T, _p(a2_fp4), _p(a2_sf), _p(padded_offsets),
                                           _p(pair_of_row), _p(w2_fp4), _p(w2_sf), _p(alpha2), _p(o_pairs), _p(ws),
                                           _s(stream)), "moe_grouped_gemm_w2")


def moe_combine(cfg, T, o_pairs, topk_w, y, stream=None):
    _check(_lib.load().moe_combine(ctypes.byref(cfg), T, _p(o_pairs), _p(topk_w), _p(y), _s(stream)), "moe_combine")


def moe_grouped_gemm_w2_combine(cfg, T, a2_fp4, a2_sf, padded_offsets, pair_of_row, w2_fp4, w2_sf, alpha2, topk_w,
                                y, ws, stream=None):
    _check(_lib.load().moe_grouped_gemm_w2_combine(ctypes.byref(cfg), T, _p(a2_fp4), _p(a2_sf), _p(padded_offsets),
                                                   _p(pair_of_row), _p(w2_fp4), _p(w2_sf), _p(alpha2), _p(topk_w),
                                                   _p(y), _p(ws), _s(stream)), "moe_grouped_gemm_w2_combine")


def moe_forward(cfg, T, x, router_w, router_bias, gs1, gs2, w1_fp4, w1_sf, alpha1, w2_fp4, w2_sf, alpha2, y,
                topk_ids_out, topk_w_out, ws, stream=None):
    _check(_lib.load().moe_forward(ctypes.byref(cfg), T, _p(x), _p(router_w), _p(router_bias), _p(gs1), _p(gs2),
                                   _p(w1_fp4), _p(w1_sf), _p(alpha1), _p(w2_fp4), _p(w2_sf), _p(alpha2), _p(y),
                                   _p(topk_ids_out), _p(topk_w_out), _p(ws), _s(stream)), "moe_forward")


def fp4moe_quantize_weights(cfg, which, n_experts, w, codes_out, sf_out, gs_out, stream=None):
    _check(_lib.load().fp4moe_quantize_weights(ctypes.byref(cfg), which, n_experts, _p(w), _p(codes_out),
                                               _p(sf_out), _p(gs_out), _s(stream)), "fp4moe_quantize_weights")


def fp4moe_mxfp4_as_nvfp4(cfg, which, n_experts, mx_codes, mx_sf, codes_out, sf_out, gw_out, err, stream=None):
    _check(_lib.load().fp4moe_mxfp4_as_nvfp4(ctypes.byref(cfg), which, n_experts, _p(mx_codes), _p(mx_sf),
                                             _p(codes_out), _p(sf_out), _p(gw_out), _p(err), _s(stream)),
           "fp4moe_mxfp4_as_nvfp4")


def fp4moe_tp_shard_units(width, tp, align, kernel_align, rank, unit):
    """(source offset, units copied, zero tail) of one rank's slice, in storage units (host arithmetic)."""
    out = [ctypes.c_int32() for _ in range(3)]
    _check(_lib.load().fp4moe_tp_shard_units(width, tp, align, kernel_align, rank, unit,
                                             *[ctypes.byref(v) for v in out]), "fp4moe_tp_shard_units")
    return tuple(v.value for v in out)


def fp4moe_shard_mxfp4(cfg, which, n_experts, full_inter, tp, tp_rank, ck_codes, ck_sf, codes_out, sf_out,
                       stream=None):
    _check(_lib.load().fp4moe_shard_mxfp4(ctypes.byref(cfg), which, n_experts, full_inter, tp, tp_rank, _p(ck_codes),
                                          _p(ck_sf), _p(codes_out), _p(sf_out), _s(stream)), "fp4moe_shard_mxfp4")


def fp4moe_make_alpha(n, gs_act, gs_w, alpha, stream=None):
    _check(_lib.load().fp4moe_make_alpha(n, _p(gs_act), _p(gs_w), _p(alpha), _s(stream)), "fp4moe_make_alpha")


def fp4moe_calibrate(cfg, T, x_warm, router_w, router_bias, w1_fp4, w1_sf, gw1, gs1_out, gs2_out, ws, stream=None):
    _check(_lib.load().fp4moe_calibrate(ctypes.byref(cfg), T, _p(x_warm), _p(router_w), _p(router_bias), _p(w1_fp4),
                                        _p(w1_sf), _p(gw1), _p(gs1_out), _p(gs2_out), _p(ws), _s(stream)),
           "fp4moe_calibrate")


def fp4moe_batch_gs1(cfg, T, x, gw1, gs1_out, alpha1_out, ws, stream=None):
    _check(_lib.load().fp4moe_batch_gs1(ctypes.byref(cfg), T, _p(x), _p(gw1), _p(gs1_out), _p(alpha1_out), _p(ws),
                                        _s(stream)), "fp4moe_batch_gs1")


def fp4moe_quantize_rows_f32(rows, K, inp, g, codes, sf, stream=None):
    _check(_lib.load().fp4moe_quantize_rows_f32(rows, K, _p(inp), _p(g), _p(codes), _p(sf), _s(stream)),
           "fp4moe_quantize_rows_f32")


def fp4moe_tensor_peak_probe(n, iters, err, stream=None):
    """Launch the dense FP4 tensor-core rate probe (see include/fp4moe.h); the caller times it."""
    _check(_lib.load().fp4moe_tensor_peak_probe(n, iters, _p(err), _s(stream)), "fp4moe_tensor_peak_probe")


def fp4moe_selftest_wait_timeout(err, limit_ns, result, stream=None):
    """One bounded wait that runs out on purpose (a test of the failure path; see include/fp4moe.h)."""
    _check(_lib.load().fp4moe_selftest_wait_timeout(_p(err), int(limit_ns), _p(result), _s(stream)),
           "fp4moe_selftest_wait_timeout")


def _sw(se):
    """fp4moe_shared_weights from a SharedWeights holder (device pointers of its four tensors)."""
    return ctypes.byref(_lib.SharedWeights(_p(se.w1), _p(se.w1_scales), _p(se.w2), _p(se.w2_scales)))


def shared_weight_bytes(cfg: Config):
    v = [ctypes.c_size_t() for _ in range(4)]
    _check(_lib.load().fp4moe_shared_weight_bytes(ctypes.byref(cfg), *[ctypes.byref(x) for x in v]),
           "fp4moe_shared_weight_bytes")
    return tuple(x.value for x in v)


def fp4moe_shared_quantize_weights(cfg, which, w, codes_out, scales_out, stream=None):
    _check(_lib.load().fp4moe_shared_quantize_weights(ctypes.byref(cfg), which, _p(w), _p(codes_out),
                                                      _p(scales_out), _s(stream)), "fp4moe_shared_quantize_weights")


def moe_shared_expert(cfg, T, x, se, o_shared, ws, stream=None):
    _check(_lib.load().moe_shared_expert(ctypes.byref(cfg), T, _p(x), _sw(se), _p(o_shared), _p(ws), _s(stream)),
           "moe_shared_expert")


def moe_combine_shared(cfg, T, o_pairs, topk_w, slot_of_pair, o_shared, y, stream=None):
    _check(_lib.load().moe_combine_shared(ctypes.byref(cfg), T, _p(o_pairs), _p(topk_w), _p(slot_of_pair),
                                          _p(o_shared), _p(y), _s(stream)), "moe_combine_shared")


def moe_forward_shared(cfg, T, x, router_w, router_bias, gs1, gs2, w1_fp4, w1_sf, alpha1, w2_fp4, w2_sf, alpha2, se,
                       y, topk_ids_out, topk_w_out, ws, stream=None):
    _check(_lib.load().moe_forward_shared(ctypes.byref(cfg), T, _p(x), _p(router_w), _p(router_bias), _p(gs1),
                                          _p(gs2), _p(w1_fp4), _p(w1_sf), _p(alpha1), _p(w2_fp4), _p(w2_sf),
                                          _p(alpha2), _sw(se), _p(y), _p(topk_ids_out), _p(topk_w_out), _p(ws),
                                          _s(stream)), "moe_forward_shared")


def fp4moe_read_error(ws, clear=True, stream=None) -> int:
    v = ctypes.c_uint32()
    _check(_lib.load().fp4moe_read_error(_p(ws), ctypes.byref(v), 1 if clear else 0, _s(stream)), "fp4moe_read_error")
    return v.value


def fp4moe_read_scale_status(ws, clear=True, stream=None):
    """(FP4MOE_SAT_* flags, running amax|h| since the last gs2 refresh)."""
    v, a = ctypes.c_uint32(), ctypes.c_float()
    _check(_lib.load().fp4moe_read_scale_status(_p(ws), ctypes.byref(v), ctypes.byref(a), 1 if clear else 0,
                                                _s(stream)), "fp4moe_read_scale_status")
    return v.value, a.value


def fp4moe_refresh_gs2(cfg, ws, gw2, gs2_inout, alpha2_out, stream=None):
    _check(_lib.load().fp4moe_refresh_gs2(ctypes.byref(cfg), _p(ws), _p(gw2), _p(gs2_inout), _p(alpha2_out),
                                          _s(stream)), "fp4moe_refresh_gs2")


def moe_shared_expert_fp8(cfg, T, x_codes, x_scales, se, o_shared, ws, stream=None):
    """moe_shared_expert on the FP8 copy that fp4moe_add_rmsnorm writes (x_scales [H / 128, at least T])."""
    _check_fp8(x_codes, x_scales, T, cfg.hidden, _current_device())
    _check(_lib.load().moe_shared_expert_fp8(ctypes.byref(cfg), T, _p(x_codes), _p(x_scales), x_scales.shape[1],
                                             _sw(se), _p(o_shared), _p(ws), _s(stream)), "moe_shared_expert_fp8")


def moe_forward_shared_fp8(cfg, T, x, x_codes, x_scales, router_w, router_bias, gs1, gs2, w1_fp4, w1_sf, alpha1,
                           w2_fp4, w2_sf, alpha2, se, y, topk_ids_out, topk_w_out, ws, stream=None):
    """moe_forward_shared with the shared expert fed from x's FP8 copy."""
    _check_fp8(x_codes, x_scales, T, cfg.hidden, _current_device())
    _check(_lib.load().moe_forward_shared_fp8(ctypes.byref(cfg), T, _p(x), _p(x_codes), _p(x_scales),
                                              x_scales.shape[1], _p(router_w), _p(router_bias), _p(gs1), _p(gs2),
                                              _p(w1_fp4), _p(w1_sf), _p(alpha1), _p(w2_fp4), _p(w2_sf), _p(alpha2),
                                              _sw(se), _p(y), _p(topk_ids_out), _p(topk_w_out), _p(ws), _s(stream)),
           "moe_forward_shared_fp8")


# ---------------------------------------------------------- dense operators
# Their sizes and types come from the tensors, so the shapes are checked here: the library sees only pointers.
# A small call is bound by the host, so each tensor is checked and turned into its pointer in one go. `dev` is the
# current device: kernels run there, and a matrix on another one would be read through a peer mapping or not at all.
_DTYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.FP16, torch.float32: _lib.FP32}
_BYTE_TYPES = (torch.uint8, torch.float8_e4m3fn)
_U8, _F32 = torch.uint8, torch.float32


def _place(name, t, dev):
    if t.get_device() != dev or not t.is_contiguous():  # (-1 for a CPU tensor)
        raise Fp4MoeError(f"{name}: expected a contiguous CUDA tensor on the current device")


def _arg(name, t, shape, dtype, dev):
    """The pointer of a contiguous tensor of this shape and type on the device; None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape:
        raise Fp4MoeError(f"{name}: expected {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous():
        _place(name, t, dev)
    return t.data_ptr()


def _arg_bytes(name, t, nbytes, dev):
    if t.dtype is not _U8 or t.numel() != nbytes:
        raise Fp4MoeError(f"{name}: expected {nbytes} bytes (uint8), got {t.numel()} of {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous():
        _place(name, t, dev)
    return t.data_ptr()


def _arg_scalar(name, t, dev):
    if t is None:
        return None
    if t.dtype is not _F32 or t.numel() < 1:
        raise Fp4MoeError(f"{name}: expected one float32, got {t.numel()} of {t.dtype}")
    _place(name, t, dev)
    return t.data_ptr()


def _arg_matrix(name, t, dev):
    """(shape, dtype, fp4moe_dtype, pointer) of a matrix whose sizes the call takes."""
    dt, shape = t.dtype, t.shape
    d = _DTYPES.get(dt)
    if d is None:
        raise Fp4MoeError(f"{name}: unsupported dtype {dt}: bfloat16, float16 or float32")
    if len(shape) != 2:
        raise Fp4MoeError(f"{name}: expected a matrix, got {tuple(shape)}")
    if t.get_device() != dev or not t.is_contiguous():
        _place(name, t, dev)
    return shape, dt, d, t.data_ptr()


def _check_fp8(codes, scales, T, H, dev):
    """Check block-FP8 activations: codes [T, H], scales [ceil(H / 128), at least T]. Returns the scales' columns."""
    if codes.dtype not in _BYTE_TYPES or codes.shape != (T, H):
        raise Fp4MoeError(f"codes: expected {(T, H)} of {' or '.join(map(str, _BYTE_TYPES))}, got "
                          f"{tuple(codes.shape)} of {codes.dtype}")
    shape = scales.shape
    if scales.dtype is not _F32 or len(shape) != 2 or shape[0] != (H + 127) // 128 or shape[1] < T:
        raise Fp4MoeError(f"scales: expected [{(H + 127) // 128}, at least {T}] of torch.float32, got "
                          f"{tuple(shape)} of {scales.dtype}")
    if codes.get_device() != dev or not codes.is_contiguous():
        _place("codes", codes, dev)
    if scales.get_device() != dev or not scales.is_contiguous():
        _place("scales", scales, dev)
    return shape[1]


def fp4moe_add_rmsnorm(x, residual, gamma, eps, residual_out, y, y_codes=None, y_scales=None, stream=None):
    """h = x + residual -> residual_out; y = h * rsqrt(mean(h^2) + eps) * gamma; y in E4M3 with a scale per 1 x 128
    group -> y_codes [T, H] (uint8 or float8_e4m3fn), y_scales [ceil(H / 128), at least T] float32.

    x [T, H] bfloat16, float16 or float32, and residual, residual_out, y, gamma [H] of its type. residual with
    residual_out, and y_codes with y_scales, may be None; so may gamma (ones), and y where y_codes is given.
    residual_out and y may each be x or residual."""
    dev = _current_device()
    shape, dt, d, px = _arg_matrix("x", x, dev)
    T, H = shape
    if y_codes is not None and y_scales is not None:
        stride = _check_fp8(y_codes, y_scales, T, H, dev)
        pc, ps = y_codes.data_ptr(), y_scales.data_ptr()
    else:  # both None, or refused by the call
        stride, pc, ps = 0, _p(y_codes), _p(y_scales)
    _check(_lib.load().fp4moe_add_rmsnorm(d, T, H, px, _arg("residual", residual, shape, dt, dev),
                                          _arg("gamma", gamma, (H,), dt, dev), eps,
                                          _arg("residual_out", residual_out, shape, dt, dev),
                                          _arg("y", y, shape, dt, dev),
                                          pc, ps, stride, _s(stream)), "fp4moe_add_rmsnorm")


def mx_row_bytes(K: int) -> int:
    """Bytes of one row of 4-bit codes: K rounded up to whole 32-element groups."""
    return (K + 31) // 32 * 16


def mx_sf_bytes(fmt: int, rows: int, K: int) -> int:
    """Bytes of a microscaled matrix's scale tiles (128 rows x 4 scale columns, 512 bytes each)."""
    span = 128 if fmt == _lib.W_MXFP4 else 64  # elements of K across a tile
    return (rows + 127) // 128 * ((K + span - 1) // span) * 512


def fp4moe_mx_bytes(fmt: int, rows: int, K: int):
    """(code bytes, scale bytes) of a [rows, K] matrix in the format W_MXFP4 or W_NVFP4."""
    v = [ctypes.c_size_t() for _ in range(2)]
    _check(_lib.load().fp4moe_mx_bytes(fmt, rows, K, *[ctypes.byref(x) for x in v]), "fp4moe_mx_bytes")
    return tuple(x.value for x in v)


def fp4moe_mx_quantize(fmt, x, gs, codes, sf, stream=None):
    """x [rows, K] to E2M1 codes and block scales (fmt W_MXFP4, or W_NVFP4 under the global scale gs)."""
    dev = _current_device()
    (rows, K), _, d, px = _arg_matrix("x", x, dev)
    _check(_lib.load().fp4moe_mx_quantize(fmt, d, rows, K, px, _arg_scalar("gs", gs, dev),
                                          _arg_bytes("codes", codes, rows * mx_row_bytes(K), dev),
                                          _arg_bytes("sf", sf, mx_sf_bytes(fmt, rows, K), dev), _s(stream)),
           "fp4moe_mx_quantize")


def fp4moe_mx_dequantize(fmt, codes, sf, gs, out, stream=None):
    """The values of a microscaled matrix into out [rows, K]."""
    dev = _current_device()
    (rows, K), _, d, po = _arg_matrix("out", out, dev)
    _check(_lib.load().fp4moe_mx_dequantize(fmt, d, rows, K,
                                            _arg_bytes("codes", codes, rows * mx_row_bytes(K), dev),
                                            _arg_bytes("sf", sf, mx_sf_bytes(fmt, rows, K), dev),
                                            _arg_scalar("gs", gs, dev), po, _s(stream)), "fp4moe_mx_dequantize")


def fp4moe_mx_gemm_plan(M: int, N: int, K: int, sms: int):
    """(tile rows, tile columns, K slices) of an M x N x K product on a device of `sms` SMs (host arithmetic)."""
    v = [ctypes.c_int32() for _ in range(3)]
    _check(_lib.load().fp4moe_mx_gemm_plan(M, N, K, sms, *[ctypes.byref(x) for x in v]), "fp4moe_mx_gemm_plan")
    return tuple(x.value for x in v)


def fp4moe_mx_gemm(fmt, K, a_codes, a_sf, b_codes, b_sf, alpha, out, err, stream=None):
    """out [M, N] = alpha * A B^T for microscaled A [M, K] and B [N, K]; alpha a device float32 or None (1); err a
    zeroed device word (int32) that the caller keeps."""
    dev = _current_device()
    (M, N), _, d, po = _arg_matrix("out", out, dev)
    row = mx_row_bytes(K)
    if err.element_size() * err.numel() < 4:
        raise Fp4MoeError("err: expected a device word of 4 bytes")
    _place("err", err, dev)
    _check(_lib.load().fp4moe_mx_gemm(fmt, d, M, N, K, _arg_bytes("a_codes", a_codes, M * row, dev),
                                      _arg_bytes("a_sf", a_sf, mx_sf_bytes(fmt, M, K), dev),
                                      _arg_bytes("b_codes", b_codes, N * row, dev),
                                      _arg_bytes("b_sf", b_sf, mx_sf_bytes(fmt, N, K), dev),
                                      _arg_scalar("alpha", alpha, dev), po, err.data_ptr(), _s(stream)),
           "fp4moe_mx_gemm")


# ------------------------------------------------- the paged key-value cache
_I32, _F64 = torch.int32, torch.float64
_KvCache = _lib.KvCache
_KV_DTYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.FP16}


def _arg_ints(name, t, n, dev):
    """The pointer of n int32 values (n None: any number of them)."""
    shape = t.shape
    if t.dtype is not _I32 or len(shape) != 1 or (n is not None and shape[0] != n):
        raise Fp4MoeError(f"{name}: expected {'a vector' if n is None else n} of {_I32}, got {tuple(t.shape)} of {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous():
        _place(name, t, dev)
    return t.data_ptr()


def _arg_table(name, t, B, dev):
    """(columns, pointer) of a page table of B rows."""
    if t.dtype is not _I32 or t.dim() != 2 or t.shape[0] != B:
        raise Fp4MoeError(f"{name}: expected [{B}, columns] of {_I32}, got {tuple(t.shape)} of {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous():
        _place(name, t, dev)
    return t.shape[1], t.data_ptr()


def _arg_err(err, dev):
    if err.nbytes < 4:
        raise Fp4MoeError("err: expected a device word of 4 bytes")
    if err.get_device() != dev or not err.is_contiguous():
        _place("err", err, dev)
    return err.data_ptr()


def _kv_cache(k_cache, v_cache, dev):
    """(fp4moe_kv_cache, pointer of k, pointer of v) of two caches [pages, page size, kv heads, head dim], each
    contiguous or a view of another order of pages, tokens and heads (the same for both)."""
    shape, dt = k_cache.shape, k_cache.dtype
    d = _KV_DTYPES.get(dt)
    if d is None or len(shape) != 4:
        raise Fp4MoeError("k_cache: expected [pages, page size, kv heads, head dim] of bfloat16 or float16, got "
                          f"{tuple(shape)} of {dt}")
    if v_cache.shape != shape or v_cache.dtype is not dt:
        raise Fp4MoeError(f"v_cache: expected {tuple(shape)} of {dt}, got {tuple(v_cache.shape)} of {v_cache.dtype}")
    if k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise Fp4MoeError("k_cache, v_cache: expected CUDA tensors on the current device")
    P, S, H, D = shape
    if k_cache.is_contiguous() and v_cache.is_contiguous():
        row = H * D
        return _KvCache(d, H, D, S, P, S * row, row, D), k_cache.data_ptr(), v_cache.data_ptr()
    # (the stride of a dimension of one element says nothing)
    st = [0 if n == 1 else s for n, s in zip(shape, k_cache.stride())]
    if st != [0 if n == 1 else s for n, s in zip(shape, v_cache.stride())] or st[3] != 1 or any(s % 8 for s in st[:3]):
        raise Fp4MoeError("k_cache, v_cache: expected the same strides, head dim contiguous, the others multiples of 8")
    return _lib.KvCache(d, H, D, S, P, st[0], st[1], st[2]), k_cache.data_ptr(), v_cache.data_ptr()


def _arg_heads(name, t, T, D, dt, dev):
    """(heads, row stride, pointer) of [T, heads, D]: whole rows, any distance apart."""
    shape = t.shape
    if t.dtype is not dt or len(shape) != 3 or shape[0] != T or shape[2] != D:
        raise Fp4MoeError(f"{name}: expected [{T}, heads, {D}] of {dt}, got {tuple(shape)} of {t.dtype}")
    row, head, one = t.stride()
    H = shape[1]
    if T <= 1:
        row = H * D
    if t.get_device() != dev or one != 1 or (H > 1 and head != D) or row % 8 or row < H * D:
        raise Fp4MoeError(f"{name}: expected rows of contiguous heads on the current device, a multiple of 8 elements apart")
    return H, row, t.data_ptr()


def rope_inv_freq(rot_dim: int, base: float = 10000.0, factor: float = 1.0, original_len: int | None = None,
                  slow: float = 1.0, fast: float = 32.0, device="cuda") -> torch.Tensor:
    """fp64 radians per position of the rot_dim / 2 pairs: base^(-2 i / rot_dim), scaled for contexts `factor` times as
    long. Without original_len all are divided by factor (positions are interpolated). With it, pairs that turn at least
    `fast` times in original_len positions keep their frequency, those that turn at most `slow` times are divided by
    factor, and in between the two are mixed linearly in the number of turns (YaRN, arXiv:2309.00071, section 3.2, which
    goes with an amplitude of 0.1 ln(factor) + 1)."""
    if rot_dim < 0 or rot_dim % 2 or not base > 0 or not factor > 0 or not fast > slow:
        raise Fp4MoeError("rope_inv_freq: rot_dim must be even, base and factor positive, fast above slow")
    f = torch.tensor([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], dtype=_F64)
    if original_len is None:
        f = f / factor
    else:
        keep = ((original_len * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f.to(device)


def fp4moe_kv_plan(page_size, cached_len, new_len, page_table, free_pages, free_count, kv_len, free_count_out, q_offset,
                   position, slot, err, stream=None):
    """A step's pages, row offsets, positions and cache slots from its sequences' lengths (all int32, on the device):
    cached_len, new_len (negative: tokens given back), kv_len [B]; page_table [B, columns]; free_pages [pages];
    free_count, free_count_out [1]; q_offset [B + 1]; position, slot [rows]. kv_len may be cached_len and free_count_out
    may be free_count."""
    dev = _current_device()
    B = cached_len.shape[0]
    columns, pt = _arg_table("page_table", page_table, B, dev)
    rows = slot.shape[0]
    _check(_lib.load().fp4moe_kv_plan(B, page_size, free_pages.shape[0], _arg_ints("cached_len", cached_len, B, dev),
                                      _arg_ints("new_len", new_len, B, dev), pt, columns,
                                      _arg_ints("free_pages", free_pages, None, dev),
                                      _arg_ints("free_count", free_count, 1, dev), _arg_ints("kv_len", kv_len, B, dev),
                                      _arg_ints("free_count_out", free_count_out, 1, dev),
                                      _arg_ints("q_offset", q_offset, B + 1, dev), rows,
                                      _arg_ints("position", position, rows, dev), _arg_ints("slot", slot, rows, dev),
                                      _arg_err(err, dev), _s(stream)), "fp4moe_kv_plan")


def fp4moe_rope_cache(q, k, v, position, slot, inv_freq, q_out, k_cache, v_cache, err, first=0, interleaved=False,
                      amplitude=1.0, stream=None):
    """Rotary positions of q [T, heads, D] -> q_out, and of k; k and v [T, kv heads, D] -> their slots of the caches
    [pages, page size, kv heads, D]. q, k and v may be column slices of one projection's rows; q_out may be q; q and
    q_out, or k and v, may be None. position, slot [T] int32; inv_freq fp64: the pairs of the turned part of the head,
    which starts at element `first` (rope_inv_freq)."""
    dev = _current_device()
    c, pk, pv = _kv_cache(k_cache, v_cache, dev)
    dt, D = k_cache.dtype, c.head_dim
    T = slot.shape[0]
    pairs = inv_freq.shape
    if inv_freq.dtype is not _F64 or len(pairs) != 1:
        raise Fp4MoeError(f"inv_freq: expected a vector of {_F64}, got {tuple(pairs)} of {inv_freq.dtype}")
    if inv_freq.get_device() != dev or not inv_freq.is_contiguous():
        _place("inv_freq", inv_freq, dev)
    Hq = q_stride = q_out_stride = k_stride = v_stride = 0
    ptr_q = ptr_qo = ptr_k = ptr_v = None
    if (q is None) != (q_out is None) or (k is None) != (v is None):
        raise Fp4MoeError("q and q_out, and k and v, are both given or both None")
    if q is not None:
        Hq, q_stride, ptr_q = _arg_heads("q", q, T, D, dt, dev)
        Ho, q_out_stride, ptr_qo = _arg_heads("q_out", q_out, T, D, dt, dev)
        if Ho != Hq:
            raise Fp4MoeError(f"q_out: expected {Hq} heads, got {Ho}")
        if ptr_q == ptr_qo and q_stride != q_out_stride:
            raise Fp4MoeError("q_out: in place means with q's own stride")
    if k is not None:
        Hk, k_stride, ptr_k = _arg_heads("k", k, T, D, dt, dev)
        Hv, v_stride, ptr_v = _arg_heads("v", v, T, D, dt, dev)
        if Hk != c.kv_heads or Hv != c.kv_heads:
            raise Fp4MoeError(f"k, v: expected the caches' {c.kv_heads} heads, got {Hk} and {Hv}")
    else:
        pk = pv = None
    _check(_lib.load().fp4moe_rope_cache(c, T, Hq, ptr_q, q_stride, ptr_k, k_stride, ptr_v, v_stride,
                                         _arg_ints("position", position, T, dev), _arg_ints("slot", slot, T, dev), first,
                                         2 * pairs[0], interleaved, inv_freq.data_ptr(), amplitude, ptr_qo,
                                         q_out_stride, pk, pv, _arg_err(err, dev), _s(stream)), "fp4moe_rope_cache")


def fp4moe_paged_attention_plan(num_seqs: int, T: int, heads: int, kv_heads: int, head_dim: int) -> int:
    """Rows of a tile (16, 32 or 256) of the kernel that fp4moe_paged_attention takes for these sizes (host arithmetic)."""
    v = ctypes.c_int32()
    c = _lib.KvCache(_lib.BF16, kv_heads, head_dim, 1, 1, 0, 0, 0)
    _check(_lib.load().fp4moe_paged_attention_plan(c, num_seqs, T, heads, ctypes.byref(v)), "fp4moe_paged_attention_plan")
    return v.value


def fp4moe_paged_attention(q, k_cache, v_cache, page_table, kv_len, q_offset, scale, out, lse, ws, err, causal=True,
                           window=0, stream=None):
    """out [T, heads, D] of q [T, heads, D] over each sequence's pages: rows q_offset[b] .. q_offset[b + 1] read the
    kv_len[b] keys of page_table[b]. causal: they are its last tokens, and each sees the keys up to its own (window > 0:
    the last `window` of them); else every row sees all keys. lse [T, heads] float32 or None; ws: a zeroed workspace of
    ATTENTION_WORKSPACE_BYTES that the caller keeps."""
    dev = _current_device()
    c, pk, pv = _kv_cache(k_cache, v_cache, dev)
    T, D, dt = q.shape[0], c.head_dim, k_cache.dtype
    H, q_stride, ptr_q = _arg_heads("q", q, T, D, dt, dev)
    Ho, out_stride, ptr_o = _arg_heads("out", out, T, D, dt, dev)
    if Ho != H:
        raise Fp4MoeError(f"out: expected {H} heads, got {Ho}")
    B = kv_len.shape[0]
    columns, pt = _arg_table("page_table", page_table, B, dev)
    if ws.nbytes < _lib.ATTENTION_WORKSPACE_BYTES:
        raise Fp4MoeError(f"ws: expected {_lib.ATTENTION_WORKSPACE_BYTES} bytes")
    if ws.get_device() != dev or not ws.is_contiguous():
        _place("ws", ws, dev)
    _check(_lib.load().fp4moe_paged_attention(c, pk, pv, B, T, H, ptr_q, q_stride, pt, columns,
                                              _arg_ints("kv_len", kv_len, B, dev),
                                              _arg_ints("q_offset", q_offset, B + 1, dev), scale, causal, window, ptr_o,
                                              out_stride, _arg("lse", lse, (T, H), _F32, dev), ws.data_ptr(),
                                              _arg_err(err, dev), _s(stream)), "fp4moe_paged_attention")


# --------------------------------------------------------------------------
@dataclass
class Weights:
    w1_fp4: torch.Tensor
    w1_sf: torch.Tensor
    gw1: torch.Tensor
    w2_fp4: torch.Tensor
    w2_sf: torch.Tensor
    gw2: torch.Tensor


@dataclass
class SharedWeights:
    """The shared expert's block-FP8 weights in the layout of include/fp4moe.h."""
    w1: torch.Tensor         # [2 Is][H] E4M3 bytes, kernel row order
    w1_scales: torch.Tensor  # [2 Is / 128][H / 128] fp32
    w2: torch.Tensor         # [H][Is]
    w2_scales: torch.Tensor  # [H / 128][Is / 128]


class MoELayer:
    """Owns the device buffers of one layer configuration and calls the C ABI on them."""

    def __init__(self, cfg: Config, device: str = "cuda"):
        self.cfg = cfg
        self.device = device
        E, H, I = (cfg.ep_count or cfg.num_experts), cfg.hidden, cfg.inter
        b1, s1, b2, s2 = weight_bytes(cfg)
        u8 = dict(dtype=torch.uint8, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.weights = Weights(torch.empty(b1, **u8), torch.empty(s1, **u8), torch.empty(E, **f32),
                               torch.empty(b2, **u8), torch.empty(s2, **u8), torch.empty(E, **f32))
        self.ws = torch.zeros(workspace_bytes(cfg), **u8)
        self.gs1 = torch.ones(1, **f32)
        self.gs2 = torch.ones(1, **f32)
        self.alpha1 = torch.empty(E, **f32)
        self.alpha2 = torch.empty(E, **f32)
        self.router_w = None
        self.router_bias = None
        self.shared = None
        if cfg.shared_inter > 0:
            sb = shared_weight_bytes(cfg)
            self.shared = SharedWeights(torch.empty(sb[0], **u8), torch.empty(sb[1] // 4, **f32),
                                        torch.empty(sb[2], **u8), torch.empty(sb[3] // 4, **f32))

    # ---- load-time prep
    def quantize_weights(self, which: int, e0: int, w: torch.Tensor):
        """Quantise experts [e0, e0 + w.shape[0]) of W1 (which=1, [n, 2I, H]) or W2 (which=2, [n, H, I]).

        NVFP4 layers quantise to E2M1 with E4M3 scales per 16 and a global scale per expert. MXFP4 layers
        (w_format MXFP4) quantise to E2M1 with E8M0 scales per 32; their rows are the rank's kernel-local
        shard, zero past the logical width.
        """
        cfg, W = self.cfg, self.weights
        n = w.shape[0]
        E = cfg.ep_count or cfg.num_experts
        b1, s1, b2, s2 = weight_bytes(cfg)
        if which == 1:
            per_c, per_s = b1 // E, s1 // E
            codes, sf, gs = W.w1_fp4, W.w1_sf, W.gw1
        else:
            per_c, per_s = b2 // E, s2 // E
            codes, sf, gs = W.w2_fp4, W.w2_sf, W.gw2
        fp4moe_quantize_weights(cfg, which, n, w.contiguous(), codes[e0 * per_c:(e0 + n) * per_c],
                                sf[e0 * per_s:(e0 + n) * per_s], gs[e0:e0 + n])

    def shard_mxfp4_weights(self, which: int, e0: int, ck_codes: torch.Tensor, ck_sf: torch.Tensor,
                            full_inter: int, tp: int, tp_rank: int):
        """Cut rank tp_rank's shard of experts [e0, e0 + n) from a quantised full-width MXFP4 checkpoint.

        which=1: ck_codes [n, 2 full_inter, H / 2] bytes (gate rows first), ck_sf [n, 2 full_inter, H / 32];
        which=2: ck_codes [n, H, full_inter / 2], ck_sf [n, H, full_inter / 32] (see fp4moe_shard_mxfp4).
        """
        cfg, W = self.cfg, self.weights
        n = ck_codes.shape[0]
        E = cfg.ep_count or cfg.num_experts
        b1, s1, b2, s2 = weight_bytes(cfg)
        per_c, per_s = (b1 // E, s1 // E) if which == 1 else (b2 // E, s2 // E)
        codes, sf = (W.w1_fp4, W.w1_sf) if which == 1 else (W.w2_fp4, W.w2_sf)
        fp4moe_shard_mxfp4(cfg, which, n, full_inter, tp, tp_rank, ck_codes.contiguous(), ck_sf.contiguous(),
                           codes[e0 * per_c:(e0 + n) * per_c], sf[e0 * per_s:(e0 + n) * per_s])

    def load_mxfp4_weights(self, which: int, e0: int, mx_codes: torch.Tensor, mx_sf: torch.Tensor,
                           err: torch.Tensor):
        """NVFP4 layers: take experts [e0, e0 + n) of W1 (which=1) or W2 (which=2) from MXFP4 weights in the
        atom-tiled MX layout (fp4moe_mxfp4_as_nvfp4); n follows from the buffer sizes of an MXFP4 layer of the
        same hidden and inter. err receives FP4MOE_ERR_SCALE_RANGE for a scale without an exact form."""
        cfg, W = self.cfg, self.weights
        E = cfg.ep_count or cfg.num_experts
        b1, s1, b2, s2 = weight_bytes(cfg)
        rows, K = (2 * cfg.inter, cfg.hidden) if which == 1 else (cfg.hidden, cfg.inter)
        n = mx_codes.numel() // (rows * K // 2)
        per_c, per_s = (b1 // E, s1 // E) if which == 1 else (b2 // E, s2 // E)
        codes, sf, gw = (W.w1_fp4, W.w1_sf, W.gw1) if which == 1 else (W.w2_fp4, W.w2_sf, W.gw2)
        fp4moe_mxfp4_as_nvfp4(cfg, which, n, mx_codes.contiguous(), mx_sf.contiguous(),
                              codes[e0 * per_c:(e0 + n) * per_c], sf[e0 * per_s:(e0 + n) * per_s], gw[e0:e0 + n], err)

    def quantize_shared_weights(self, which: int, w: torch.Tensor):
        """Block-FP8 of the shared expert's W1 (which=1, [2 Is, H], gate rows then up) or W2 (which=2, [H, Is])."""
        se = self.shared
        codes, scales = (se.w1, se.w1_scales) if which == 1 else (se.w2, se.w2_scales)
        fp4moe_shared_quantize_weights(self.cfg, which, w.contiguous(), codes, scales)

    def set_router(self, router_w: torch.Tensor, router_bias: torch.Tensor | None = None):
        self.router_w = router_w.contiguous()
        self.router_bias = None if router_bias is None else router_bias.contiguous()

    def calibrate(self, x_warm: torch.Tensor):
        T = x_warm.shape[0]
        W = self.weights
        fp4moe_calibrate(self.cfg, T, x_warm, self.router_w, self.router_bias, W.w1_fp4, W.w1_sf, W.gw1, self.gs1,
                         self.gs2, self.ws)
        self.update_alpha()

    def set_global_scales(self, gs1: float, gs2: float):
        self.gs1.fill_(gs1)
        self.gs2.fill_(gs2)
        self.update_alpha()

    def batch_gs1(self, x: torch.Tensor, stream=None):
        """Take gs1 (and alpha1) from this batch's own amax, on the device (see fp4moe_batch_gs1)."""
        fp4moe_batch_gs1(self.cfg, x.shape[0], x, self.weights.gw1, self.gs1, self.alpha1, self.ws, stream)

    def update_alpha(self):
        E = self.cfg.ep_count or self.cfg.num_experts
        fp4moe_make_alpha(E, self.gs1, self.weights.gw1, self.alpha1)
        fp4moe_make_alpha(E, self.gs2, self.weights.gw2, self.alpha2)

    # ---- hot path
    def forward(self, x: torch.Tensor, y: torch.Tensor, topk_ids: torch.Tensor | None = None,
                topk_w: torch.Tensor | None = None, stream=None, x_fp8=None):
        """y [T, H] of x [T, H]. x_fp8 = (codes, scales), x's block-FP8 copy as fp4moe_add_rmsnorm writes it, spares a
        layer with a shared expert that expert's quantisation of x."""
        W = self.weights
        if x_fp8 is not None:
            if self.shared is None:
                raise Fp4MoeError("x_fp8: the layer has no shared expert")
            moe_forward_shared_fp8(self.cfg, x.shape[0], x, x_fp8[0], x_fp8[1], self.router_w, self.router_bias,
                                   self.gs1, self.gs2, W.w1_fp4, W.w1_sf, self.alpha1, W.w2_fp4, W.w2_sf, self.alpha2,
                                   self.shared, y, topk_ids, topk_w, self.ws, stream)
            return
        if self.shared is not None:  # routed experts plus the shared expert, one combine
            moe_forward_shared(self.cfg, x.shape[0], x, self.router_w, self.router_bias, self.gs1, self.gs2,
                               W.w1_fp4, W.w1_sf, self.alpha1, W.w2_fp4, W.w2_sf, self.alpha2, self.shared, y,
                               topk_ids, topk_w, self.ws, stream)
            return
        moe_forward(self.cfg, x.shape[0], x, self.router_w, self.router_bias, self.gs1, self.gs2, W.w1_fp4, W.w1_sf,
                    self.alpha1, W.w2_fp4, W.w2_sf, self.alpha2, y, topk_ids, topk_w, self.ws, stream)

    def read_error(self, clear=True) -> int:
        return fp4moe_read_error(self.ws, clear)

    def read_scale_status(self, clear=True):
        """(FP4MOE_SAT_* flags, running amax|h|) of this layer's workspace."""
        return fp4moe_read_scale_status(self.ws, clear)

    def refresh_gs2(self, stream=None):
        """gs2 and alpha2 from the amax|h| of the calls since the last refresh (lagged, on the device)."""
        fp4moe_refresh_gs2(self.cfg, self.ws, self.weights.gw2, self.gs2, self.alpha2, stream)


class MxLinear:
    """A projection y = x W^T with microscaled 4-bit weights and activations (W [N, K], at most max_tokens rows of x).

    fmt W_MXFP4 needs nothing more. fmt W_NVFP4 has a global scale for each operand: the weights' is taken from W here,
    the activations' from a warm-up batch (calibrate) or set by the caller (set_activation_scale); forward refuses to
    run before it has one.

    All calls of one object use its buffers of codes and its error word, so they must be ordered on one stream (or by
    events), like calls of the layer that share a workspace."""

    def __init__(self, weight: torch.Tensor, max_tokens: int, fmt: int = _lib.W_MXFP4):
        self.N, self.K = weight.shape
        self.fmt, self.max_tokens = fmt, max_tokens
        u8 = dict(dtype=torch.uint8, device=weight.device)
        code_bytes, sf_bytes = fp4moe_mx_bytes(fmt, self.N, self.K)
        self.w_codes, self.w_sf = torch.empty(code_bytes, **u8), torch.empty(sf_bytes, **u8)
        self.gw = self.gx = self.alpha = None
        if fmt == _lib.W_NVFP4:
            self.gw = self._global_scale(weight)
            self.gx, self.alpha = torch.empty_like(self.gw), torch.empty_like(self.gw)
        fp4moe_mx_quantize(fmt, weight.contiguous(), self.gw, self.w_codes, self.w_sf)
        self.x_codes = torch.empty(max_tokens * mx_row_bytes(self.K), **u8)
        self.x_sf = torch.empty(mx_sf_bytes(fmt, max_tokens, self.K), **u8)
        self.err = torch.zeros(4, dtype=torch.int32, device=weight.device)
        self.calibrated = fmt != _lib.W_NVFP4

    @staticmethod
    def _global_scale(t):
        amax = t.abs().amax().to(torch.float32).reshape(1)
        return torch.where(amax > 0, 2688.0 / amax, torch.ones_like(amax))

    def calibrate(self, x_warm: torch.Tensor):
        """NVFP4: the activations' global scale RN(2688 / amax) from a warm-up batch (outside any graph)."""
        if self.fmt == _lib.W_NVFP4:
            self.set_activation_scale(self._global_scale(x_warm))

    def set_activation_scale(self, gs):
        """NVFP4: the activations' global scale."""
        if self.gx is None:
            raise Fp4MoeError("set_activation_scale: MXFP4 has no global scale")
        self.gx.copy_(torch.as_tensor(gs, dtype=torch.float32).reshape(1))
        fp4moe_make_alpha(1, self.gx, self.gw, self.alpha)
        self.calibrated = True

    def forward(self, x: torch.Tensor, out: torch.Tensor, stream=None):
        """out [T, N] (bfloat16, float16 or float32) of x [T, K]."""
        # fp4moe_mx_quantize and fp4moe_mx_gemm on this object's own buffers, which need no checks (nor slices for T)
        dev = _current_device()
        (T, K), _, dx, px = _arg_matrix("x", x, dev)
        shape, _, do, po = _arg_matrix("out", out, dev)
        if self.err.get_device() != dev:
            raise Fp4MoeError(f"MxLinear: the weights are on device {self.err.get_device()}, the current one is {dev}")
        if T > self.max_tokens or K != self.K or shape != (T, self.N):
            raise Fp4MoeError(f"expected x [at most {self.max_tokens}, {self.K}] and out [T, {self.N}], got "
                              f"{(T, K)} and {tuple(shape)}")
        if not self.calibrated:
            raise Fp4MoeError("MxLinear: NVFP4 activations have no global scale yet (calibrate, set_activation_scale)")
        lib, s = _lib.load(), _s(stream)
        codes, sf = self.x_codes.data_ptr(), self.x_sf.data_ptr()
        _check(lib.fp4moe_mx_quantize(self.fmt, dx, T, K, px, _p(self.gx), codes, sf, s), "fp4moe_mx_quantize")
        _check(lib.fp4moe_mx_gemm(self.fmt, do, T, self.N, K, codes, sf, self.w_codes.data_ptr(),
                                  self.w_sf.data_ptr(), _p(self.alpha), po, self.err.data_ptr(), s), "fp4moe_mx_gemm")

    def read_error(self, clear=True) -> int:
        return fp4moe_read_error(self.err, clear)


class PagedKvCache:
    """Keys and values of `layers` layers in pages, for at most max_seqs sequences of at most max_len tokens and steps of at
    most max_rows rows. The layers share page tables and lengths; every sequence starts empty.

    A step: plan(new_len) once, then for each layer append(...) and attend(...). All are calls on the device's own lengths,
    so a step of given numbers of sequences and rows can be captured into a CUDA graph; plan advances the lengths at every
    replay. Calls of one object must be ordered on one stream (or by events)."""

    def __init__(self, num_pages: int, page_size: int, kv_heads: int, head_dim: int, max_seqs: int, max_len: int,
                 max_rows: int, layers: int = 1, dtype: torch.dtype = torch.bfloat16, device: str = "cuda"):
        shape = (num_pages, page_size, kv_heads, head_dim)
        self.k, self.v = ([torch.zeros(shape, dtype=dtype, device=device) for _ in range(layers)] for _ in range(2))
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = page_size
        self.page_table = torch.full((max_seqs, (max_len + page_size - 1) // page_size), -1, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)  # page 0 is taken first
        self.free_count = torch.full((1,), num_pages, **i32)
        self.kv_len = torch.zeros(max_seqs, **i32)
        self.q_offset = torch.zeros(max_seqs + 1, **i32)
        self.position, self.slot = torch.zeros(max_rows, **i32), torch.full((max_rows,), -1, **i32)
        self.ws = torch.zeros(_lib.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
        self.err = torch.zeros(4, **i32)

    def plan(self, new_len: torch.Tensor, stream=None, rows: int | None = None):
        """new_len [max_seqs] int32 on the device: tokens that each sequence adds (negative: gives back). rows: the rows of
        the step's q, k and v (max_rows if None): a sequence whose tokens pass them takes nothing, and the error word says so
        (ERR_CAPACITY). Rows beyond those that append and attend are given are not noticed there: their keys would be missing,
        and the last sequence's positions be counted from the rows that are left."""
        position, slot = self.position, self.slot
        if rows is not None:
            if not 0 <= rows <= slot.shape[0]:
                raise Fp4MoeError(f"rows: expected 0 to {slot.shape[0]}, got {rows}")
            position, slot = position[:rows], slot[:rows]
        fp4moe_kv_plan(self.page_size, self.kv_len, new_len, self.page_table, self.free_pages, self.free_count,
                       self.kv_len, self.free_count, self.q_offset, position, slot, self.err, stream)

    def append(self, q, k, v, inv_freq, q_out, first: int = 0, interleaved: bool = False, amplitude: float = 1.0,
               layer: int = 0, stream=None):
        """The step's q [T, heads, D] turned into q_out (may be q), its k and v [T, kv heads, D] into the cache. q and q_out, or
        k and v (of layers that read another one's keys), may be None."""
        if q is None and k is None:
            raise Fp4MoeError("append: q, or k and v, must be given")
        T = (q if k is None else k).shape[0]
        fp4moe_rope_cache(q, k, v, self.position[:T], self.slot[:T], inv_freq, q_out, self.k[layer], self.v[layer],
                          self.err, first, interleaved, amplitude, stream)

    def attend(self, q, scale: float, out, lse=None, window: int = 0, layer: int = 0, stream=None, causal: bool = True):
        """out [T, heads, D] of the step's turned q over the sequences' pages: each row over the keys up to its own (window > 0:
        the last `window` of them), or, not causal, over all keys of its sequence."""
        fp4moe_paged_attention(q, self.k[layer], self.v[layer], self.page_table, self.kv_len, self.q_offset, scale, out,
                               lse, self.ws, self.err, causal, window, stream)

    def read_error(self, clear=True) -> int:
        """The error word. A call that gave up leaves the workspace's counters as they were, and the next call would take
        them for arrivals of its own: with a timeout that is cleared, the workspace is zeroed (on the current stream)."""
        bits = fp4moe_read_error(self.err, clear)
        if clear and bits & _lib.ERR_TIMEOUT:
            self.ws.zero_()
        return bits
