"""The dense operators on the CPU: sizes, and every refusal of the C calls and of the binding. No call here
reaches a CUDA API: each fails validation first."""
import ctypes

import pytest
import torch

from dense_ref import MX, NV, scale_tile_shape
from helpers import ensure_built


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    from block_scaled_fp4_top_gb300 import _lib
    return _lib.load()


P = ctypes.c_void_p(0x10000)     # aligned, never dereferenced
BAD = ctypes.c_void_p(0x10008)


def test_sizes_match_the_layout(lib):
    from block_scaled_fp4_top_gb300 import api
    for fmt in (NV, MX):
        for rows in (0, 1, 127, 128, 129, 1000):
            for K in (1, 31, 32, 33, 64, 255, 256, 1000, 4096):
                R, C = scale_tile_shape(fmt, rows, K)
                assert api.fp4moe_mx_bytes(fmt, rows, K) == (rows * -(-K // 32) * 16, R * C), (fmt, rows, K)
                assert api.mx_row_bytes(K) * rows == rows * -(-K // 32) * 16
                assert api.mx_sf_bytes(fmt, rows, K) == R * C
    assert lib.fp4moe_mx_bytes(MX, 4, 32, None, None) == 0       # outputs optional


def test_mx_refusals(lib):
    from block_scaled_fp4_top_gb300 import _lib
    q = lambda fmt=MX, dt=0, r=4, K=64, x=P, gs=P, c=P, s=P: lib.fp4moe_mx_quantize(fmt, dt, r, K, x, gs, c, s, None)
    d = lambda fmt=MX, dt=0, r=4, K=64, x=P, gs=P, c=P, s=P: lib.fp4moe_mx_dequantize(fmt, dt, r, K, c, s, gs, x, None)
    for f in (q, d):
        assert f(fmt=2) == _lib.UNSUPPORTED
        assert f(dt=3) == _lib.UNSUPPORTED and f(dt=-1) == _lib.UNSUPPORTED
        assert f(r=-1) == _lib.INVALID_ARG
        assert f(K=0) == _lib.INVALID_ARG and f(K=-32) == _lib.INVALID_ARG
        for name in ("x", "c", "s"):
            assert f(**{name: None}) == _lib.INVALID_ARG, name
            assert f(**{name: BAD}) == _lib.MISALIGNED, name
        assert f(fmt=NV, gs=None) == _lib.INVALID_ARG            # NVFP4 needs its global scale
        assert f(fmt=NV, gs=BAD) == _lib.MISALIGNED
        assert f(r=2**31 - 1, K=2**31 - 1) == _lib.UNSUPPORTED   # scale tiles past 32-bit indices
        assert f(r=0) == _lib.OK                                 # nothing to do, nothing launched


def test_mx_gemm_refusals(lib):
    from block_scaled_fp4_top_gb300 import _lib

    def g(fmt=MX, dt=0, M=4, N=4, K=64, a=P, asf=P, b=P, bsf=P, alpha=None, out=P, err=P):
        return lib.fp4moe_mx_gemm(fmt, dt, M, N, K, a, asf, b, bsf, alpha, out, err, None)

    assert g(fmt=5) == _lib.UNSUPPORTED and g(dt=7) == _lib.UNSUPPORTED
    assert g(M=-1) == _lib.INVALID_ARG and g(N=0) == _lib.INVALID_ARG and g(N=-4) == _lib.INVALID_ARG
    assert g(K=0) == _lib.INVALID_ARG
    assert g(M=2**31 - 1, N=2**31 - 1, K=1) == _lib.UNSUPPORTED
    for name in ("a", "asf", "b", "bsf", "out", "err"):
        assert g(**{name: None}) == _lib.INVALID_ARG, name
        assert g(**{name: BAD}) == _lib.MISALIGNED, name
    assert g(alpha=BAD) == _lib.MISALIGNED
    assert g(M=0) == _lib.OK


def test_norm_refusals(lib):
    from block_scaled_fp4_top_gb300 import _lib

    def n(dt=0, T=4, H=256, x=P, r=P, gamma=P, eps=1e-6, h=P, y=P, c=P, s=P, stride=4):
        return lib.fp4moe_add_rmsnorm(dt, T, H, x, r, gamma, eps, h, y, c, s, stride, None)

    assert n(dt=3) == _lib.UNSUPPORTED
    assert n(T=-1) == _lib.INVALID_ARG and n(H=0) == _lib.INVALID_ARG
    for eps in (-1e-6, float("nan"), float("inf")):
        assert n(eps=eps) == _lib.INVALID_ARG
    assert n(r=None) == _lib.INVALID_ARG and n(h=None) == _lib.INVALID_ARG      # both or neither
    assert n(c=None) == _lib.INVALID_ARG and n(s=None) == _lib.INVALID_ARG
    assert n(y=None, c=None, s=None) == _lib.INVALID_ARG                        # nothing to compute
    assert n(stride=3) == _lib.INVALID_ARG
    assert n(x=None) == _lib.INVALID_ARG
    for name in ("x", "r", "gamma", "h", "y", "c", "s"):
        assert n(**{name: BAD}) == _lib.MISALIGNED, name
    assert n(T=0, stride=0) == _lib.OK


def test_norm_refuses_one_buffer_for_two_results(lib):
    from block_scaled_fp4_top_gb300 import _lib
    other = ctypes.c_void_p(0x20000)
    assert lib.fp4moe_add_rmsnorm(0, 4, 256, P, P, None, 1e-6, other, other, None, None, 0, None) == _lib.INVALID_ARG


def test_widths_whose_column_index_would_pass_32_bits(lib):
    from block_scaled_fp4_top_gb300 import _lib
    top = 2**31 - 1 - 8192
    for K, want in ((top, _lib.OK), (top + 1, _lib.UNSUPPORTED), (2**31 - 1, _lib.UNSUPPORTED)):
        assert lib.fp4moe_mx_bytes(MX, 1, K, None, None) == want
        assert lib.fp4moe_mx_quantize(MX, 0, 0, K, None, None, None, None, None) == want
        assert lib.fp4moe_mx_dequantize(MX, 0, 0, K, None, None, None, None, None) == want
        assert lib.fp4moe_add_rmsnorm(0, 0, K, None, None, None, 1e-6, None, None, None, None, 0, None) == want


def test_shared_fp8_refusals(lib):
    from block_scaled_fp4_top_gb300 import _lib, api
    cfg = api.config(4096, 2048, 256, 6, 64, 10.0, shared_inter=2048)
    se = _lib.SharedWeights(0x10000, 0x10000, 0x10000, 0x10000)
    ref = ctypes.byref

    def f(c=cfg, T=8, codes=P, scales=P, stride=8, w=se, o=P, ws=P):
        return lib.moe_shared_expert_fp8(ref(c), T, codes, scales, stride, ref(w) if w else None, o, ws, None)

    assert f(stride=7) == _lib.INVALID_ARG
    assert f(T=65, stride=65) == _lib.CAPACITY
    assert f(w=None) == _lib.INVALID_ARG
    assert f(c=api.config(4096, 2048, 256, 6, 64, 10.0)) == _lib.INVALID_ARG    # no shared expert
    for name in ("codes", "scales", "o", "ws"):
        assert f(**{name: None}) == _lib.INVALID_ARG, name
        assert f(**{name: BAD}) == _lib.MISALIGNED, name
    tail = [P] * 10 + [ref(se)] + [P] * 5
    assert lib.moe_forward_shared_fp8(ref(cfg), 8, P, P, P, 7, *tail) == _lib.INVALID_ARG
    assert lib.moe_forward_shared_fp8(ref(cfg), 8, P, None, P, 8, *tail) == _lib.INVALID_ARG
    assert lib.moe_forward_shared_fp8(ref(cfg), 8, P, P, BAD, 8, *tail) == _lib.MISALIGNED


def test_binding_refuses_wrong_shapes_and_types():
    """The C calls see pointers only, so the binding holds every tensor to its shape and type."""
    from block_scaled_fp4_top_gb300 import api
    E = api.Fp4MoeError
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x = torch.zeros(4, 100, dtype=bf)
    z = lambda *s, d=bf: torch.zeros(*s, dtype=d)
    for bad in [dict(residual=z(4, 99), residual_out=z(4, 100)), dict(residual=z(4, 100, d=f32)), dict(gamma=z(99)),
                dict(gamma=z(100, d=f32)), dict(y=z(3, 100)), dict(y_codes=z(4, 99, d=u8), y_scales=z(1, 4, d=f32)),
                dict(y_codes=z(4, 100, d=u8), y_scales=z(1, 3, d=f32)),
                dict(y_codes=z(4, 100, d=u8), y_scales=z(2, 4, d=f32)),
                dict(y_codes=z(4, 100, d=bf), y_scales=z(1, 4, d=f32)),
                dict(y_codes=z(4, 100, d=u8), y_scales=z(1, 4))]:
        a = dict(residual=None, gamma=None, residual_out=None, y=z(4, 100), y_codes=None, y_scales=None) | bad
        with pytest.raises(E):
            api.fp4moe_add_rmsnorm(x, a["residual"], a["gamma"], 1e-6, a["residual_out"], a["y"], a["y_codes"],
                                   a["y_scales"])
    with pytest.raises(E):
        api.fp4moe_add_rmsnorm(x.double(), None, None, 1e-6, None, x.double())
    with pytest.raises(E):
        api.fp4moe_add_rmsnorm(x.view(-1), None, None, 1e-6, None, x.view(-1))
    codes, sf = z(4 * 64, d=u8), z(512, d=u8)                    # [4, 100] in MXFP4: 4 rows of 64 bytes, one tile
    with pytest.raises(E):
        api.fp4moe_mx_quantize(MX, x, None, codes[1:], sf)
    with pytest.raises(E):
        api.fp4moe_mx_quantize(MX, x, None, codes, sf[1:])
    with pytest.raises(E):
        api.fp4moe_mx_quantize(NV, x, torch.ones(1, dtype=bf), codes, z(1024, d=u8))
    with pytest.raises(E):
        api.fp4moe_mx_quantize(MX, x.int(), None, codes, sf)
    with pytest.raises(E):
        api.fp4moe_mx_dequantize(MX, codes, sf, None, z(4, 200))
    err = torch.zeros(4, dtype=torch.int32)
    for bad in [dict(out=z(5, 4)), dict(K=200), dict(a=codes.to(torch.int8)), dict(err=z(1)), dict(b=codes[:64])]:
        a = dict(out=z(4, 4), K=100, a=codes, b=codes, err=err) | bad
        with pytest.raises(E):
            api.fp4moe_mx_gemm(MX, a["K"], a["a"], sf, a["b"], sf, None, a["out"], a["err"])
    # right shapes, but not on the device: refused before any call
    with pytest.raises(E):
        api.fp4moe_mx_gemm(MX, 100, codes, sf, codes, sf, None, z(4, 4), err)
    with pytest.raises(E):
        api.fp4moe_mx_quantize(MX, x, None, codes, sf)


def test_no_load_writes_into_several_ctas():
    """The library also runs as replicas on several GPUs, where a bulk or tensor load that writes into more than one CTA
    of a cluster must not be part of it. (A commit that signals two CTAs' barriers is no load.)"""
    import os
    import re
    from helpers import ROOT
    load = re.compile(r"\bcp\.(?:reduce\.)?async\.bulk[^;\[]*" + "multi" + "cast")
    csrc = os.path.join(ROOT, "block_scaled_fp4_top_gb300", "csrc")
    names = [n for n in sorted(os.listdir(csrc)) if n.endswith((".cu", ".cuh", ".h"))]
    assert len(names) > 10
    for name in names:
        with open(os.path.join(csrc, name)) as f:
            text = re.sub(r'"\s*\n\s*"', "", f.read())  # adjacent string literals are one instruction
        assert not load.search(text), name


def test_mx_gemm_plans_of_the_test_sizes(lib):
    """The sizes that stand for each kernel do take it: a change of the choice shows here."""
    from block_scaled_fp4_top_gb300 import api
    from mx_plans import CASES, SMS
    for plan, size in CASES:
        assert api.fp4moe_mx_gemm_plan(*size, SMS) == plan, size


def test_mx_gemm_plans_hold_over_the_range(lib):
    """Every size has a plan of a kernel that there is; K is split only where each slice has a stage of 256 elements."""
    import random
    from block_scaled_fp4_top_gb300 import api
    from mx_plans import PLANS
    rng = random.Random(1)
    size = lambda: int(2 ** rng.uniform(0, 15))
    for _ in range(5000):
        M, N, K, sms = size(), size(), size(), rng.choice((1, 8, 84, 148, 152))
        plan = api.fp4moe_mx_gemm_plan(M, N, K, sms)
        assert plan in PLANS and plan[2] <= -(-K // 256), (M, N, K, sms)
    top = 2**31 - 1 - 8192
    for s in ((1, 1, top), (1, 100, top), (129, 1, top), (top, 1, 1), (1, top, 1)):
        assert api.fp4moe_mx_gemm_plan(*s, 152) in PLANS, s


def test_mx_gemm_plan_refusals(lib):
    from block_scaled_fp4_top_gb300 import _lib
    p = lib.fp4moe_mx_gemm_plan
    for bad in ((0, 1, 1, 152), (1, 0, 1, 152), (1, 1, 0, 152), (1, 1, 1, 0), (-1, 1, 1, 152)):
        assert p(*bad, None, None, None) == _lib.INVALID_ARG
    assert p(1, 1, 2**31 - 1, 152, None, None, None) == _lib.UNSUPPORTED
    assert p(4, 4, 64, 152, None, None, None) == _lib.OK         # outputs optional
