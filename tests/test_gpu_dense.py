"""GPU: the dense operators against their 64-bit definitions.

Tolerances are sums of the roundings that the definitions allow:
* a stored result is off by half a step of its type (HALF_STEP, TINY);
* the norm's statistics: a sum of H squares in fp32 (H / 256 sequential additions, then a tree), a division, a
  square root and a reciprocal, two products: (H / 256 + 16) 2^-24 relative;
* the product: fp32 additions of exact products, at worst one rounding of 2^-22 of the running magnitude per
  64-element instruction (truncation included), against the sum of the magnitudes |a| |b|;
* quantisation is exact arithmetic or fixed fp32 steps: codes and scale bytes are compared bit for bit.
"""
import numpy as np
import pytest

import mx_plans
from dense_ref import (BLOCK, HALF_STEP, MX, NV, TINY, Guarded, e4m3_half_step, pack, quantize, rms_norm,
                       scale_tile_shape, values)
from helpers import ensure_built
from oracle import codecs, nvfp4

pytestmark = pytest.mark.gpu
DTYPES = ["bfloat16", "float16", "float32"]
OVERFLOW = {"bfloat16": 3.39e38, "float16": 65520.0, "float32": 3.4e38}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def rnd(shape, dtype, seed, spread=1.0):
    import torch
    rng = np.random.default_rng(seed)
    v = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[-1]))
    return torch.from_numpy(v.astype(np.float32)).to(getattr(torch, dtype)).cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------------- norm
def check_norm(T, H, dtype, residual=True, gamma=True, y=True, fp8=True, eps=1e-6, seed=0, x=None, pad_stride=0,
               alias=None):
    import torch
    from block_scaled_fp4_top_gb300 import api
    dt = getattr(torch, dtype)
    x = rnd((T, H), dtype, seed) if x is None else x
    r = rnd((T, H), dtype, seed + 1) if residual else None
    g = rnd((H,), dtype, seed + 2, 0.0) if gamma else None
    G = (H + 127) // 128
    xb = Guarded((T, H), dt, x)
    rb = Guarded((T, H), dt, r) if residual else None
    hb = {"h=x": xb, "h=r": rb, None: Guarded((T, H), dt) if residual else None, "y=x": Guarded((T, H), dt)
          if residual else None, "h=r,y=x": rb}[alias]
    yb = xb if alias in ("y=x", "h=r,y=x") else Guarded((T, H), dt)
    cb, sb = Guarded((T, H), torch.uint8), Guarded((G, T + pad_stride), torch.float32)
    api.fp4moe_add_rmsnorm(xb.t, rb.t if residual else None, g, eps, hb.t if residual else None, yb.t if y else None,
                           cb.t if fp8 else None, sb.t if fp8 else None)
    torch.cuda.synchronize()
    for b in (xb, rb, hb, yb, cb, sb):
        if b is not None:
            b.check()
    h = x
    if residual:
        h = (x.float() + r.float()).to(dt)
        assert torch.equal(hb.t, h), "residual stream"
    n = rms_norm(f64(h), f64(g) if gamma else None, eps)
    rel = (H / 256 + 16) * 2.0 ** -24
    if y:
        err = np.abs(f64(yb.t) - n)
        assert (err <= np.abs(n) * (rel + HALF_STEP[dtype] * (1 + rel)) + TINY[dtype]).all(), err.max()
    if fp8:
        s = sb.t[:, :T].cpu().numpy().astype(np.float64)
        pad = np.zeros((T, G * 128))
        pad[:, :H] = n
        amax = np.abs(pad.reshape(T, G, 128)).max(2).T
        assert (np.abs(s - amax / 448) <= amax / 448 * (rel + 2.0 ** -23) + 2.0 ** -149).all()
        v = codecs.E4M3_TABLE[cb.t.cpu().numpy()]
        sc = np.repeat(s.T, 128, axis=1)[:, :H]
        q = np.where(sc == 0, 0.0, n / np.where(sc == 0, 1.0, sc))
        assert (np.abs(v - q) <= e4m3_half_step(q) * (1 + 2.0 ** -10) + np.abs(q) * 2 * rel).all()
        if pad_stride:
            raw = sb.t[:, T:].contiguous().view(torch.uint8)
            assert (raw == 0xA5).all(), "scales written past the tokens"
    else:
        assert (cb.t == 0xA5).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 3, 8, 100, 127, 128, 129, 256, 1000, 2048, 4090, 4096, 4097, 8192, 20000, 40960])
def test_norm_widths(dtype, H):
    check_norm(3, H, dtype, seed=H)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", [(1, 4096), (2, 4096), (64, 4096), (65, 4090), (700, 4096), (700, 4090), (701, 129),
                                 (703, 1001), (900, 8191), (153, 20001)])
def test_norm_rows(dtype, T, H):
    check_norm(T, H, dtype, seed=T)


@pytest.mark.parametrize("H", [4090, 1001])
@pytest.mark.parametrize("alias", ["h=x", "h=r,y=x"])
def test_norm_many_rows_in_place(H, alias):
    check_norm(400, H, "bfloat16", alias=alias)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [384, 1001])
@pytest.mark.parametrize("opts", [dict(residual=False), dict(gamma=False), dict(fp8=False), dict(y=False),
                                  dict(residual=False, gamma=False, y=False), dict(eps=0.0), dict(pad_stride=5)])
def test_norm_options(dtype, H, opts):
    check_norm(9, H, dtype, seed=H, **opts)


@pytest.mark.parametrize("H", [4096, 1001, 40960])
@pytest.mark.parametrize("alias", ["h=x", "h=r", "y=x", "h=r,y=x"])
def test_norm_in_place(H, alias):
    check_norm(5, H, "bfloat16", alias=alias)


@pytest.mark.parametrize("H", [512, 333])
def test_norm_zero_and_tiny_rows(H):
    import torch
    x = torch.zeros(4, H, dtype=torch.float32, device="cuda")
    x[1, 0] = 1e-30
    x[2] = 1e-12
    x[3, -1] = 1e4
    check_norm(4, H, "float32", residual=False, x=x)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("H", [512, 333])
@pytest.mark.parametrize("opts", [dict(), dict(gamma=False), dict(eps=0.0), dict(residual=False, eps=0.0)])
def test_norm_rows_of_many_magnitudes(dtype, H, opts):
    """Both ways to the FP8 codes, and the border between them, in rows side by side and in groups of one row."""
    import torch
    e = torch.tensor([-55, -51, -50, -49, -30, 0, 30, 49, 50, 51, 55], dtype=torch.float32, device="cuda")
    x = rnd((len(e), H), dtype, 7, 0.0) * torch.exp2(e)[:, None].to(getattr(torch, dtype))
    x[5, 128:256] = 0
    x[6, :128] *= 2.0 ** -100
    check_norm(len(e), H, dtype, seed=8, x=x, **opts)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("H", [512, 333])
def test_norm_nonfinite_rows_stay_in_their_row(dtype, H):
    import torch
    from block_scaled_fp4_top_gb300 import api
    x = rnd((6, H), dtype, 3)
    x[1, 5], x[3, H - 1], x[4, 0] = float("nan"), float("inf"), float("-inf")
    y = torch.empty_like(x)
    codes = torch.empty(6, H, dtype=torch.uint8, device="cuda")
    scales = torch.empty((H + 127) // 128, 6, device="cuda")
    api.fp4moe_add_rmsnorm(x, None, None, 1e-6, None, y, codes, scales)
    torch.cuda.synchronize()
    assert y[1].isnan().all() and (codes[1] & 127 == 127).all()
    # an infinity makes the statistics infinite: 0 elsewhere, inf * 0 = NaN in its own place
    for row, col in ((3, H - 1), (4, 0)):
        assert y[row, col].isnan() and int(codes[row, col]) & 127 == 127
        rest = torch.arange(H, device="cuda") != col
        assert (y[row][rest] == 0).all()
    clean = [0, 2, 5]
    assert y[clean].isfinite().all() and scales[:, clean].isfinite().all() and (codes[clean] & 127 != 127).all()


@pytest.mark.parametrize("gamma", [False, True])
@pytest.mark.parametrize("T,H", [(16, 4096), (200, 512), (9, 1001), (200, 1002)])
def test_norm_codes_of_bf16_are_those_of_exact_arithmetic(T, H, gamma):
    """n / s is 448 p / max|p| with p = h * gamma: in fp64 that side and a midpoint of the E4M3 grid times max|p| are
    exact products, so every code, ties to even included, follows from comparisons."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    h = rnd((T, H), "bfloat16", H, 0.5)
    g = rnd((H,), "bfloat16", H + 1, 0.0) if gamma else None
    y, codes = torch.empty_like(h), torch.empty(T, H, dtype=torch.uint8, device="cuda")
    G = (H + 127) // 128
    api.fp4moe_add_rmsnorm(h, None, g, 1e-6, None, y, codes, torch.empty(G, T, device="cuda"))
    p = np.zeros((T, G * 128))
    p[:, :H] = f64(h) * (f64(g) if gamma else 1.0)
    top = np.repeat(np.abs(p).reshape(T, G, 128).max(2), 128, axis=1)
    grid = codecs.E4M3_TABLE[:127].astype(np.float64)
    want = np.zeros(p.shape, dtype=np.int64)
    for i, mid in enumerate((grid[1:] + grid[:-1]) / 2):
        side, bar = 448.0 * np.abs(p), mid * top
        want += (side > bar) | ((side == bar) & (i % 2 == 1))
    want |= (p < 0) << 7
    torch.cuda.synchronize()
    got = codes.cpu().numpy().astype(np.int64)
    differ = (got != want[:, :H]) & ~((got & 127 == 0) & (want[:, :H] & 127 == 0))     # the sign of a zero is free
    assert not differ.any(), f"{differ.sum()} codes of {differ.size}"


def test_norm_empty():
    import torch
    from block_scaled_fp4_top_gb300 import api
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    api.fp4moe_add_rmsnorm(x, x, None, 1e-6, x, torch.empty_like(x))


# ------------------------------------------------------------------------- quantisation
def gpu_quantize(fmt, x, g):
    import torch
    from block_scaled_fp4_top_gb300 import api
    rows, K = x.shape
    R, C = scale_tile_shape(fmt, rows, K)
    cb = Guarded((rows, api.mx_row_bytes(K)), torch.uint8)
    sb = Guarded((R * C,), torch.uint8)
    gt = torch.tensor([g], dtype=torch.float32, device="cuda") if fmt == NV else None
    api.fp4moe_mx_quantize(fmt, x, gt, cb.t, sb.t)
    torch.cuda.synchronize()
    cb.check()
    sb.check()
    return cb.t, sb.t, gt


def check_quantize(fmt, x, g=1.0):
    import torch
    from block_scaled_fp4_top_gb300 import api
    rows, K = x.shape
    codes, sf, gt = gpu_quantize(fmt, x, g)
    q, s = quantize(fmt, x.float().cpu().numpy(), g)
    pc, ps = pack(fmt, q, s, K)
    assert (sf.cpu().numpy() == ps).all(), f"{(sf.cpu().numpy() != ps).sum()} scale bytes differ"
    assert (codes.cpu().numpy() == pc).all(), f"{(codes.cpu().numpy() != pc).sum()} code bytes differ"
    v = values(fmt, q, s, K)
    for dtype in DTYPES:
        ob = Guarded((rows, K), getattr(torch, dtype))
        api.fp4moe_mx_dequantize(fmt, codes, sf, gt, ob.t)
        torch.cuda.synchronize()
        ob.check()
        w = v.astype(np.float32)                                  # exact: at most 6 significant bits
        assert (w == v).all()
        if fmt == NV:
            w = w / np.float32(g)                                 # RN in fp32 by definition
        want = torch.from_numpy(w).to(getattr(torch, dtype))
        assert torch.equal(ob.t.cpu(), want), dtype


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 16), (2, 31), (3, 32), (5, 33), (1, 64), (7, 100), (127, 128), (128, 96),
                                    (129, 160), (130, 4096), (64, 1000), (300, 520), (1, 8191), (700, 1023),
                                    (40, 700), (400, 5000)])
def test_quantize_bits(fmt, dtype, rows, K):
    check_quantize(fmt, rnd((rows, K), dtype, rows * 10007 + K, 1.5), 37.5)


@pytest.mark.parametrize("fmt", [NV, MX])
def test_quantize_ties_and_extremes(fmt):
    """Every midpoint of the element grid at several block scales, zeros of both signs, subnormals, the largest
    finite values, blocks of one nonzero element."""
    import torch
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1, 1.5, 2, 3, 4, 0, -0.0])
    rows = []
    for scale in (2.0 ** -126, 2.0 ** -10, 1.0, 2.0 ** 20, 2.0 ** 120):
        for sign in (1, -1):
            rows.append(np.tile(sign * mids * scale, 4))
            rows.append(np.tile(sign * np.nextafter(np.float32(mids), np.float32(9)) * scale, 4))
            rows.append(np.tile(sign * np.nextafter(np.float32(mids), np.float32(-9)) * scale, 4))
    rows.append(np.zeros(64))
    rows.append(np.full(64, -0.0))
    rows.append(np.full(64, 2.0 ** -149))
    rows.append(np.full(64, 3.4028234663852886e38))
    one = np.zeros(64)
    one[[7, 40]] = (2.0 ** -140, -1e30)
    rows.append(one)
    x = torch.from_numpy(np.array(rows).astype(np.float32)).cuda()
    for g in (1.0, 1e-3, 2688.0, 1e20):
        check_quantize(fmt, x, g)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_nonfinite_blocks(fmt, dtype):
    import torch
    from block_scaled_fp4_top_gb300 import api
    x = rnd((4, 100), dtype, 9)
    clean = x.clone()
    bad = [(0, 0, float("nan")), (1, 33, float("inf")), (2, 63, float("-inf")), (3, 99, float("nan"))]
    for r, c, v in bad:
        x[r, c] = v
    codes, sf, gt = gpu_quantize(fmt, x, 3.0)
    B = BLOCK[fmt]
    R, C = scale_tile_shape(fmt, 4, 100)
    s = nvfp4.unswizzle(sf.cpu().numpy(), R, C)
    out, ref = torch.empty_like(x), torch.empty_like(x)
    api.fp4moe_mx_dequantize(fmt, codes, sf, gt, out)
    cc, cs, _ = gpu_quantize(fmt, clean, 3.0)
    api.fp4moe_mx_dequantize(fmt, cc, cs, gt, ref)
    torch.cuda.synchronize()
    hit = torch.zeros(4, 100, dtype=torch.bool, device="cuda")
    for r, c, _ in bad:
        assert s[r, c // B] == (0xFF if fmt == MX else 0x7F)
        hit[r, c // B * B:(c // B + 1) * B] = True
    assert out[hit].isnan().all()
    assert torch.equal(out[~hit], ref[~hit])


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [64, 36])
def test_dequantize_every_code_under_every_scale(fmt, dtype, K):
    """One scale byte a row, zero scales under nonzero codes among them; K = 36: rows that no vector divides."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    scales = np.arange(0, 0x7F if fmt == NV else 0xFF, dtype=np.uint8)
    rows = len(scales)
    q = np.tile(np.arange(16, dtype=np.uint8), (rows, 4))
    q[:, K:] = 0
    s = np.repeat(scales[:, None], -(-K // BLOCK[fmt]), axis=1)
    pc, ps = (torch.from_numpy(t).cuda() for t in pack(fmt, q, s, K))
    v = values(fmt, q, s, K).astype(np.float32)
    for g in (1.0, 1e-3, 3e20, 2.0 ** -120) if fmt == NV else (1.0,):
        gt = torch.tensor([g], dtype=torch.float32, device="cuda")
        ob = Guarded((rows, K), getattr(torch, dtype))
        api.fp4moe_mx_dequantize(fmt, pc, ps, gt, ob.t)
        torch.cuda.synchronize()
        ob.check()
        with np.errstate(over="ignore"):
            w = v / np.float32(g) if fmt == NV else v
        assert torch.equal(ob.t.cpu(), torch.from_numpy(w).to(getattr(torch, dtype))), g


# ------------------------------------------------------------------------- product
def gemm_operands(fmt, M, N, K, seed):
    """Codes and scales with every code value and a range of scales, as the library stores them; their values."""
    import torch
    rng = np.random.default_rng(seed)
    out = []
    for rows in (M, N):
        q = rng.integers(0, 16, (rows, -(-K // 32) * 32), dtype=np.uint8)
        q[:, K:] = 0
        n = -(-K // BLOCK[fmt])
        s = rng.integers(117, 133, (rows, n)) if fmt == MX else rng.integers(0, 0x7F, (rows, n))
        s = s.astype(np.uint8)
        pc, ps = pack(fmt, q, s, K)
        out += [torch.from_numpy(pc).cuda(), torch.from_numpy(ps).cuda(), values(fmt, q, s, K)]
    return out


def hold_product(got, ref, mag, K, dtype):
    bar = mag * (K / 64 + 8) * 2.0 ** -22 + np.abs(ref) * (HALF_STEP[dtype] + 2.0 ** -23) + TINY[dtype]
    e = np.abs(got - ref)
    # past the type's range a result rounds to infinity (fp16: from 65520 on)
    over = (e > bar) & ~(np.isinf(got) & (np.sign(got) == np.sign(ref)) & (np.abs(ref) + bar >= OVERFLOW[dtype]))
    assert not over.any(), f"{over.sum()} of {over.size} over, first {np.argwhere(over)[:4].tolist()}, worst {(e / bar).max()}"


def check_gemm(fmt, M, N, K, dtype, seed=0, alpha=None, operands=None):
    import torch
    from block_scaled_fp4_top_gb300 import api
    a, asf, av, b, bsf, bv = operands or gemm_operands(fmt, M, N, K, seed)
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    ob = Guarded((M, N), getattr(torch, dtype))
    al = None if alpha is None else torch.tensor([alpha], dtype=torch.float32, device="cuda")
    api.fp4moe_mx_gemm(fmt, K, a, asf, b, bsf, al, ob.t, err)
    torch.cuda.synchronize()
    assert err.cpu().numpy()[0] == 0
    ob.check()
    sc = 1.0 if alpha is None else float(np.float32(alpha))
    ref = av @ bv.T * sc
    mag = np.abs(av) @ np.abs(bv).T * abs(sc)
    hold_product(f64(ob.t), ref, mag, K, dtype)
    return ob.t


SHAPES = [(1, 1, 1), (1, 128, 32), (3, 5, 33), (127, 129, 64), (128, 128, 128), (129, 257, 192), (128, 128, 256),
          (130, 300, 1000), (257, 513, 320), (64, 1024, 2048), (16, 70, 4096), (33, 1, 700), (1, 4096, 4096)]


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_shapes(fmt, M, N, K):
    check_gemm(fmt, M, N, K, "float32", seed=M + N + K)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(100, 264, 288), (100, 265, 288), (1300, 4100, 160), (2000, 3600, 520)])
def test_gemm_types_and_many_tiles(fmt, dtype, M, N, K):
    check_gemm(fmt, M, N, K, dtype, seed=K, alpha=2.0 ** -9 if dtype == "float16" else 0.37)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [
    (1, 1000, 4096), (16, 1024, 1280), (17, 333, 1100), (33, 257, 2047), (64, 64, 8192),     # K over four CTAs
    (1, 4096, 4095), (20, 4090, 4096), (64, 4000, 3999),                                     # over two
    (65, 65, 4096), (129, 2000, 600),                                                        # 128 x 64 tiles
    (400, 8000, 300), (513, 4104, 1999),                                                     # 128 x 128
    (1025, 3001, 2100), (2000, 1528, 2048), (1500, 3000, 2000),                              # two pairs in a cluster
])
def test_gemm_every_kernel(fmt, dtype, M, N, K):
    check_gemm(fmt, M, N, K, dtype, seed=M, alpha=2.0 ** -9 if dtype == "float16" else -1.75)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(8192, 4096, 2048), (8100, 4051, 2080)])                  # one pair a cluster
def test_gemm_pairs_many_rounds(fmt, dtype, M, N, K):
    """Large products against fp64 matmul on the device, at sampled rows and every column."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    rng = np.random.default_rng(K)
    codes, sfs, vals = [], [], []
    for rows in (M, N):
        q = rng.integers(0, 16, (rows, -(-K // 32) * 32), dtype=np.uint8)
        q[:, K:] = 0
        s = rng.integers(117, 133, (rows, -(-K // 32))) if fmt == MX else rng.integers(0, 0x7F, (rows, -(-K // 16)))
        pc, ps = pack(fmt, q, s.astype(np.uint8), K)
        codes.append(torch.from_numpy(pc).cuda())
        sfs.append(torch.from_numpy(ps).cuda())
        vals.append((q, s.astype(np.uint8)))
    out = Guarded((M, N), getattr(torch, dtype))
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    al = torch.tensor([2.0 ** -9], device="cuda")
    api.fp4moe_mx_gemm(fmt, K, codes[0], sfs[0], codes[1], sfs[1], al, out.t, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    out.check()
    pick = np.unique(np.concatenate([np.arange(0, M, 97), [127, 128, 255, 256, 511, 512, M - 1]]))
    av = torch.from_numpy(values(fmt, vals[0][0][pick], vals[0][1][pick], K)).cuda()
    bv = torch.from_numpy(values(fmt, *vals[1], K)).cuda()
    ref = (av @ bv.T).cpu().numpy() * 2.0 ** -9
    mag = (av.abs() @ bv.abs().T).cpu().numpy() * 2.0 ** -9
    hold_product(f64(out.t[torch.from_numpy(pick).cuda()]), ref, mag, K, dtype)
    # every other row was computed too: the same product again, bit for bit, and no canary value left
    again = torch.empty_like(out.t)
    api.fp4moe_mx_gemm(fmt, K, codes[0], sfs[0], codes[1], sfs[1], al, again, err)
    torch.cuda.synchronize()
    assert torch.equal(out.t, again)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(128, 1024, 14336), (65, 100, 9000), (200, 513, 8200), (513, 130, 8192)])
def test_gemm_k_split_of_more_than_64_rows(fmt, dtype, M, N, K):
    check_gemm(fmt, M, N, K, dtype, seed=M)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("M,N,K", [(5, 300, 512), (700, 4096, 1024), (8, 1024, 4096), (64, 4096, 4096)])
def test_gemm_is_deterministic(fmt, M, N, K):
    import torch
    ops = gemm_operands(fmt, M, N, K, 4)
    first = check_gemm(fmt, M, N, K, "float32", operands=ops).clone()
    for _ in range(5):
        assert torch.equal(first, check_gemm(fmt, M, N, K, "float32", operands=ops))


@pytest.mark.parametrize("fmt", [NV, MX])
def test_gemm_zero_and_nan_blocks(fmt):
    """A zero matrix gives zeros; a NaN block makes its own row (of A) or column (of B) NaN and nothing else."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    M, N, K = 130, 200, 288
    x, w = rnd((M, K), "bfloat16", 1), rnd((N, K), "bfloat16", 2)
    x[3], w[5] = 0, 0
    x[17, 40], x[129, K - 1], w[199, 0] = float("nan"), float("inf"), float("-inf")
    a, asf, _ = gpu_quantize(fmt, x, 8.0)
    b, bsf, _ = gpu_quantize(fmt, w, 8.0)
    out = torch.empty(M, N, dtype=torch.float32, device="cuda")
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    api.fp4moe_mx_gemm(fmt, K, a, asf, b, bsf, None, out, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[[17, 129]] = True
    bad[:, 199] = True
    assert torch.equal(out.isnan(), bad)
    assert (out[3][~bad[3]] == 0).all() and (out[:, 5][~bad[:, 5]] == 0).all()


def test_gemm_skips_its_work_under_a_raised_error_word():
    import torch
    from block_scaled_fp4_top_gb300 import _lib, api
    a, asf, _, b, bsf, _ = gemm_operands(MX, 8, 64, 64, 1)
    out = torch.full((8, 64), 7.0, device="cuda")
    err = torch.tensor([_lib.ERR_TIMEOUT, 0, 0, 0], dtype=torch.int32, device="cuda")
    api.fp4moe_mx_gemm(MX, 64, a, asf, b, bsf, None, out, err)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and api.fp4moe_read_error(err) == _lib.ERR_TIMEOUT
    api.fp4moe_mx_gemm(MX, 64, a, asf, b, bsf, None, out, err)      # cleared by the read
    torch.cuda.synchronize()
    assert (out != 7.0).any()


# ------------------------------------------------------------------------- streams and graphs
@pytest.mark.parametrize("fmt", [NV, MX])
def test_chain_on_a_side_stream_and_in_a_graph(fmt):
    """norm -> quantise -> product -> norm, eager on another stream and replayed from a graph with new inputs: the
    same bits as eager on the default stream."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    T, H, N = 40, 512, 320
    w = rnd((N, H), "bfloat16", 5)
    gw = torch.tensor([50.0], device="cuda")
    ga = torch.tensor([300.0], device="cuda")
    alpha = 1.0 / (gw * ga)
    bc, bs = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in api.fp4moe_mx_bytes(fmt, N, H))
    api.fp4moe_mx_quantize(fmt, w, gw, bc, bs)
    x, r = rnd((T, H), "bfloat16", 6), rnd((T, H), "bfloat16", 7)
    h, y = torch.empty_like(x), torch.empty_like(x)
    ac, as_ = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in api.fp4moe_mx_bytes(fmt, T, H))
    o, z = (torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    codes = torch.empty(T, N, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((N + 127) // 128, T, device="cuda")
    err = torch.zeros(4, dtype=torch.int32, device="cuda")

    def chain(stream=None):
        api.fp4moe_add_rmsnorm(x, r, None, 1e-6, h, y, stream=stream)
        api.fp4moe_mx_quantize(fmt, y, ga, ac, as_, stream)
        api.fp4moe_mx_gemm(fmt, H, ac, as_, bc, bs, alpha if fmt == NV else None, o, err, stream)
        api.fp4moe_add_rmsnorm(o, None, None, 1e-6, None, z, codes, scales, stream)

    def outputs():
        torch.cuda.synchronize()
        assert int(err[0]) == 0
        return [t.clone() for t in (h, y, ac, as_, o, z, codes.view(torch.uint8), scales)]

    chain()
    want = outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (h, y, o, z):
        t.zero_()
    torch.cuda.synchronize()
    chain(side)
    assert all(torch.equal(a, b) for a, b in zip(want, outputs()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for seed in (6, 60, 61):
        x.copy_(rnd((T, H), "bfloat16", seed))
        graph.replay()
        got = outputs()
        chain()
        assert all(torch.equal(a, b) for a, b in zip(got, outputs())), seed


# ------------------------------------------------------------------------- calls that find or meet an error
@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (64, 4096, 4096), (20, 8192, 4096), (128, 1024, 14336)])
def test_gemm_k_split_under_a_raised_error_word(fmt, M, N, K):
    """Every CTA of a cluster skips its part, and the next call's partial sums are whole."""
    import torch
    from block_scaled_fp4_top_gb300 import _lib, api
    ops = gemm_operands(fmt, M, N, K, 5)
    a, asf, _, b, bsf, _ = ops
    want = check_gemm(fmt, M, N, K, "float32", operands=ops).clone()
    ob = Guarded((M, N), torch.float32)
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    for _ in range(5):
        ob.t.fill_(7.0)
        err[0] = _lib.ERR_TIMEOUT
        for _ in range(3):
            api.fp4moe_mx_gemm(fmt, K, a, asf, b, bsf, None, ob.t, err)
        torch.cuda.synchronize()
        assert (ob.t == 7.0).all() and api.fp4moe_read_error(err) == _lib.ERR_TIMEOUT
        api.fp4moe_mx_gemm(fmt, K, a, asf, b, bsf, None, ob.t, err)
        torch.cuda.synchronize()
        assert int(err[0]) == 0 and torch.equal(ob.t, want)
        ob.check()


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (64, 8192, 8192), (128, 1024, 14336), (512, 4096, 4096)])
def test_gemm_under_an_error_word_that_is_raised_while_it_runs(M, N, K):
    """CTAs of one cluster may see it at different times. Each call ends, and leaves nothing to the next one."""
    import torch
    from block_scaled_fp4_top_gb300 import _lib, api
    ops = gemm_operands(MX, M, N, K, 6)
    a, asf, _, b, bsf, _ = ops
    ob = Guarded((M, N), torch.float32)
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    raised = torch.full((1,), _lib.ERR_TIMEOUT, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    call = lambda: api.fp4moe_mx_gemm(MX, K, a, asf, b, bsf, None, ob.t, err)
    call()
    torch.cuda.synchronize()
    want = ob.t.clone()
    for i in range(24):
        gate = torch.cuda.Event()
        torch.cuda._sleep(200_000)
        gate.record()
        for _ in range(8):
            call()
        with torch.cuda.stream(side):
            side.wait_event(gate)
            torch.cuda._sleep(1 + 4000 * i)
            err[:1].copy_(raised)
        torch.cuda.synchronize()
        assert api.fp4moe_read_error(err) == _lib.ERR_TIMEOUT
        ob.check()
        call()
        torch.cuda.synchronize()
        assert int(err[0]) == 0 and torch.equal(ob.t, want)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(9216, 4096, 1000), (2049, 3841, 4097)])
def test_gemm_large_tiles_with_every_scale_row(fmt, dtype, M, N, K):
    """Scales that differ from row to row across both halves of a 256 x 256 tile, and tile rows past the matrices."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    gen = torch.Generator("cuda").manual_seed(K)
    sides = []
    for rows in (M, N):
        x = torch.randn(rows, K, generator=gen, device="cuda") * torch.exp2(torch.arange(rows, device="cuda") % 9 - 4.0)[:, None]
        c, s = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in api.fp4moe_mx_bytes(fmt, rows, K))
        gs = torch.full((1,), 8.0, device="cuda")
        api.fp4moe_mx_quantize(fmt, x, gs, c, s)
        v = torch.empty(rows, K, device="cuda")
        one = torch.ones(1, device="cuda")
        api.fp4moe_mx_dequantize(fmt, c, s, one, v)                   # exact in fp32: tested on its own
        sides.append((c, s, v))
    (a, asf, av), (b, bsf, bv) = sides
    out = Guarded((M, N), getattr(torch, dtype))
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    al = torch.tensor([2.0 ** -6 if fmt == NV else 1.0], device="cuda")
    api.fp4moe_mx_gemm(fmt, K, a, asf, b, bsf, al, out.t, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    out.check()
    pick = torch.unique(torch.tensor([*range(0, M, 61), 127, 128, 255, 256, 383, 384, M - 1], device="cuda"))
    ap, bp = av[pick].double(), bv.double()
    ref = (ap @ bp.T * al.double()).cpu().numpy()
    mag = (ap.abs() @ bp.abs().T * al.double()).cpu().numpy()
    hold_product(f64(out.t[pick]), ref, mag, K, dtype)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("M,N,K", [(1025, 3001, 2100), (2000, 3600, 520)])
def test_gemm_on_pairs_under_a_raised_error_word(fmt, M, N, K):
    import torch
    from block_scaled_fp4_top_gb300 import _lib, api
    ops = gemm_operands(fmt, M, N, K, 5)
    a, asf, _, b, bsf, _ = ops
    want = check_gemm(fmt, M, N, K, "float32", operands=ops).clone()
    ob = Guarded((M, N), torch.float32)
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    for _ in range(5):
        ob.t.fill_(7.0)
        err[0] = _lib.ERR_TIMEOUT
        for _ in range(3):
            api.fp4moe_mx_gemm(fmt, K, a, asf, b, bsf, None, ob.t, err)
        torch.cuda.synchronize()
        assert (ob.t == 7.0).all() and api.fp4moe_read_error(err) == _lib.ERR_TIMEOUT
        api.fp4moe_mx_gemm(fmt, K, a, asf, b, bsf, None, ob.t, err)
        torch.cuda.synchronize()
        assert int(err[0]) == 0 and torch.equal(ob.t, want)
        ob.check()


@pytest.mark.parametrize("M,N,K", [(1025, 3001, 2100), (2048, 4096, 2048), (2000, 3600, 520)])
def test_gemm_on_pairs_under_an_error_word_that_is_raised_while_it_runs(M, N, K):
    """The two CTAs of a pair may see it at different stages. Each call ends, and leaves nothing to the next one."""
    test_gemm_under_an_error_word_that_is_raised_while_it_runs(M, N, K)


def test_tensors_on_another_device_are_refused(monkeypatch):
    """Seen from device 1, every tensor of this process is on another device. Nothing is launched."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    x = rnd((8, 128), "bfloat16", 1)
    y, codes8, scales = torch.empty_like(x), torch.empty(8, 128, dtype=torch.uint8, device="cuda"), torch.empty(1, 8, device="cuda")
    a, asf, _, b, bsf, _ = gemm_operands(MX, 8, 16, 128, 1)
    out, err = torch.full((8, 16), 7.0, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    lin = api.MxLinear(rnd((16, 128), "float32", 2), 8)
    q, s = (torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in api.fp4moe_mx_bytes(MX, 8, 128))
    calls = [lambda: api.fp4moe_add_rmsnorm(x, None, None, 1e-6, None, y, codes8, scales),
             lambda: api.fp4moe_mx_quantize(MX, x, None, q, s),
             lambda: api.fp4moe_mx_dequantize(MX, q, s, None, y),
             lambda: api.fp4moe_mx_gemm(MX, 128, a, asf, b, bsf, None, out, err),
             lambda: lin.forward(x, out)]
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(api, "_device", lambda: 1)
        for call in calls:
            with pytest.raises(api.Fp4MoeError, match="current"):
                call()
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (q == 7).all()
    for call in calls:
        call()
    torch.cuda.synchronize()
    assert int(err[0]) == 0 and (out != 7.0).any()


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("index", range(len(mx_plans.CASES)))
def test_gemm_every_plan(fmt, index):
    """Each kernel at the sizes that take it, and every element is written: a second result over other old values."""
    import torch
    from block_scaled_fp4_top_gb300 import api
    plan, (M, N, K) = mx_plans.CASES[index]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert api.fp4moe_mx_gemm_plan(M, N, K, sms) == plan
    dtype = DTYPES[index % 3]
    alpha = 2.0 ** -9 if dtype == "float16" else -1.75
    ops = gemm_operands(fmt, M, N, K, index)
    got = check_gemm(fmt, M, N, K, dtype, alpha=alpha, operands=ops)
    again = torch.full_like(got, float("nan"))
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    api.fp4moe_mx_gemm(fmt, K, ops[0], ops[1], ops[3], ops[4], torch.tensor([alpha], device="cuda"), again, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0 and not again.isnan().any() and torch.equal(got, again)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(8192, 4096, 2048), (8100, 4051, 2080)])
def test_gemm_writes_every_element_of_many_rounds(fmt, dtype, M, N, K):
    import torch
    from block_scaled_fp4_top_gb300 import api
    gen = torch.Generator("cuda").manual_seed(K)
    sides = []
    for rows in (M, N):
        c, s = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in api.fp4moe_mx_bytes(fmt, rows, K))
        api.fp4moe_mx_quantize(fmt, torch.randn(rows, K, generator=gen, device="cuda"), torch.ones(1, device="cuda"), c, s)
        sides += [c, s]
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    outs = []
    for old in (float("nan"), 7.0):
        ob = Guarded((M, N), getattr(torch, dtype))
        ob.t.fill_(old)
        api.fp4moe_mx_gemm(fmt, K, *sides, None, ob.t, err)
        torch.cuda.synchronize()
        ob.check()
        outs.append(ob.t)
    assert int(err[0]) == 0 and not outs[0].isnan().any() and torch.equal(*outs)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("M,N,K", [(8192, 8192, 1), (8192, 8192, 32), (8192, 4096, 100), (6000, 6000, 128), (5000, 7000, 129)])
def test_gemm_large_tiles_of_less_than_a_stage(fmt, M, N, K):
    """Fewer scale tiles across K than a load's box takes."""
    from block_scaled_fp4_top_gb300 import api
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert api.fp4moe_mx_gemm_plan(M, N, K, sms) == (256, 256, 1)
    test_gemm_large_tiles_with_every_scale_row(fmt, "float32", M, N, K)
