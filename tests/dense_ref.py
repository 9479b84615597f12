"""Plain 64-bit references of the dense operators (residual RMS norm, microscaled 4-bit matrices and their
product), on the oracle's codecs, and the buffers their tests use."""
from __future__ import annotations

import numpy as np

from oracle import codecs, mxfp4, nvfp4

NV, MX = 0, 1                                    # FP4MOE_W_NVFP4, FP4MOE_W_MXFP4
BLOCK = {NV: 16, MX: 32}
HALF_STEP = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": 2.0 ** -24}   # relative, of one rounding
TINY = {"bfloat16": 2.0 ** -134, "float16": 2.0 ** -25, "float32": 2.0 ** -150}     # half a subnormal step


def pad_to(v: np.ndarray, rows: int, cols: int) -> np.ndarray:
    out = np.zeros((rows, cols), dtype=v.dtype)
    out[:v.shape[0], :v.shape[1]] = v
    return out


def scale_tile_shape(fmt: int, rows: int, K: int):
    """(padded rows, padded scale columns) of the scale tiles."""
    C = -(-K // BLOCK[fmt])
    return -(-rows // 128) * 128, -(-C // 4) * 4


def quantize(fmt: int, x: np.ndarray, g) -> tuple[np.ndarray, np.ndarray]:
    """Finite fp32 x [rows, K] -> (codes [rows, ceil(K/32)*32] 0..15, scale bytes [rows, ceil(K/block)])."""
    rows, K = x.shape
    v = pad_to(x.astype(np.float32), rows, -(-K // 32) * 32)
    q, s = mxfp4.mx_quantize_rows(v) if fmt == MX else nvfp4.quantize_rows(v, np.float32(g))
    return q, s[:, :-(-K // BLOCK[fmt])]


def values(fmt: int, q: np.ndarray, s: np.ndarray, K: int) -> np.ndarray:
    """fp64 [rows, K] of codes and scale bytes, before any global scale."""
    table = codecs.E8M0_TABLE if fmt == MX else codecs.E4M3_TABLE
    return codecs.E2M1_TABLE[q[:, :K]] * np.repeat(table[s], BLOCK[fmt], axis=1)[:, :K]


def pack(fmt: int, q: np.ndarray, s: np.ndarray, K: int) -> tuple[np.ndarray, np.ndarray]:
    """(code bytes [rows, ceil(K/32)*16], scale tile bytes) as the library stores them."""
    R, C = scale_tile_shape(fmt, q.shape[0], K)
    return nvfp4.pack_codes(q), nvfp4.swizzle(pad_to(s, R, C))


def rms_norm(h: np.ndarray, gamma, eps: float) -> np.ndarray:
    """fp64 n of fp64 h."""
    n = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
    return n if gamma is None else n * gamma


def e4m3_half_step(v: np.ndarray) -> np.ndarray:
    """Half the spacing of E4M3 at |v| (3 mantissa bits, subnormals of 2^-9)."""
    a = np.abs(v)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    return np.where(a < 2.0 ** -6, 2.0 ** -10, 2.0 ** (e - 4))


class Guarded:
    """A device tensor with a canary on both sides, checked after the calls."""

    def __init__(self, shape, dtype, fill=None):
        import torch
        self.n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((self.n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        body = self.raw[256:256 + self.n]
        self.t = body.view(dtype).view(*shape) if self.n else torch.empty(shape, dtype=dtype, device="cuda")
        if fill is not None and self.n:
            self.t.copy_(fill)

    def check(self):
        assert (self.raw[:256] == 0xA5).all() and (self.raw[256 + self.n:] == 0xA5).all(), "write outside the buffer"
