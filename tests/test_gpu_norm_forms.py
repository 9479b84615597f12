"""GPU: the residual norm's results do not depend on what else a call computes, nor on a row's other groups, nor on the
kernel that the width selects: y is bit-equal with and without the FP8 copy, and the copy's codes are those of exact
arithmetic (bf16) in every kernel, beside groups of any magnitude."""
import numpy as np
import pytest

from helpers import ensure_built
from oracle import codecs
from test_gpu_dense import DTYPES, f64, rnd

pytestmark = pytest.mark.gpu
# 16-byte vectors with one, two and four a thread; 8-, 4- and 2-byte accesses; rows that no CTA's registers hold
SIZES = [(9, 4096), (200, 512), (400, 4096), (700, 1000), (9, 4092), (200, 1002), (9, 1001), (300, 4090), (3, 40960),
         (3, 40961)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def norm(x, residual, gamma, fp8=True, eps=1e-6):
    """(residual stream, y, codes, scales)"""
    import torch
    from block_scaled_fp4_top_gb300 import api
    T, H = x.shape
    h = torch.empty_like(x) if residual is not None else None
    y = torch.empty_like(x)
    codes = torch.empty(T, H, dtype=torch.uint8, device="cuda") if fp8 else None
    scales = torch.empty((H + 127) // 128, T, device="cuda") if fp8 else None
    api.fp4moe_add_rmsnorm(x, residual, gamma, eps, h, y, codes, scales)
    torch.cuda.synchronize()
    return h, y, codes, scales


def exact_codes(h, g):
    """E4M3 codes of n / s = 448 p / max|p| with p = h * gamma, for bf16 h and gamma: in fp64 that side and a midpoint of
    the E4M3 grid times max|p| are exact products, so every code, ties to even included, follows from comparisons."""
    T, H = h.shape
    G = (H + 127) // 128
    p = np.zeros((T, G * 128))
    p[:, :H] = f64(h) * (f64(g) if g is not None else 1.0)
    top = np.repeat(np.abs(p).reshape(T, G, 128).max(2), 128, axis=1)
    grid = codecs.E4M3_TABLE[:127].astype(np.float64)
    want = np.zeros(p.shape, dtype=np.int64)
    for i, mid in enumerate((grid[1:] + grid[:-1]) / 2):
        side, bar = 448.0 * np.abs(p), mid * top
        want += (side > bar) | ((side == bar) & (i % 2 == 1) & (top > 0))
    return want[:, :H], p[:, :H] < 0


def hold_codes(codes, h, g, where=None):
    want, negative = exact_codes(h, g)
    got = codes.cpu().numpy().astype(np.int64)
    differ = ((got & 127) != want) | ((got >> 7 != negative) & (want != 0))     # the sign of a zero is free
    if where is not None:
        differ &= where
    assert not differ.any(), f"{differ.sum()} codes of {differ.size}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("gamma", [False, True])
def test_y_is_the_same_with_and_without_the_fp8_copy(dtype, T, H, gamma):
    import torch
    x, r = rnd((T, H), dtype, H), rnd((T, H), dtype, H + 1)
    g = rnd((H,), dtype, H + 2, 0.0) if gamma else None
    with_copy, without = norm(x, r, g), norm(x, r, g, fp8=False)
    assert torch.equal(with_copy[0], without[0]) and torch.equal(with_copy[1], without[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_a_call_repeats_itself(dtype, T, H):
    import torch
    x, r, g = rnd((T, H), dtype, H), rnd((T, H), dtype, H + 1), rnd((H,), dtype, H + 2, 0.0)
    first = norm(x, r, g)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(first, norm(x, r, g)))


@pytest.mark.parametrize("T,H", [(64, 4096), (400, 4096), (200, 1002)])
@pytest.mark.parametrize("other", [0.0, 2.0 ** -90])
def test_codes_do_not_depend_on_the_group_beside(T, H, other):
    """Every second group is zeros, or too small for the short way to the codes."""
    h, g = rnd((T, H), "bfloat16", H, 0.5), rnd((H,), "bfloat16", H + 1, 0.0)
    group = np.arange(H) // 128
    for odd in (0, 1):
        x = h.clone()
        x[:, group % 2 == odd] *= other
        _, _, codes, _ = norm(x, None, g)
        hold_codes(codes, x, g, np.broadcast_to(group % 2 != odd, (T, H)))


@pytest.mark.parametrize("T,H", [(40, 40960), (40, 40962)])
@pytest.mark.parametrize("gamma", [False, True])
def test_codes_of_wide_rows_are_those_of_exact_arithmetic(T, H, gamma):
    h = rnd((T, H), "bfloat16", H, 0.5)
    g = rnd((H,), "bfloat16", H + 1, 0.0) if gamma else None
    _, _, codes, _ = norm(h, None, g)
    hold_codes(codes, h, g)
