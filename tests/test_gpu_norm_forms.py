"""GPU: the residual norm's results do not depend on what else a call computes: y is bit-equal with and without the
FP8 copy."""
import pytest

from helpers import ensure_built
from test_gpu_dense import DTYPES, rnd

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
