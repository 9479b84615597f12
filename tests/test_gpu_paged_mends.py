"""GPU: the paged cache's calls after a call that gave up, with values that are not finite far inside long sequences, with
weights across the range of fp16, with lengths and positions at their limits. Against the 64-bit references of paged_ref.py,
with the tolerances that test_gpu_paged.py derives."""
import math

import numpy as np
import pytest

import paged_ref as ref
from helpers import ensure_built
from test_gpu_paged import attention_case, compare, ints, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# ------------------------------------------------------------------------- after a timeout
@pytest.mark.parametrize("D,new", [(128, [1, 1]), (64, [130, 3]), (256, [2, 1])])
def test_a_cache_after_a_call_that_gave_up(D, new):
    """Counters of joins that were left counting do not reach the calls after the word has been read and cleared."""
    import torch
    from block_scaled_fp4_top_gb300 import _lib, api
    H, Hk, B = 8, 2, len(new)
    cache = api.PagedKvCache(400, 16, Hk, D, B, 3000, 3000)
    inv = api.rope_inv_freq(D)
    gen = torch.Generator("cuda").manual_seed(D)
    for lengths in ([2800, 150], new):
        T = sum(lengths)
        cache.plan(ints(lengths))
        q, k, v = (torch.randn(T, h, D, device="cuda", generator=gen).bfloat16() for h in (H, Hk, Hk))
        cache.append(q, k, v, inv, q)
    out = torch.empty_like(q)

    def attend(q, out):
        out.fill_(5.0)
        cache.attend(q, D ** -0.5, out)
        torch.cuda.synchronize()
        return out

    want = attend(-q, torch.empty_like(q))
    attend(q, out)                                            # its parts lie in the workspace now
    assert cache.read_error() == 0 and not cache.ws[:4096].any()
    cache.ws[256:4096].view(torch.int32).fill_(1)             # what a call that gives up may leave
    cache.err[0] = _lib.ERR_TIMEOUT
    assert (attend(-q, out) == 5.0).all()                     # skipped
    assert cache.read_error(clear=False) == _lib.ERR_TIMEOUT
    assert (attend(-q, out) == 5.0).all()                     # still
    assert cache.read_error() == _lib.ERR_TIMEOUT
    for _ in range(3):
        assert torch.equal(attend(-q, out).view(torch.int16), want.view(torch.int16))
        assert cache.read_error() == 0 and not cache.ws[:4096].any()
