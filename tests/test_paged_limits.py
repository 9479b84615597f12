"""The paged cache's calls at the ends of their arguments' ranges, as far as the host decides them (no GPU)."""
import pytest

from helpers import ensure_built


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("T,H,Hk,D", [(0, 32, 8, 128), (1, 1, 1, 8), (100, 32, 8, 128), (100, 64, 8, 64), (8192, 32, 8, 128),
                                      (8192, 64, 1, 64)])
def test_plan_of_no_sequences(T, H, Hk, D):
    """The header: num_seqs or T 0: 16."""
    from block_scaled_fp4_top_gb300 import api
    assert api.fp4moe_paged_attention_plan(0, T, H, Hk, D) == 16


@pytest.mark.parametrize("rows", [-1, 101])
def test_rows_of_a_step_that_the_cache_was_not_made_for(rows):
    import torch
    from block_scaled_fp4_top_gb300 import api
    ws, api._lib.ATTENTION_WORKSPACE_BYTES = api._lib.ATTENTION_WORKSPACE_BYTES, 64
    try:
        cache = api.PagedKvCache(4, 16, 1, 8, 2, 64, 100, device="cpu")
    finally:
        api._lib.ATTENTION_WORKSPACE_BYTES = ws
    with pytest.raises(api.Fp4MoeError, match="rows"):
        cache.plan(torch.zeros(2, dtype=torch.int32), rows=rows)


def test_no_read_only_loads_of_what_the_calls_write():
    """A kernel may start before the one in front of it has ended, and one output may be an input: what these calls write
    (lengths, tables, offsets, positions, slots, q, the caches) is memory that changes while a kernel lives, which loads of the
    read-only kind are not defined for and which a compiler may move in front of the wait for the kernel before."""
    import os
    import re
    from helpers import ROOT
    for name in ("kvplan.cu", "rope.cu", "attn.cu", "attn.cuh", "attntile.cu", "paged.cuh"):
        with open(os.path.join(ROOT, "block_scaled_fp4_top_gb300", "csrc", name)) as f:
            text = f.read()
        assert [m for m in re.findall(r"__ldg\(([^)]*)\)", text) if not m.startswith("p.inv_freq")] == [], name
        assert "ld.global.nc" not in text and "__restrict__" not in text, name
