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
