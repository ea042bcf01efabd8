"""Refusals of include/pi_draft.h that concern how arguments stand to one another."""
import activation_sparse_decode_rank_gb300 as pi
import pytest

P = 1 << 40  # stand-in address: every call below is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def _built():
    pi.build()


@pytest.mark.parametrize("head_dim", [64, 256])
def test_attention_refuses_to_write_over_its_queries(head_dim):
    c = pi.make_cache_desc(layers=2, pages=100, kv_heads=4, head_dim=head_dim, page_tokens=16, dtype="f16")
    size = pi.pi_tree_workspace_size(c, 4, 8, 5)
    rc = pi.pi_tree_attention(c, 0, 4, 8, 10, 5, P, P, P + 4096, None, None, P, P, P, 0.125, 0, 0, P + 4096, P, P,
                              P, size, stream=0)
    assert rc == pi.PI_ERR_SHAPE
