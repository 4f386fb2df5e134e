"""The norms, the attention of several tokens and the cut of the cache on
tensors of a GPU that is not the current one (as tests/test_current_device.py,
whose library says which GPU was current)."""
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

from test_current_device import cache, i32, where  # noqa: E402,F401


def test_norms(where):  # noqa: F811
    x, table, w = torch.zeros(3, 2, 64, requires_grad=True), torch.zeros(8, 32, 2), torch.ones(64, requires_grad=True)
    gbb.norm_rope(x, w, i32(3), table).sum().backward()
    gbb.rope(x.detach(), i32(2, 3), table, sections=(20, 12))
    gbb.rope_append(cache(), torch.zeros(3, 8 * 64, dtype=torch.float16), 4, i32(3), i32(3), table, q_norm=torch.ones(64),
                    k_norm=torch.ones(64))


@pytest.mark.parametrize("workspace", [None, torch.zeros(64, dtype=torch.uint8)])
def test_attention(where, workspace):  # noqa: F811
    c, q = cache(), torch.zeros(3, 4, 64, dtype=torch.float16)
    gbb.paged_attention(c, q[:1], i32(1, 2), i32(1), 32, workspace=workspace, softcap=3.0, window=5)
    gbb.paged_attention_tokens(c, q, i32(2), i32(1, 2), i32(1), 32, workspace=workspace, tree=i32(3, 1))
    if workspace is None:
        assert ("capturing", -1) in where


def test_keep_and_plans(where):  # noqa: F811
    gbb.cache_keep(cache(), i32(1, 2), i32(1), i32(1), i32(1, 2), i32(1))
    assert gbb.paged_attention_tokens_workspace(cache(), 3, 1, 4, 32, window=3, tree_words=1) == 64
