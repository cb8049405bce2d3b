"""Sizes of the workspaces of attn_sink_cache.h, without a GPU."""
import pytest

from attention_learnable_head_gb300 import binding
from attention_learnable_head_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    return binding.lib()


def shared(batch, groups, heads=(64, 8)):
    return binding.attn_sink_decode_shared_workspace_size(binding.AttnSinkSharedParams(
        batch, groups, *heads, 64, 16, 1 << 16, 512, 0.125))


@pytest.mark.parametrize("batch", [2, 7, 64, 4096, 65535])
@pytest.mark.parametrize("heads", [(64, 8), (8, 8), (8, 1)])
def test_groups_of_one_take_no_workspace(batch, heads):
    """A group without a second sequence has no prefix of its own: there are batch / 2 others at
    most."""
    assert shared(batch, batch, heads) == shared(batch, batch // 2, heads)
    assert shared(batch, 1, heads) <= shared(batch, batch, heads)


def test_more_groups_with_a_prefix_take_more():
    assert shared(4096, 1) < shared(4096, 100) < shared(4096, 2048)
    assert shared(1, 1) > 0
