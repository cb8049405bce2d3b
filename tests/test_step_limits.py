"""Limits that attn_sink_step.h states, and integers past 32 bits in the conveniences."""
import pytest

from attention_learnable_head_gb300 import binding
from attention_learnable_head_gb300.build import build

UNSUPPORTED, WORKSPACE = 2, 3
FAKE = 0x7F0000000000       # never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


@pytest.mark.parametrize("batch,total_q,status", [
    (1 << 24, 1 << 30, WORKSPACE), ((1 << 24) + 1, 1 << 24, UNSUPPORTED),
    (4, (1 << 30) + 1, UNSUPPORTED), ((1 << 31) - 1, (1 << 31) - 1, UNSUPPORTED)])
def test_extend_states_its_largest_sizes(batch, total_q, status):
    p = binding.AttnSinkExtendParams(batch, total_q, 1, 1, 64, 16, 64, 8, 0, 0.125)
    assert binding.attn_sink_extend(p, *[FAKE] * 9, None, 0, stream=0) == status
    assert (binding.attn_sink_extend_workspace_size(p) > 0) == (status == WORKSPACE)
