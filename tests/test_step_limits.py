"""Limits that attn_sink_step.h states, and integers past 32 bits in the conveniences."""
import pytest
import torch

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


def test_conveniences_refuse_sizes_past_32_bits():
    lens, table = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)
    sizes = dict(page_size=16, num_pages=4, max_tokens=8)
    for name in sizes:
        for n in ((1 << 32) + 16, 1 << 31):
            with pytest.raises(ValueError, match=f"{name}.*32 bits"):
                binding.page_plan(lens, lens, lens, table, **{**sizes, name: n})
    for name in ("heads_q", "heads_kv", "page_size", "num_pages"):
        kw = {"heads_q": 4, "heads_kv": 2, name: (1 << 32) + 4}
        with pytest.raises(ValueError, match=f"{name}.*32 bits"):
            binding.make_rope_params(3, rotary_dim=64, row_stride=512, **kw)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    none = torch.zeros(0, 1 << 33, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_cache.*32 bits"):
        binding.extend(q, none, none, table, lens, torch.zeros(4, dtype=torch.int32), torch.zeros(4))
