"""Calls at the limits that the parameters allow."""
import pytest
import torch

from attention_learnable_head_gb300 import binding
from cache_cases import BF16, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert binding.attn_sink_device_error() == (0, 0)


@pytest.mark.parametrize("page", [2 ** 31 - 1, 2 ** 30 + 1, 2 ** 30])
def test_pages_of_the_largest_size_without_a_table(page):
    """Pages of more than 2^30 keys are allowed where the table has no column: the calls return,
    and every head has its sink alone."""
    k = torch.empty(0, page, 2, 64, dtype=BF16, device="cuda")
    table = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    lens, q = ints([0, 0, 0]), torch.ones(3, 8, 64, dtype=BF16, device="cuda")
    sink = torch.randn(8, device="cuda")
    sel = torch.empty(3, 2, 0, dtype=torch.int32, device="cuda")
    bounds = torch.empty(0, 2, 2, 64, dtype=BF16, device="cuda")
    mass = torch.ones(3, 2, 5, device="cuda")
    for out, lse in (binding.decode(q, k, k, table, lens, sink)[:2],
                     binding.decode_shared(q, k, k, table, lens, ints([0, 2, 3]), ints([9, 0]), sink),
                     binding.decode_pages(q, k, k, table, lens, sel, sink)):
        assert not out.any()
        # times log2(e), ln(2) and both constants themselves rounded: four steps of 2^-24
        assert ((lse - sink[:, None]).abs() <= 2 ** -22 * sink[:, None].abs()).all()
    binding.page_bounds(k, table, lens, lens, bounds)
    got = binding.select_pages(q, bounds, table, lens, count=4, page_size=page)
    assert (got == -1).all()
    binding.key_mass(q, k, table, lens, ints([0, 1, 2, 3]), sink[:, None].expand(8, 3).contiguous(), mass)
    assert (mass == 1).all()
    r = binding.evict(k, k, table, lens, mass, budget=2)
    assert r.num_freed.item() == 0 and not r.mass.any() and r.seq_lens.tolist() == [0, 0, 0]
