"""attn_sink_page_plan of many sequences: the sums before each group come from a kernel
of their own there."""
import pytest
import torch

from attention_learnable_head_gb300 import binding
from test_gpu_step import DEV, _check_plan, _clean, _code, _plan_case, _run_plan
from oracle.step import oracle_plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,launches", [(40001, 1), (65535, 1), (65536, 2), (70000, 2)])
def test_many_sequences(batch, launches):
    c, n, free, table, pages = _plan_case(batch, batch, 16, 60, 5)
    ref_table = [list(r) for r in table]
    ref = oracle_plan(c, n, free, ref_table, 16, sum(n) + 9)
    before = binding.attn_sink_launch_count()
    p, t = _run_plan(c, n, free, table, 16, pages, sum(n) + 9)
    assert binding.attn_sink_launch_count() - before == launches
    _check_plan(p, t, ref, ref_table)
    _clean()


def test_the_largest_batch():
    """2^24 sequences, in time that grows with their number (not with its square: 10^12
    loads)."""
    b, page = 1 << 24, 4
    g = torch.Generator(device=DEV).manual_seed(1)
    cached = torch.randint(0, 6, (b,), generator=g, device=DEV, dtype=torch.int32)
    new = torch.randint(0, 3, (b,), generator=g, device=DEV, dtype=torch.int32)
    have, end = (cached + 3) // page, (cached + new + 3) // page
    need = end - have
    total, pages = int(new.sum()), int(need.sum())
    held = torch.arange(2 * b, device=DEV, dtype=torch.int32).view(b, 2)
    table = torch.where(torch.arange(2, device=DEV)[None] < have[:, None], held, -1)
    free = torch.arange(2 * b, 2 * b + pages, device=DEV, dtype=torch.int32)
    p = binding.page_plan(cached, new, free, table, page_size=page, num_pages=2 * b + pages,
                          max_tokens=total + 5)
    _clean()
    base = need.cumsum(0) - need
    col = torch.arange(2, device=DEV)[None]
    want = torch.where(col < have[:, None], held,
                       torch.where(col < end[:, None], base[:, None] + col - have[:, None] + 2 * b, -1))
    assert torch.equal(table, want.int())
    cu = new.cumsum(0)
    assert torch.equal(p.cu_seqlens_q[1:], cu.int()) and p.cu_seqlens_q[0].item() == 0
    assert torch.equal(p.seq_lens, cached + new) and p.pages_needed.item() == pages
    who = torch.repeat_interleave(torch.arange(b, device=DEV), new)
    pos = torch.arange(total, device=DEV) - (cu - new)[who] + cached[who]
    assert torch.equal(p.positions[:total], pos.int()) and not p.positions[total:].any()
    assert torch.equal(p.slots[:total], want[who, pos // page] * page + pos % page)
    assert (p.slots[total:] == -1).all()


def test_what_does_not_fit():
    """Far more tokens than there is room for: sums beyond 32 bits."""
    b = 66000
    i32 = dict(dtype=torch.int32, device=DEV)
    new = torch.full((b,), 1 << 20, **i32)
    table = torch.full((b, 1), -1, **i32)
    p = binding.page_plan(torch.zeros_like(new), new, torch.arange(10, **i32), table,
                          page_size=1 << 20, num_pages=10, max_tokens=100)
    assert _code() == 0x1000
    assert p.pages_needed.item() == b and p.slots.tolist() == list(range(100))
    assert p.cu_seqlens_q[0].item() == 0 and (p.cu_seqlens_q[1:] == 100).all()
    assert (p.seq_lens == 1 << 20).all()
    assert table[:10, 0].tolist() == list(range(10)) and (table[10:] == -1).all()
