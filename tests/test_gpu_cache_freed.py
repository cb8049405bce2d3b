"""The list of freed pages holds pages alone, whatever the block table has."""
import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.cache import oracle_evict
from cache_cases import Paged
from test_gpu_cache import evict_both, random_mass, recorded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert binding.attn_sink_device_error() == (0, 0)


def wipe(c, budget, share):
    """Entries outside the cache in the place of some pages that become free; whether any."""
    odd = torch.tensor([-1, c.pages, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    wiped = False
    for b, n in enumerate(c.lens):
        for col in range(-(-budget // c.page), -(-n // c.page)):
            if torch.rand(1, generator=c.g) < share:
                c.table[b, col] = odd[int(torch.randint(0, 4, (1,), generator=c.g))]
                wiped = True
    return wiped


@pytest.mark.parametrize("share", [0.1, 0.6, 1.0])
@pytest.mark.parametrize("lens,kw,budget", [
    ([300, 20, 0, 301], {}, 100),                             # moved by a second kernel
    ([5000, 7, 6000, 30], dict(page=1, hkv=1, hq=1), 20),     # more pages than threads
    ([40 + b % 30 for b in range(400)], dict(hkv=1, hq=1, page=8), 17),   # rows on their own CTAs
    ([9 + b % 5 for b in range(1500)], dict(hkv=1, hq=1, page=1), 8),     # several rounds
])
def test_entries_outside_the_cache_are_no_pages(lens, kw, budget, share):
    c = Paged(101, lens, **kw)
    wiped = wipe(c, budget, share)
    evict_both(c, random_mass(c), budget, 0, 0)
    assert recorded() == (0, 0x800 if wiped else 0)


def test_lists_that_do_not_fit():
    """num_freed counts them all; the list holds the first ones."""
    c = Paged(102, [300, 290])
    wipe(c, 50, 0.3)
    m = random_mass(c)
    freed = oracle_evict(c.k, c.v, c.table, c.lens, m, budget=50, first=0, last=0)[4]
    k, v, table, lens = c.gpu()
    for room in (0, 1, 9, len(freed)):
        p = binding.AttnSinkEvictParams(2, 2, 64, 16, c.pages, c.cols, c.cols * 16, 50, 0, 0, room)
        need = binding.attn_sink_evict_workspace_size(p)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out, new = torch.empty_like(m).cuda(), torch.empty_like(lens)
        got = torch.full((room + 3,), -7, dtype=torch.int32, device="cuda")
        count = torch.full((1,), -7, dtype=torch.int32, device="cuda")
        assert binding.attn_sink_evict(p, k.clone(), v.clone(), table, lens, m.cuda(), out, new, got,
                                       count, ws, need) == 0
        assert recorded() == (0, 0x800)
        assert count.item() == len(freed) and got.tolist() == freed[:room] + [-7] * 3


def test_the_next_plan_takes_them():
    """A step after an eviction of tables with holes: the plan gives away pages alone."""
    c = Paged(103, [300, 290, 280])
    wipe(c, 50, 0.3)
    k, v, table, lens = c.gpu()
    r = binding.evict(k, v, table, lens, random_mass(c).cuda(), budget=50)
    assert recorded() == (0, 0x800)
    new = torch.full((3,), 60, dtype=torch.int32, device="cuda")
    assert r.num_freed.item() >= 12
    plan = binding.page_plan(r.seq_lens, new, r.freed_pages, table, page_size=16,
                             num_pages=c.pages, max_tokens=180)
    used = table[:, :7].flatten().tolist()
    assert plan.seq_lens.tolist() == [110] * 3 and len(set(used)) == 21
    assert min(used) >= 0 and max(used) < c.pages
