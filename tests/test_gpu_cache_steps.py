"""The operators of attn_sink_cache.h as a serving loop uses them: after a plan and the
rotation, one after the other, captured into graphs, on other streams, called twice."""
import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.cache import oracle_attend, oracle_mass, oracle_select
from cache_cases import BF16, Paged, ints
from test_gpu_cache import SCORE, check

pytestmark = pytest.mark.gpu

HQ, HKV, PAGE = 16, 2, 16


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert binding.attn_sink_device_error() == (0, 0)


class Loop:
    """A serving loop of three sequences over one cache."""

    def __init__(self, pages=200, cols=40, batch=3):
        g = self.g = torch.Generator().manual_seed(5)
        self.kw = dict(heads_q=HQ, heads_kv=HKV)
        self.k = torch.zeros(pages, PAGE, HKV, 64, dtype=BF16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.bounds = torch.zeros(pages, HKV, 2, 64, dtype=BF16, device="cuda")
        self.table = torch.full((batch, cols), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
        self.lens = ints([0] * batch)
        self.positions = ints([0] * batch)                    # of the next token: own count
        self.inv_freq = (10000.0 ** (-torch.arange(32) / 32)).cuda()
        self.sink = torch.randn(HQ, generator=g).cuda()
        self.mass = torch.zeros(batch, HKV, cols * PAGE, device="cuda")

    def step(self, new):
        """Plan, rotation and bounds of a step; (q, plan)."""
        plan = binding.page_plan(self.lens, ints(new), self.free, self.table, page_size=PAGE,
                                 num_pages=self.k.shape[0], max_tokens=sum(new))
        qkv = torch.randn(sum(new), HQ + 2 * HKV, 64, generator=self.g).to(BF16).cuda()
        # the tokens' own positions: those of the plan, moved by what was evicted
        seq = torch.arange(len(new), device="cuda").repeat_interleave(ints(new).long())
        pos = plan.positions + (self.positions - self.lens)[seq]
        q, _, _ = binding.qkv_rope(qkv, pos, self.inv_freq, slots=plan.slots, k_cache=self.k,
                                   v_cache=self.v, **self.kw)
        binding.page_bounds(self.k, self.table, self.lens, plan.seq_lens, self.bounds)
        taken = int(plan.pages_needed)
        self.free = self.free[taken:].contiguous()
        self.lens = plan.seq_lens
        self.positions = self.positions + ints(new)
        return q, plan

    def keys(self):
        n = self.lens.tolist()
        return lambda b, h: range(n[b])

    def want(self, q, keys):
        return oracle_attend(q.cpu(), self.k.cpu(), self.v.cpu(), self.table.cpu(), keys,
                             self.sink.cpu(), scale=0.125)


def test_sparse_decode_steps():
    s = Loop()
    s.step([300, 17, 411])
    for _ in range(3):
        q, plan = s.step([1, 1, 1])
        sel = binding.select_pages(q, s.bounds, s.table, s.lens, count=8, page_size=PAGE)
        lens = s.lens.tolist()
        assert torch.equal(sel.cpu(), oracle_select(q.cpu(), s.bounds.cpu(), s.table.cpu(), lens,
                                                    page=PAGE, count=8, first=1, last=1))
        out, lse = binding.decode_pages(q, s.k, s.v, s.table, s.lens, sel, s.sink)
        cols = sel.cpu()
        check(out, lse, s.want(q, lambda b, h: [
            j for x in cols[b, h].tolist() if x >= 0
            for j in range(x * PAGE, min(lens[b], (x + 1) * PAGE))]))


def test_eviction_steps():
    s = Loop()
    mass = s.mass
    held = 0
    for new in ([300, 60, 411], [1, 1, 1], [1, 1, 1], [40, 1, 40], [1, 1, 1]):
        q, plan = s.step(new)
        cu = plan.cu_seqlens_q
        before = mass.clone()
        out, lse = binding.extend(q, s.k, s.v, s.table, s.lens, cu, s.sink)
        binding.key_mass(q, s.k, s.table, s.lens, cu, lse, mass)
        want = oracle_mass(q.cpu(), s.k.cpu(), s.table.cpu(), s.lens.tolist(), cu.tolist(),
                           lse.cpu(), before.cpu(), scale=0.125)
        assert ((mass.double().cpu() - want).abs() <= 1e-3 * want + 1e-30).all()
        if new == [1, 1, 1]:
            one, z, _ = binding.decode(q, s.k, s.v, s.table, s.lens, s.sink)
            check(one, z, s.want(q, s.keys()))
        r = binding.evict(s.k, s.v, s.table, s.lens, mass, budget=128, keep_first=4, keep_last=32)
        count = int(r.num_freed)
        held += count
        s.free = torch.cat([s.free, r.freed_pages[:count]])
        mass, s.lens = r.mass, r.seq_lens
        assert max(s.lens.tolist()) <= 128
        binding.page_bounds(s.k, s.table, ints([0, 0, 0]), s.lens, s.bounds)
    assert held > 0
    # no page is held twice: free ones and those of the sequences are all of them
    used = [int(x) for b in range(3) for x in s.table[b, : -(-int(s.lens[b]) // PAGE)]]
    assert sorted(used + s.free.tolist()) == list(range(s.k.shape[0]))


def test_shared_prefix_steps():
    """Two prompts, four samples each, that go on by themselves."""
    s = Loop(batch=8)
    prompts = [256, 96]
    s.step([prompts[0], 0, 0, 0, prompts[1], 0, 0, 0])
    for first, n in ((0, prompts[0]), (4, prompts[1])):
        s.table[first + 1:first + 4, : n // PAGE] = s.table[first, : n // PAGE]
    s.lens = ints([prompts[0]] * 4 + [prompts[1]] * 4)
    s.positions = s.lens.clone()
    for new in ([1] * 8, [3, 1, 2, 1, 20, 1, 1, 1], [1] * 8):
        q, plan = s.step(new)
        if new == [1] * 8:
            out, lse = binding.decode_shared(q, s.k, s.v, s.table, s.lens, ints([0, 4, 8]),
                                             ints(prompts), s.sink)
            check(out, lse, s.want(q, s.keys()), p_step=2 ** -8)


def operators(c, seed=7):
    """Every operator as a call without arguments on buffers of its own, and those outputs."""
    g = torch.Generator().manual_seed(seed)
    k, v, table, lens = c.gpu()
    q = c.q().cuda()
    sink = c.sink.cuda()
    cu = ints(list(range(len(c.lens) + 1)))
    bounds = torch.zeros(c.pages, c.hkv, 2, 64, dtype=BF16, device="cuda")
    none = torch.zeros_like(lens)
    mass = torch.rand(len(c.lens), c.hkv, c.cols * c.page, generator=g).cuda()
    one, z, _ = binding.decode(q, k, v, table, lens, sink)
    sel = torch.arange(5, dtype=torch.int32).expand(len(c.lens), c.hkv, 5).contiguous().cuda()
    groups, prefix = ints([0, len(c.lens)]), ints([128])
    return dict(
        shared=lambda **kw: binding.decode_shared(q, k, v, table, lens, groups, prefix, sink, **kw),
        bounds=lambda **kw: (binding.page_bounds(k, table, none, lens, bounds, **kw), bounds)[1:],
        select=lambda **kw: (binding.select_pages(q, bounds, table, lens, count=6, page_size=c.page,
                                                  **kw),),
        pages=lambda **kw: binding.decode_pages(q, k, v, table, lens, sel, sink, **kw),
        mass=lambda **kw: (binding.key_mass(q, k, table, lens, cu, z, mass, accumulate=False, **kw),),
        evict=lambda **kw: binding.evict(k, v, table, lens, mass, budget=100, keep_last=8, **kw))


def shared_table(seed=71):
    c = Paged(seed, [300, 200, 260, 150], hq=HQ, hkv=HKV)
    c.table[1:, :8] = c.table[0, :8]
    return c


def bits(results):
    return [x.cpu().contiguous().view(torch.uint8) for x in results]


@pytest.mark.parametrize("name", ["shared", "bounds", "select", "pages", "mass", "evict"])
def test_captured_replayed_and_on_another_stream(name):
    """The same bits from a plain call, a second one, one on a side stream and a graph that is
    replayed after its inputs' buffers were used by other calls."""
    ops = operators(shared_table())
    ops["bounds"](), ops["mass"]()
    call = ops[name]
    want = bits(call())
    assert all(torch.equal(a, b) for a, b in zip(bits(call()), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bits(got), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        for x in got:
            if name not in ("bounds", "mass"):
                x.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bits(got), want))


@pytest.mark.parametrize("name", ["shared", "pages", "select", "evict"])
def test_two_calls_at_once(name):
    """Calls that overlap on two streams, each with buffers of its own."""
    one, two = operators(shared_table(72)), operators(shared_table(73), 8)
    for ops in (one, two):
        ops["bounds"](), ops["mass"]()
    want = [bits(ops[name]()) for ops in (one, two)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [ops[name](stream=s) for ops, s in zip((one, two), streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(bits(g), w))


def test_given_outputs_are_used():
    c = shared_table(74)
    q = c.q().cuda()
    k, v, table, lens = c.gpu()
    out, lse = torch.empty_like(q), torch.empty(HQ, 4, device="cuda")
    sel = torch.arange(5, dtype=torch.int32).expand(4, HKV, 5).contiguous().cuda()
    a = binding.decode_pages(q, k, v, table, lens, sel, c.sink.cuda(), out=out, lse=lse)
    assert a[0].data_ptr() == out.data_ptr() and a[1].data_ptr() == lse.data_ptr()
    b = binding.decode_shared(q, k, v, table, lens, ints([0, 4]), ints([128]), c.sink.cuda(),
                              out=out, lse=lse)
    assert b[0].data_ptr() == out.data_ptr() and b[1].data_ptr() == lse.data_ptr()
