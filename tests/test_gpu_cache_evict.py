"""What an eviction leaves in the caches themselves, bit for bit: in every form of the call
(moves by the row's own CTA or by a second kernel, listed in shared memory or in the
workspace), repeated, on another stream, replayed from a graph, and two at once."""
import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.cache import oracle_evict
from cache_cases import Paged
from test_gpu_cache import evict_both, random_mass

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert binding.attn_sink_device_error() == (0, 0)


@pytest.mark.parametrize("keys,budget", [
    (10200, 400),                                             # lists in the workspace
    (3000, 900),                                              # in shared memory
    (130, 100),
])
def test_rows_that_move_themselves(keys, budget):
    """160 rows and more are moved by the CTAs that choose."""
    c = Paged(121, [max(keys - 7 * b, 0) for b in range(20)], hq=8, hkv=8)
    evict_both(c, random_mass(c), budget, 4, 32)


def bits(x):
    return x.cpu().contiguous().view(torch.int16)


class Case:
    def __init__(self, seed, lens, budget, **kw):
        c = self.c = Paged(seed, lens, **kw)
        m = random_mass(c)
        self.budget = budget
        self.k0, self.v0, self.table, self.lens = c.gpu()
        self.k, self.v, self.mass = self.k0.clone(), self.v0.clone(), m.cuda()
        want = oracle_evict(c.k, c.v, c.table, c.lens, m, budget=budget, first=2, last=9)
        self.want_k, self.want_v, self.want_mass = bits(want[0]), bits(want[1]), want[2]

    def call(self, **kw):
        return binding.evict(self.k, self.v, self.table, self.lens, self.mass, budget=self.budget,
                             keep_first=2, keep_last=9, **kw)

    def restore(self):
        self.k.copy_(self.k0)
        self.v.copy_(self.v0)
        torch.cuda.synchronize()

    def check(self, r):
        torch.cuda.synchronize()
        assert torch.equal(bits(self.k), self.want_k) and torch.equal(bits(self.v), self.want_v)
        assert torch.equal(r.mass.cpu(), self.want_mass)


CASES = [dict(lens=[300, 200, 260, 150], budget=100, hq=16, hkv=2),          # a second kernel moves
         dict(lens=[200 - b for b in range(90)], budget=100, hq=2, hkv=2)]   # the rows' own CTAs


@pytest.mark.parametrize("kw", CASES)
def test_repeated_on_another_stream_and_replayed(kw):
    case = Case(122, **kw)
    for _ in range(3):
        case.restore()
        case.check(case.call())
    side = torch.cuda.Stream()
    case.restore()
    r = case.call(stream=side)
    side.synchronize()
    case.check(r)
    graph = torch.cuda.CUDAGraph()
    case.restore()
    with torch.cuda.graph(graph):
        r = case.call()
    for _ in range(3):
        case.restore()
        r.mass.fill_(-7)
        graph.replay()
        case.check(r)


@pytest.mark.parametrize("one", CASES)
@pytest.mark.parametrize("two", CASES)
def test_two_at_once(one, two):
    """Calls that overlap on two streams, each on caches of its own, time after time."""
    cases = [Case(123, **one), Case(124, **two)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for x in cases:
            x.restore()
        got = [x.call(stream=s) for x, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for x, r in zip(cases, got):
            x.check(r)


@pytest.mark.parametrize("kw", CASES)
def test_a_step_behind_sees_the_moved_keys(kw):
    """The next call of the stream reads the caches as the moves leave them."""
    case = Case(125, **kw)
    q, sink = case.c.q().cuda(), case.c.sink.cuda()
    cu = torch.arange(len(case.c.lens) + 1, dtype=torch.int32, device="cuda")
    none = torch.zeros(len(case.c.lens), dtype=torch.int32, device="cuda")
    got = []
    for wait in (True, False):
        case.restore()
        r = case.call()
        if wait:
            torch.cuda.synchronize()
        got.append(binding.decode_shared(q, case.k, case.v, case.table, r.seq_lens, cu, none, sink))
    for a, b in zip(*got):
        assert torch.equal(a, b)
