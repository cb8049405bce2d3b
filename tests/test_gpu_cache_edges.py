"""attn_sink_cache.h where it can go wrong: slices that a kernel of its own joins, groups
that leave sequences out, caches beyond 32 bits of bytes, heads and scales that take
another path, waits that run out."""
import ctypes
import math
import time

import pytest
import torch

from attention_learnable_head_gb300 import binding
from attention_learnable_head_gb300.build import build
from oracle.cache import oracle_attend, oracle_bounds, oracle_evict, oracle_mass, oracle_select
from cache_cases import BF16, Paged, ints
from test_gpu_cache import (SCORE, all_keys, check, decode_shared, mass_both, mass_case,
                            random_bounds, random_lists, random_mass, recorded, shared_case)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert binding.attn_sink_device_error() == (0, 0)


# ----------------------------------------------------------------------------- joined slices
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("groups", [[(512, [600, 3000, 5000])], [(0, [5000]), (640, [700, 641, 2600])],
                                    [(200, [9000, 200, 230]), (64, [0, 70])]])
def test_shared_with_long_own_keys(groups, page):
    """Few sequences behind a table of thousands of keys: several slices each."""
    c, cu, prefix = shared_case(81, groups, page=page, hq=8, hkv=1)
    q = c.q()
    out, lse = decode_shared(c, q, cu, prefix)
    check(out, lse, oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125),
          p_step=2 ** -8)


@pytest.mark.parametrize("cols", [20, 600])
@pytest.mark.parametrize("cu,prefix,same", [
    ([1, 3], [128], True),                                    # sequences before and behind the group
    ([0, 2], [128], True), ([2, 4], [128], True),
    ([0, 4, 0, 4], [128] * 3, False), ([0, 9, 4, 4], [128] * 3, False),
    ([-7, 2, 2 ** 31 - 1], [2 ** 31 - 1, -5], False)])
def test_shared_groups_that_are_none(cu, prefix, same, cols):
    """Sequences outside every group read all keys themselves; groups that overlap or leave
    the batch are recorded, and nothing outside the buffers is read.  Short tables (one
    slice) and long ones (several)."""
    c, _, _ = shared_case(82, [(128, [140, 200, 150, 129])], cols=cols, hq=8, hkv=1)
    q = c.q()
    # buffers that held something else before
    torch.full((1 << 22,), 2 ** 30 - 1, dtype=torch.int32, device="cuda")
    out, lse = decode_shared(c, q, cu, prefix)
    assert recorded() == (0, 0x800)
    if same:
        check(out, lse, oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125),
              p_step=2 ** -8)


# ----------------------------------------------------------------------------- beyond 32 bits
class Far:
    """A small cache at the end of one of more than 2^32 bytes."""

    def __init__(self, c):
        row = c.page * c.hkv * 64
        self.at = (2 ** 32 + 2 ** 31) // (2 * row) + 5
        self.pages = self.at + c.pages
        self.k, self.v = (torch.empty(self.pages, c.page, c.hkv, 64, dtype=BF16, device="cuda")
                          for _ in range(2))
        self.k[self.at:], self.v[self.at:] = c.k.cuda(), c.v.cuda()
        self.table = torch.where(c.table >= 0, c.table + self.at, c.table).cuda()
        self.lens = c.lens_gpu()


@pytest.mark.parametrize("page", [16, 24])
def test_caches_beyond_32_bits_of_bytes(page):
    c, cu, prefix = shared_case(83, [(192, [300, 200, 410])], page=page, hq=16, hkv=2)
    f = Far(c)
    q, sink = c.q(), c.sink.cuda()
    out, lse = binding.decode_shared(q.cuda(), f.k, f.v, f.table, f.lens, ints(cu), ints(prefix), sink)
    check(out, lse, oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125),
          p_step=2 ** -8)
    bounds = torch.zeros(f.pages, 2, 2, 64, dtype=BF16, device="cuda")
    binding.page_bounds(f.k, f.table, ints([0] * 3), f.lens, bounds)
    near = oracle_bounds(c.k, c.table, [0] * 3, c.lens, torch.zeros(c.pages, 2, 2, 64, dtype=BF16))
    assert torch.equal(bounds[f.at:].cpu(), near) and not bounds[:f.at].any()
    sel = binding.select_pages(q.cuda(), bounds, f.table, f.lens, count=5, page_size=page)
    assert torch.equal(sel.cpu(), oracle_select(q, near, c.table, c.lens, page=page, count=5, first=1,
                                                last=1))
    out, lse = binding.decode_pages(q.cuda(), f.k, f.v, f.table, f.lens, sel, sink)
    cols = sel.cpu()
    check(out, lse, oracle_attend(q, c.k, c.v, c.table, lambda b, h: [
        j for x in cols[b, h].tolist() if x >= 0
        for j in range(x * page, min(c.lens[b], (x + 1) * page))], c.sink, scale=0.125))
    for new in ([1, 1, 1], [40, 9, 30]):
        at = torch.tensor([0] + new).cumsum(0).tolist()
        qq = c.q(at[-1])
        z = 3 + torch.rand(16, at[-1], generator=c.g)
        mass = torch.zeros(3, 2, c.cols * page, device="cuda")
        binding.key_mass(qq.cuda(), f.k, f.table, f.lens, ints(at), z.cuda(), mass)
        want = oracle_mass(qq, c.k, c.table, c.lens, at, z, torch.zeros(mass.shape), scale=0.125)
        assert ((mass.double().cpu() - want).abs() <= (2 * SCORE + 56 * 2 ** -24) * want + 1e-30).all()
    c = Paged(84, [300, 200, 410], page=page)                 # no page in two tables
    f = Far(c)
    m = random_mass(c)
    r = binding.evict(f.k, f.v, f.table, f.lens, m.cuda(), budget=100, keep_first=1, keep_last=9)
    k, v, wm, wl, freed = oracle_evict(c.k, c.v, c.table, c.lens, m, budget=100, first=1, last=9)
    assert torch.equal(f.k[f.at:].cpu().view(torch.int16), k.view(torch.int16))
    assert torch.equal(f.v[f.at:].cpu().view(torch.int16), v.view(torch.int16))
    assert torch.equal(r.mass.cpu(), wm) and r.seq_lens.tolist() == wl
    assert r.freed_pages[:len(freed)].tolist() == [x + f.at for x in freed]


# ----------------------------------------------------------------------------- weights, other paths
@pytest.mark.parametrize("group", [3, 7, 12, 33, 64, 96, 97, 128])
def test_key_mass_group_sizes(group):
    mass_both(*mass_case(85, [9, 40], [300, 513], hq=group, hkv=1))


@pytest.mark.parametrize("scale", [1e-4, 2.0 ** -10, 3.0, 2.0 ** 10, 5000.0])
def test_key_mass_scales(scale):
    """Scores of about one for every scale: the queries are divided by it."""
    c, cu, _, lse = mass_case(86, [40, 70], [300, 513])
    q = (torch.randn(cu[-1], c.hq, 64, generator=c.g) * 0.125 / scale).to(BF16)
    k, _, table, lens = c.gpu()
    mass = torch.zeros(2, 2, c.cols * c.page, device="cuda")
    binding.key_mass(q.cuda(), k, table, lens, ints(cu), lse.cuda(), mass, softmax_scale=scale)
    want = oracle_mass(q, c.k, c.table, c.lens, cu, lse, torch.zeros(mass.shape), scale=scale)
    assert ((mass.double().cpu() - want).abs() <= (2 * SCORE + 300 * 2 ** -24) * want + 1e-30).all()


@pytest.mark.parametrize("new", [[1, 1], [40, 70]])
def test_key_mass_large_lse(new):
    """lse of hundreds, with the scores next to them or far below, and rows that differ by much."""
    c, cu, q, lse = mass_case(87, new, [300, 513])
    c.k *= 20
    k, _, table, lens = c.gpu()
    _, lse = binding.extend(q.cuda(), k, c.v.cuda(), table, lens, ints(cu), c.sink.cuda())
    lse = lse.cpu()
    lse[1] += 300
    lse[2, ::2] = 30000.0
    mass = torch.zeros(2, 2, c.cols * c.page, device="cuda")
    binding.key_mass(q.cuda(), k, table, lens, ints(cu), lse.cuda(), mass)
    want = oracle_mass(q, c.k, c.table, c.lens, cu, lse, torch.zeros(mass.shape), scale=0.125)
    # scores of up to about 160: 20 times SCORE, and an lse's own rounding of 2^-24 * 500
    assert ((mass.double().cpu() - want).abs() <= 40 * SCORE * want + 1e-30).all()


@pytest.mark.parametrize("new", [[1, 1], [40, 70]])
def test_key_mass_lse_at_the_ends_of_fp32(new):
    """The largest lse gives no weight, the smallest an infinite one, NaN NaN."""
    for end, at in ((3.3e38, 1), (3.3e38, 0), (-3.3e38, 1), (math.nan, 2)):
        c, cu, q, lse = mass_case(90, new, [300, 513])
        lse[at, 0] = end                                      # of the first sequence, head 0
        k, _, table, lens = c.gpu()
        mass = torch.zeros(2, 2, c.cols * c.page, device="cuda")
        binding.key_mass(q.cuda(), k, table, lens, ints(cu), lse.cuda(), mass)
        want = oracle_mass(q, c.k, c.table, c.lens, cu, lse, torch.zeros(mass.shape), scale=0.125)
        got = mass.double().cpu()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        fine = torch.isfinite(want)
        assert ((got - want)[fine].abs() <= (2 * SCORE + 60 * 2 ** -24) * want[fine] + 1e-30).all()


def test_key_mass_nan_and_infinite_scores():
    """A NaN key has NaN weight; an infinite one infinite or no weight; others are as before."""
    for new in ([1, 1], [40, 70]):
        c, cu, q, lse = mass_case(88, new, [300, 513], hq=10, hkv=2)
        q[:, :, 3] = q[:, :, 3].abs() + 1
        c.k[int(c.table[0, 1]), 5, 0, 9] = math.nan
        c.k[int(c.table[0, 2]), 5, 0, 3] = -math.inf
        c.k[int(c.table[0, 3]), 5, 0, 3] = math.inf
        k, _, table, lens = c.gpu()
        mass = torch.zeros(2, 2, c.cols * c.page, device="cuda")
        binding.key_mass(q.cuda(), k, table, lens, ints(cu), lse.cuda(), mass)
        want = oracle_mass(q, c.k, c.table, c.lens, cu, lse, torch.zeros(mass.shape), scale=0.125)
        got = mass.double().cpu()
        assert torch.equal(got.isnan(), want.isnan()) and want.isnan().any()
        assert torch.equal(got.isinf(), want.isinf()) and want.isinf().any()
        fine = torch.isfinite(want)
        assert ((got - want)[fine].abs() <= (2 * SCORE + 60 * 2 ** -24) * want[fine] + 1e-30).all()


# ----------------------------------------------------------------------------- waits that run out
def device_error(L):
    code = ctypes.c_int(0)
    st = L.attn_sink_device_error(torch.cuda.current_stream().cuda_stream, ctypes.byref(code))
    return st, code.value


def test_waits_that_run_out():
    """In the test build a tile is withheld: each call comes back, the status says so, and the
    next calls are right."""
    L = binding.load_library(build(test=True))
    c, cu, prefix = shared_case(89, [(512, [700, 650, 600])], hq=16, hkv=2)
    k, v, table, lens = c.gpu()
    q, sink = c.q().cuda(), c.sink.cuda()
    new = ints([0, 40, 80, 120])
    rows = c.q(120).cuda()
    z = (3 + torch.rand(16, 120, generator=c.g)).cuda()
    sel = random_lists(c, 30).cuda()
    mass = torch.zeros(3, 2, c.cols * 16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(16, 3, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    P = ctypes.byref
    ps = binding.AttnSinkSharedParams(3, 1, 16, 2, 64, 16, c.pages, c.cols, 0.125)
    pp = binding.AttnSinkPagesParams(3, 16, 2, 64, 16, c.pages, c.cols, 30, 0.125)
    pm = binding.AttnSinkMassParams(3, 120, 16, 2, 64, 16, c.pages, c.cols, mass.shape[2], 0, 0.125)
    ws = torch.empty(max(L.attn_sink_decode_shared_workspace_size(P(ps)),
                         L.attn_sink_decode_pages_workspace_size(P(pp))), dtype=torch.uint8,
                     device="cuda")
    d = lambda *ts: [t.data_ptr() for t in ts]                # noqa: E731
    gs, pl = ints(cu), ints(prefix)
    calls = [
        lambda: L.attn_sink_decode_shared(P(ps), *d(q, k, v, table, lens, gs, pl, sink, out, lse, ws),
                                          ws.numel(), stream),
        lambda: L.attn_sink_decode_pages(P(pp), *d(q, k, v, table, lens, sel, sink, out, lse, ws),
                                         ws.numel(), stream),
        lambda: L.attn_sink_key_mass(P(pm), *d(rows, k, table, lens, new, z, mass), stream)]
    results = [(out, lse), (out, lse), (mass,)]
    # a slice of the list has one block a warp at least, the others two
    for call, res, tile in zip(calls, results, (1, 0, 1)):
        assert L.attn_sink_test_withhold(-1, -1) == 0
        assert call() == 0 and device_error(L) == (0, 0)
        want = [x.clone() for x in res]
        assert L.attn_sink_test_withhold(tile, -1) == 0
        t0 = time.perf_counter()
        assert call() == 0
        st, code = device_error(L)
        assert st == 5 and code & 0xF00 == 0x100, (st, hex(code))
        assert time.perf_counter() - t0 < 1.0
        assert L.attn_sink_test_withhold(-1, -1) == 0
        assert call() == 0 and device_error(L) == (0, 0)
        assert all(torch.equal(a, b) for a, b in zip(res, want))
