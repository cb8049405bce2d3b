"""attn_sink_cache.h on the GPU against the float64 definitions.

Tolerances.  A bf16 output is off by half a step, 2^-9 of its power of two, at most 2^-8
of its size.  In O = P v the own keys' probabilities and values enter as fp16 (2^-11
each), a shared prefix's probabilities as bf16 (2^-8): times sum_j P_j |v_j|.  Scores are
fp32 sums of 64 exact products: an error of 64 * 2^-24 * sum |q_d k_d| * scale, below
64 * 2^-24 * 64 * 0.125 * 2 = 6e-5 for unit normal numbers (|q_d k_d| averages 0.64, and
twice that covers every row), as relative error of a probability and absolute one of lse."""
import math

import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.cache import (oracle_attend, oracle_bounds, oracle_evict, oracle_mass, oracle_select)
from cache_cases import BF16, Paged, ints

pytestmark = pytest.mark.gpu

SCORE = 6e-5


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert binding.attn_sink_device_error() == (0, 0)


def check(out, lse, want, *, p_step=2 ** -11):
    o, z, spread = want
    err = (out.double().cpu() - o).abs()
    allowed = 2 ** -8 * o.abs() + (p_step + 2 ** -11 + 2 * SCORE) * spread + 1e-30
    worst = (err / allowed).max().item() if err.numel() else 0.0
    assert worst <= 1, worst
    zerr = (lse.double().cpu() - z).abs()
    zerr = torch.where(z == lse.double().cpu(), 0.0, zerr)            # infinities
    assert (zerr <= SCORE + 2 ** -22 * z.abs()).all(), zerr.max()


def recorded():
    return binding.attn_sink_device_error()


# ----------------------------------------------------------------------------- shared prefixes
def shared_case(seed, groups, *, page=16, **kw):
    """groups: [(prefix, [lengths])]; every sequence of a group holds the prefix's keys, through
    the same pages where they are full, a copy of its own where one is not."""
    lens = [n for _, ls in groups for n in ls]
    c = Paged(seed, lens, page=page, **kw)
    at = 0
    for prefix, ls in groups:
        for i, n in enumerate(ls):
            same = min(prefix, n, *(ls[:1]))
            for j in range(same):
                if j % page == 0 and j + page <= same:
                    c.table[at + i, j // page] = c.table[at, j // page]
                src = (int(c.table[at, j // page]), j % page)
                dst = (int(c.table[at + i, j // page]), j % page)
                c.k[dst], c.v[dst] = c.k[src].clone(), c.v[src].clone()
        at += len(ls)
    cu, total = [0], 0
    for _, ls in groups:
        total += len(ls)
        cu.append(total)
    return c, cu, [p for p, _ in groups]


def decode_shared(c, q, cu, prefix, **kw):
    k, v, table, lens = c.gpu()
    return binding.decode_shared(q.cuda(), k, v, table, lens, ints(cu), ints(prefix),
                                 c.sink.cuda(), **kw)


def all_keys(c):
    return lambda b, h: range(c.lens[b])


@pytest.mark.parametrize("groups,kw", [
    ([(128, [130, 200, 129])], {}),
    ([(64, [65] * 17)], dict(hq=16, hkv=2)),
    ([(1024, [1030, 1500, 1024, 1100, 1025]), (320, [400] * 9), (100, [120])],
     dict(hq=64, hkv=8)),
    ([(512, [600, 700]), (0, [5, 300]), (256, [256, 257, 258])], dict(hq=4, hkv=4, page=64)),
    ([(200, [230, 201, 500])], dict(page=24)),               # copies key by key where pages are odd
    ([(77, [100, 78, 90, 1000])], dict(page=1)),
    ([(333, [400, 350, 340])], dict(page=128)),              # the prefix ends inside a page
    ([(256, [300, 200, 290])], dict(page=16)),               # a sequence shorter than the prefix
    ([(256, [300, 0, 290])], dict(page=16)),                 # and one without keys
    ([(5000, [5001] * 33)], dict(hq=8, hkv=1, page=8)),
    ([(640, [700] * 130)], dict(hq=1, hkv=1)),               # more than a tile of one head
    ([(70, [71] * 3)] * 40, dict(hq=2, hkv=1)),              # more groups than the plan has warps
    ([(64, [65, 66])] * 1100, dict(hq=1, hkv=1, page=64)),   # more than it keeps at hand
    ([(64, [1]), (10 ** 9, [2, 2])], {}),
])
def test_decode_shared(groups, kw):
    c, cu, prefix = shared_case(11, groups, **kw)
    q = c.q()
    out, lse = decode_shared(c, q, cu, prefix)
    check(out, lse, oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125),
          p_step=2 ** -8)


def test_decode_shared_is_decode():
    c, cu, prefix = shared_case(12, [(512, [600, 700, 513, 900])], hq=16, hkv=2)
    q = c.q()
    k, v, table, lens = c.gpu()
    out, lse = decode_shared(c, q, cu, prefix, softmax_scale=0.3)
    one, z, _ = binding.decode(q.cuda(), k, v, table, lens, c.sink.cuda(), softmax_scale=0.3)
    assert (lse - z).abs().max() < 4 * SCORE * 0.3 / 0.125
    assert (out.float() - one.float()).abs().max() < 2 ** -6


@pytest.mark.parametrize("sink", [math.inf, -math.inf, 100.0])
def test_decode_shared_sinks(sink):
    c, cu, prefix = shared_case(13, [(128, [140, 200]), (0, [0, 3])])
    c.sink[:4] = sink
    q = c.q()
    out, lse = decode_shared(c, q, cu, prefix)
    o, z, spread = oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125)
    check(out, lse, (torch.where(o.isnan(), 0.0, o), z, torch.where(spread.isnan(), 0.0, spread)),
          p_step=2 ** -8)


def test_decode_shared_large_scores():
    """Scores of several hundred: the softmax is relative to the largest, over both parts."""
    c, cu, prefix = shared_case(14, [(256, [300, 400, 270])])
    c.k *= 30
    q = c.q()
    out, lse = decode_shared(c, q, cu, prefix)
    o, z, spread = oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125)
    grown = 30 * SCORE                                        # of the scores' errors
    assert ((out.double().cpu() - o).abs() <= 2 ** -8 * o.abs() + (2 ** -7 + 2 * grown) * spread).all()
    assert ((lse.double().cpu() - z).abs() <= grown + 2 ** -22 * z.abs()).all()


@pytest.mark.parametrize("cu", [[0, 2, 1, 4], [0, 9, 4, 4], [-1, 2, 3, 4], [1, 2, 3, 4], [0, 1, 2, 3],
                                [0, 4, 0, 4]])
def test_decode_shared_bad_groups(cu):
    c, _, _ = shared_case(15, [(128, [140, 200, 150, 129])])
    out, lse = decode_shared(c, c.q(), cu, [128, 128, 128])
    assert recorded() == (0, 0x800)
    assert out.shape == (4, 8, 64)


def test_decode_shared_bad_pages_and_lengths():
    """A missing prefix page is missing for all, an own one for its sequence; lengths are clamped."""
    c, cu, prefix = shared_case(16, [(128, [140, 200, 150])])
    c.table[:, 2] = -1
    c.table[1, 10] = c.pages
    q = c.q()
    out, lse = decode_shared(c, q, cu, prefix)
    check(out, lse, oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125),
          p_step=2 ** -8)
    assert recorded() == (0, 0x800)
    c.lens[0] = -5
    decode_shared(c, q, cu, [-3])
    assert recorded() == (0, 0x800)


def test_decode_shared_nan_reaches_its_rows():
    c, cu, prefix = shared_case(17, [(128, [140, 200]), (0, [9, 9])])
    c.k[int(c.table[0, 1]), 3, 0, 5] = math.nan               # of the prefix, kv head 0
    c.k[int(c.table[2, 0]), 3, 1, 5] = math.nan               # of sequence 2 alone, kv head 1
    out, lse = decode_shared(c, c.q(), cu, prefix)
    bad = lse.isnan().cpu()
    want = torch.zeros(8, 4, dtype=torch.bool)
    want[:4, :2], want[4:, 2] = True, True
    assert torch.equal(bad, want)


# ----------------------------------------------------------------------------- bounds
@pytest.mark.parametrize("page", [1, 8, 16, 24, 100])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_page_bounds(page, hkv):
    lens = [300, 1, 0, 77, 128]
    cached = [0, 0, 0, 70, 128]
    c = Paged(21, lens, hkv=hkv, hq=hkv, page=page)
    old = torch.randn(c.pages, hkv, 2, 64, generator=c.g).to(BF16)
    bounds = old.cuda()
    k, _, table, n = c.gpu()
    binding.page_bounds(k, table, ints(cached), n, bounds)
    assert torch.equal(bounds.cpu(), oracle_bounds(c.k, c.table, cached, lens, old))


def test_page_bounds_nan_bad_pages_and_lengths():
    c = Paged(22, [40, 40, 20])
    c.k[int(c.table[0, 1]), 3, 0, 7] = math.nan
    c.table[1, 0] = c.pages
    old = torch.zeros(c.pages, 2, 2, 64, dtype=BF16)
    bounds = old.cuda()
    k, _, table, _ = c.gpu()
    binding.page_bounds(k, table, ints([0, -4, 50]), ints([40, 40, 20]), bounds)
    want = oracle_bounds(c.k, c.table, [0, 0, 20], c.lens, old)
    assert torch.equal(bounds.cpu().isnan(), want.isnan()) and want.isnan().any()
    assert torch.equal(bounds.cpu().nan_to_num(), want.nan_to_num())
    assert recorded() == (0, 0x800)


def test_page_bounds_of_many_sequences():
    lens = [1 + b % 19 for b in range(3000)]
    c = Paged(23, lens, hkv=1, hq=1, page=8)
    bounds = torch.zeros(c.pages, 1, 2, 64, dtype=BF16, device="cuda")
    k, _, table, n = c.gpu()
    binding.page_bounds(k, table, ints([0] * 3000), n, bounds)
    want = oracle_bounds(c.k, c.table, [0] * 3000, lens, torch.zeros(c.pages, 1, 2, 64, dtype=BF16))
    assert torch.equal(bounds.cpu(), want)


# ----------------------------------------------------------------------------- selection
def random_bounds(c, spread=1.0):
    a = torch.randn(c.pages, c.hkv, 2, 64, generator=c.g) * spread
    return a.sort(2).values.to(BF16)


def select(c, q, bounds, count, first=1, last=1, lens=None):
    return binding.select_pages(q.cuda(), bounds.cuda(), c.table.cuda(), ints(lens or c.lens),
                                count=count, page_size=c.page, keep_first=first, keep_last=last)


def select_both(c, q, bounds, count, first=1, last=1):
    got = select(c, q, bounds, count, first, last).cpu()
    want = oracle_select(q, bounds, c.table, c.lens, page=c.page, count=count, first=first,
                         last=last)
    assert torch.equal(got, want)


@pytest.mark.parametrize("lens,kw,count,first,last", [
    ([500, 20, 0, 301], {}, 6, 1, 1),
    ([500, 20, 0, 301], dict(hq=2, hkv=2), 5, 0, 0),
    ([700, 999], dict(hq=16, hkv=4, page=1), 100, 3, 5),
    ([700, 999], dict(hq=24, hkv=3, page=8), 60, 0, 10),
    ([5000], dict(hq=2, hkv=1, page=1), 777, 1, 1),          # more pages than a CTA's words
    ([300] * 40, dict(page=16), 4, 2, 2),                    # nothing left to choose
    ([300] * 3, dict(page=16), 18, 1, 1),                    # all but one
    ([300] * 3, dict(page=16), 100, 1, 1),                   # all
    ([300] * 3, dict(page=16), 1, 0, 0),
])
def test_select_pages(lens, kw, count, first, last):
    c = Paged(31, lens, **kw)
    select_both(c, c.q(), random_bounds(c), count, first, last)


def test_select_pages_long_rows():
    """A row that does not fit shared memory, against the definition on all pages at once."""
    c = Paged(32, [20011, 13000], hq=8, hkv=1, page=1)
    select_both(c, c.q(), random_bounds(c), 4000, 1, 1)
    c = Paged(37, [40000], hq=1, hkv=1, page=1)               # more than a bitmap's pages, too
    select_both(c, c.q(), random_bounds(c), 9000, 1, 1)
    b = random_bounds(c)[:3].repeat(c.pages // 3 + 1, 1, 1, 1)[:c.pages].contiguous()
    select_both(c, c.q(), b, 9000, 1, 1)


@pytest.mark.parametrize("page", [1, 16])
def test_select_pages_ties(page):
    """Equal scores go to the lower column: pages alike, pages given twice, queries of zero."""
    c = Paged(33, [640 * page, 300 * page], page=page)
    q, b = c.q(), random_bounds(c)
    select_both(c, torch.zeros_like(q), b, 40)
    select_both(c, q, b[:1].expand_as(b).contiguous(), 40)
    c.table[:, 50:] = torch.where(c.table[:, 50:] >= 0, c.table[:, :1], -1)
    select_both(c, q, b, 40)
    two = torch.where(torch.arange(c.pages)[:, None, None, None] % 2 == 0, b[:1], b[1:2])
    select_both(c, q, two.contiguous(), 400)


def test_select_pages_close_scores():
    """Scores that 32 bits do not tell apart: a bound changed by one step of a dimension whose
    query is tiny."""
    c = Paged(34, [400 * 16], hq=2, hkv=1)
    q = c.q(scale=4)
    q[:, :, 9] = torch.tensor(2.0 ** -20).to(BF16)
    b = random_bounds(c)[:1].expand(c.pages, -1, -1, -1).contiguous().clone()
    b[:, :, 1, 9] = (1 + torch.randint(0, 100, (c.pages, 1), generator=c.g) / 128).to(BF16)
    for count in (3, 40, 200, 399):
        select_both(c, q, b, count)


def test_select_pages_infinities_and_missing_pages():
    c = Paged(35, [640, 640])
    b = random_bounds(c)
    b[int(c.table[0, 9]), :, 1, 3] = math.inf
    b[int(c.table[1, 12]), :, 0, 3] = math.nan
    q = c.q()
    q[:, :, 3] = 1
    select_both(c, q, b, 4)
    b = random_bounds(c, 1e30)                                # beyond fp32 for many
    select_both(c, c.q(scale=1e10), b, 7)
    c.table[0, 5:30] = c.pages
    b = random_bounds(c)
    select_both(c, q, b, 30)
    assert recorded() == (0, 0x800)


def test_select_pages_lengths_are_clamped():
    c = Paged(36, [640, 640])
    got = select(c, c.q(), random_bounds(c), 8, lens=[-3, 10 ** 6])
    assert recorded() == (0, 0x800)
    assert (got[0] == -1).all() and (got[1] >= 0).all() and (got[1] < c.cols).all()


# ----------------------------------------------------------------------------- selected pages
def pages_both(c, sel, **kw):
    q = c.q()
    k, v, table, lens = c.gpu()
    out, lse = binding.decode_pages(q.cuda(), k, v, table, lens, sel.cuda(), c.sink.cuda(), **kw)

    def keys(b, h):
        have = -(-c.lens[b] // c.page)
        cols = [int(x) for x in sel[b, h, :have] if 0 <= x < have]
        return [j for x in cols for j in range(x * c.page, min(c.lens[b], (x + 1) * c.page))]

    check(out, lse, oracle_attend(q, c.k, c.v, c.table, keys, c.sink, scale=0.125))


def random_lists(c, count):
    sel = torch.full((len(c.lens), c.hkv, count), -1, dtype=torch.int32)
    for b, n in enumerate(c.lens):
        have = -(-n // c.page)
        for h in range(c.hkv):
            some = torch.randperm(have, generator=c.g)[:count].to(torch.int32)
            sel[b, h, :some.numel()] = some
    return sel


@pytest.mark.parametrize("page", [1, 8, 16, 24, 64, 128, 256])
@pytest.mark.parametrize("heads", [(8, 8), (4, 2), (8, 2), (16, 2)])
def test_decode_pages(page, heads):
    lens = [20 * page + 3, page, 1, 0, 7 * page - 1, 33 * page]
    c = Paged(41, lens, hq=heads[0], hkv=heads[1], page=page)
    pages_both(c, random_lists(c, 9))


def test_decode_pages_of_a_long_list():
    c = Paged(42, [9000, 4097], hq=64, hkv=8)
    pages_both(c, random_lists(c, 300))


def test_decode_pages_holes_in_the_list():
    c = Paged(43, [640, 333])
    sel = random_lists(c, 20)
    sel[:, :, ::3] = -1
    sel[0, 0, 1] = -7
    pages_both(c, sel)
    pages_both(c, torch.full_like(sel, -1))
    pages_both(c, sel[:, :, :0].contiguous())


def test_decode_pages_bad_columns_pages_and_lengths():
    c = Paged(44, [640, 333], hq=8, hkv=1)
    sel = random_lists(c, 20)
    sel[0, 0, 3] = 40
    sel[1, 0, 4] = 2 ** 31 - 1
    pages_both(c, sel)
    assert recorded() == (0, 0x800)
    sel = random_lists(c, 20)
    c.table[0, 7] = c.pages
    pages_both(c, sel)
    assert recorded() == (0, 0x800)
    for page in (24,):
        c = Paged(45, [640, 333], page=page)
        sel = random_lists(c, 10)
        sel[0, 0, 3] = 2 ** 31 - 1
        pages_both(c, sel)
        assert recorded() == (0, 0x800)


def test_decode_pages_all_is_decode():
    c = Paged(46, [640, 333, 1000], hq=64, hkv=8)
    q = c.q()
    k, v, table, lens = c.gpu()
    sel = torch.arange(63, dtype=torch.int32).expand(3, 8, 63)
    have = torch.tensor([-(-n // 16) for n in c.lens])[:, None, None]
    sel = torch.where(sel < have, sel, -1).contiguous().cuda()
    out, lse = binding.decode_pages(q.cuda(), k, v, table, lens, sel, c.sink.cuda())
    one, z, _ = binding.decode(q.cuda(), k, v, table, lens, c.sink.cuda())
    assert (lse - z).abs().max() < 2 * SCORE
    assert (out.float() - one.float()).abs().max() < 2 ** -6


# ----------------------------------------------------------------------------- weights of keys
def mass_case(seed, new, lens, **kw):
    c = Paged(seed, lens, **kw)
    cu = torch.tensor([0] + list(new)).cumsum(0).tolist()
    q = c.q(cu[-1])
    lse = 3 + torch.rand(c.hq, cu[-1], generator=c.g)
    return c, cu, q, lse


def mass_both(c, cu, q, lse, keys=None, accumulate=True, tail=3):
    keys = c.cols * c.page if keys is None else keys
    mass = torch.rand(len(c.lens), c.hkv, keys, generator=c.g)
    if accumulate:
        start = mass
    else:
        start = torch.zeros_like(mass)
        mass = mass + math.nan
    want = oracle_mass(q, c.k, c.table, c.lens, cu, lse, start, scale=0.125)
    k, _, table, lens = c.gpu()
    pad = torch.full((tail, c.hq, 64), math.nan).to(BF16)     # rows behind the last token
    qq, zz = torch.cat([q, pad]).cuda(), torch.cat([lse, torch.full((c.hq, tail), math.nan)], 1)
    got = binding.key_mass(qq, k, table, lens, ints(cu), zz.cuda(), mass.cuda(),
                           accumulate=accumulate).double().cpu()
    # each weight to SCORE, and up to rows / 8 additions of a thread, its lanes' and the old value
    rows = max([cu[i + 1] - cu[i] for i in range(len(cu) - 1)], default=0) * (c.hq // c.hkv)
    allowed = (2 * SCORE + (rows / 8 + 16) * 2 ** -24) * want + 1e-30
    assert ((got - want).abs() <= allowed).all(), ((got - want).abs() / allowed).max()


@pytest.mark.parametrize("new,lens,kw", [
    ([1, 1, 1], [300, 1, 513], dict(hq=16, hkv=2)),
    ([1, 1, 0], [300, 1, 513], dict(hq=2, hkv=2, page=24)),
    ([5, 0, 17], [300, 0, 17], dict(hq=8, hkv=2, page=1)),
    ([130, 7, 64], [300, 400, 1000], dict(hq=8, hkv=1)),
    ([33, 300], [290, 301], dict(hq=15, hkv=3, page=64)),      # more tokens than keys
    ([9], [1030], dict(hq=128, hkv=1, page=8)),
    ([3, 2], [257, 256], dict(hq=5, hkv=5, page=128)),
    ([70], [2000], dict(hq=64, hkv=8)),
])
@pytest.mark.parametrize("accumulate", [True, False])
def test_key_mass(new, lens, kw, accumulate):
    mass_both(*mass_case(51, new, lens, **kw), accumulate=accumulate)


def test_key_mass_rows_without_weight_and_missing_pages():
    c, cu, q, lse = mass_case(52, [4, 9], [300, 280])
    lse[:, 1], lse[3] = math.inf, -math.inf
    mass_both(c, cu, q, lse)
    c.table[0, 3] = c.pages
    mass_both(c, cu, q, lse)
    assert recorded() == (0, 0x800)


def test_key_mass_short_rows_and_bad_lengths():
    c, cu, q, lse = mass_case(53, [4, 9], [300, 280])
    mass_both(c, cu, q, lse, keys=290)
    assert recorded() == (0, 0x800)
    mass_both(c, cu, q, lse, keys=0)
    k, _, table, _ = c.gpu()
    mass = torch.zeros(2, 2, 400, device="cuda")
    binding.key_mass(q.cuda(), k, table, ints([-1, 10 ** 6]), ints([0, 4, 99]), lse.cuda(), mass)
    assert recorded() == (0, 0x800)
    assert (mass[0] == 0).all()


def test_key_mass_sums_to_the_tokens():
    """What extend gives away to the keys and to the sink is each row's whole weight."""
    c, cu, q, _ = mass_case(54, [40, 3], [200, 90], hq=8, hkv=2)
    k, v, table, lens = c.gpu()
    sink = c.sink.cuda()
    _, lse = binding.extend(q.cuda(), k, v, table, lens, ints(cu), sink)
    mass = torch.zeros(2, 2, 224, device="cuda")
    binding.key_mass(q.cuda(), k, table, lens, ints(cu), lse, mass)
    away = torch.exp(sink[:, None] - lse).double()            # [H_q, T]
    for b in range(2):
        t = slice(cu[b], cu[b + 1])
        want = (cu[b + 1] - cu[b]) * 4 - away[:, t].view(2, 4, -1).sum((1, 2))
        assert ((mass[b].double().sum(1) - want).abs() <= 4 * SCORE * want).all()


# ----------------------------------------------------------------------------- eviction
def evict_both(c, mass, budget, first=0, last=0):
    k, v, table, lens = c.gpu()
    r = binding.evict(k, v, table, lens, mass.cuda(), budget=budget, keep_first=first,
                      keep_last=last)
    wk, wv, wm, wl, wf = oracle_evict(c.k, c.v, c.table, c.lens, mass, budget=budget, first=first,
                                      last=last)
    as_bits = lambda x: x.cpu().contiguous().view(torch.int16)   # noqa: E731  (NaN in unused rows)
    assert torch.equal(as_bits(k), as_bits(wk)) and torch.equal(as_bits(v), as_bits(wv))
    assert torch.equal(r.mass.cpu().view(torch.int32), wm.view(torch.int32))
    assert r.seq_lens.tolist() == wl and r.num_freed.item() == len(wf)
    freed = r.freed_pages.tolist()
    assert freed[:len(wf)] == wf and all(x == -1 for x in freed[len(wf):])


def random_mass(c, keys=None):
    return torch.rand(len(c.lens), c.hkv, c.cols * c.page if keys is None else keys, generator=c.g)


@pytest.mark.parametrize("lens,kw,budget,first,last", [
    ([300, 20, 0, 301], {}, 100, 4, 32),
    ([300, 20, 0, 301], dict(page=1, hkv=3, hq=3), 36, 4, 32),     # nothing left to choose
    ([300, 20, 100, 101], dict(page=24), 100, 0, 0),
    ([300, 290], dict(page=64), 0, 0, 0),                          # everything goes
    ([5000, 7, 6000, 30], dict(page=1, hkv=1, hq=1), 20, 1, 1),    # many pages of few sequences
    ([300, 290], dict(page=64), 1, 0, 0),
    ([300, 290], dict(page=64), 299, 0, 1),
    ([300, 290], {}, 1000, 4, 4),                                  # nothing does
    ([9000, 4000], dict(page=128, hkv=1, hq=1), 3001, 4, 32),      # rows of several words a thread
    ([40 + b % 30 for b in range(400)], dict(hkv=1, hq=1, page=8), 50, 1, 3),
])
def test_evict(lens, kw, budget, first, last):
    c = Paged(61, lens, **kw)
    evict_both(c, random_mass(c), budget, first, last)


def test_evict_long_rows():
    """A row of weights that does not fit shared memory."""
    c = Paged(62, [50001], hq=1, hkv=1, page=128)
    evict_both(c, random_mass(c), 20000, 4, 32)


@pytest.mark.parametrize("budget", [7, 100, 290])
def test_evict_equal_weights(budget):
    c = Paged(63, [300, 290])
    evict_both(c, torch.zeros(2, 2, c.cols * 16), budget)
    few = torch.randint(0, 3, (2, 2, c.cols * 16), generator=c.g).float()
    evict_both(c, few, budget, 1, 2)


def test_evict_odd_weights():
    c = Paged(64, [300, 290])
    m = random_mass(c) - 0.5
    m[0, 0, 7], m[0, 1, 200], m[1, 0, 3], m[1, 1, :200] = math.nan, math.nan, math.inf, -math.inf
    m[1, 1, 5] = -0.0
    evict_both(c, m, 100, 1, 1)


def test_evict_missing_pages_and_lengths():
    c = Paged(65, [300, 290])
    c.table[0, 1], c.table[1, 17] = c.pages, -1
    evict_both(c, random_mass(c), 100)
    assert recorded() == (0, 0x800)
    k, v, table, _ = c.gpu()
    r = binding.evict(k, v, table, ints([-1, 10 ** 6]), random_mass(c, 200).cuda(), budget=50)
    assert recorded() == (0, 0x800)
    assert r.seq_lens.tolist() == [0, 50] and r.num_freed.item() == 13 - 4


def test_evict_without_sequences():
    c = Paged(66, [])
    k, v = c.k.cuda(), c.v.cuda()
    r = binding.evict(k, v, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), ints([]),
                      torch.zeros(0, 2, 48, device="cuda"), budget=5)
    assert r.num_freed.item() == 0 and r.seq_lens.numel() == 0
