"""The size of the decode steps' error, which the bounds of test_gpu_cache.py (the worst
case of one rounding of P to bf16) do not see.

P enters O = P v as the sum of two bf16, at most 2^-16 off (of a shared prefix 2^-14: the
first bf16 is cut off, and the sum 2^-17 more than P), and values as they are; scores
are off by SCORE at most (test_gpu_cache.py), which a probability and the sum each feel.  So
before it is rounded an output is within (2^-14 + 2 SCORE) sum_j P_j |v_j| of the formula's,
and its rounding to bf16 adds 2^-8 of its size.  A single bf16 P would be off by up to 2^-8
of each term: where two keys have all the weight and opposite values, the terms cancel and
that error is left."""
import math

import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.cache import oracle_attend
from cache_cases import BF16, Paged
from test_gpu_cache import SCORE, all_keys, decode_shared, random_lists, shared_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert binding.attn_sink_device_error() == (0, 0)


def near(out, want, score=SCORE, p_step=2.0 ** -14):
    o, _, spread = want
    err = (out.double().cpu() - o).abs()
    allowed = 2.0 ** -8 * o.abs() + (p_step + 2 * score) * spread + 1e-30
    worst = (err / allowed).max().item()
    assert worst <= 1, worst


def norm(out, want):
    """The outputs' distance from the formula's, both rounded to bf16, as a part of their norm.
    Where they are off by a small part x of a step before the rounding, x of them end on
    another step: sqrt(x) 2^-8 in the mean square, or less where the value lies high in its
    binade.  P's own error is below 2^-14 / 2 in the mean square and that of the scores, whose
    worst case is SCORE, less: together below 2^-14, x = 2^-6, so 2^-11."""
    o = want[0].to(BF16).double()
    rel = ((out.double().cpu() - o).norm() / o.norm()).item()
    assert rel <= 2.0 ** -11, rel


def two_keys(c, at, q):
    """Two keys of every sequence that have all weight, about the same of it, and opposite
    values: the first two of the list at(b, h)."""
    for b in range(len(c.lens)):
        for h in range(c.hkv):
            for n, j in enumerate(list(at(b, h))[:2]):
                place = (int(c.table[b, j // c.page]), j % c.page, h)
                c.k[place] = 0
                c.k[place][0] = 512
                c.k[place][1 + n] = 4
                c.v[place] = (1 - 2 * n) * torch.linspace(1, 2, 64).to(BF16)
    q[:, :, 0] = 1
    q[:, :, 1:3] = (0.1 * torch.rand(len(c.lens), c.hq, 2, generator=c.g) - 0.05).to(BF16)
    return q


# Their scores: two products of at most 512.2 together, cut below 2^-23 of it and times 0.125,
# 2^-17; times log2(e) 92.4, rounded at 2^-18; the others are smaller by more than 50.
TWO = 2.0 ** -16


@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("groups,kw", [
    ([(128, [130, 200, 129])], dict(hq=16, hkv=2)),
    ([(1024, [1030, 1500, 1024, 1100]), (320, [400] * 9)], dict(hq=64, hkv=8)),
    ([(5000, [5001, 5030, 6000])], dict(hq=4, hkv=4)),
    ([(0, [90, 200, 300])], dict(hq=8, hkv=1)),
])
def test_shared_values_that_cancel(groups, kw, page):
    """The two keys are in the prefix, where there is one."""
    c, cu, prefix = shared_case(91, groups, page=page, **kw)
    q = two_keys(c, lambda b, h: [3, 40], c.q())
    out, _ = decode_shared(c, q, cu, prefix)
    near(out, oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125),
         score=TWO)


@pytest.mark.parametrize("page", [16, 24])
def test_pages_values_that_cancel(page):
    c = Paged(92, [700, 640, 333], hq=16, hkv=2, page=page)
    sel = random_lists(c, 9)
    q = two_keys(c, lambda b, h: [int(sel[b, h, 0]) * page + 1, int(sel[b, h, 5]) * page + 7], c.q())
    k, v, table, lens = c.gpu()
    out, _ = binding.decode_pages(q.cuda(), k, v, table, lens, sel.cuda(), c.sink.cuda())
    keys = lambda b, h: [j for x in sel[b, h].tolist() if x >= 0       # noqa: E731
                         for j in range(x * page, min(c.lens[b], (x + 1) * page))]
    near(out, oracle_attend(q, c.k, c.v, c.table, keys, c.sink, scale=0.125),
         score=TWO, p_step=2.0 ** -16)


@pytest.mark.parametrize("groups,kw", [
    ([(1024, [1030, 1500, 1024, 1100, 1025]), (320, [400] * 9)], dict(hq=64, hkv=8)),
    ([(2048, [2050] * 40)], dict(hq=8, hkv=1, page=64)),
    ([(777, [800] * 20)], dict(hq=16, hkv=2, page=24)),
])
def test_shared_norm(groups, kw):
    c, cu, prefix = shared_case(93, groups, **kw)
    q = c.q()
    out, _ = decode_shared(c, q, cu, prefix)
    want = oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125)
    near(out, want)
    norm(out, want)


def test_pages_norm():
    c = Paged(94, [9000, 4097], hq=64, hkv=8)
    q, sel = c.q(), random_lists(c, 100)
    k, v, table, lens = c.gpu()
    out, _ = binding.decode_pages(q.cuda(), k, v, table, lens, sel.cuda(), c.sink.cuda())
    keys = lambda b, h: [j for x in sel[b, h].tolist() if x >= 0       # noqa: E731
                         for j in range(x * 16, min(c.lens[b], (x + 1) * 16))]
    want = oracle_attend(q, c.k, c.v, c.table, keys, c.sink, scale=0.125)
    near(out, want)
    norm(out, want)


def infinite(out, lse, want, rows, heads):
    """Dimension 3 infinite, 9 minus infinite and 20 NaN in these rows and heads, nothing else."""
    o, z, spread = want
    out, fine = out.double().cpu(), torch.isfinite(o)
    assert (out[rows, heads, 3] == math.inf).all() and (out[rows, heads, 9] == -math.inf).all()
    assert out[rows, heads, 20].isnan().all()
    assert (~fine).sum() == 3 * out[rows, heads, 0].numel() and not lse.isnan().any()
    near(torch.where(fine, out, 0.0), (torch.where(fine, o, 0.0), z, torch.where(fine, spread, 0.0)))


def put_infinite(c, b, h, keys):
    for j, d, x in zip(keys, (3, 9, 20, 20), (math.inf, -math.inf, math.inf, -math.inf)):
        c.v[int(c.table[b, j // c.page]), j % c.page, h, d] = x


def test_shared_infinite_values():
    """An infinite value of the prefix makes the outputs of its dimension infinite, two of
    opposite signs NaN, and no other."""
    c, cu, prefix = shared_case(95, [(320, [330, 400, 325]), (200, [200, 230])], hq=16, hkv=2)
    q = c.q()
    put_infinite(c, 0, 1, [5, 130, 7, 300])
    out, lse = decode_shared(c, q, cu, prefix)
    infinite(out, lse, oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125),
             slice(0, 3), slice(8, 16))


@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("cols", [30, 600])                   # a slice, several joined
def test_infinite_values_of_own_keys(page, cols):
    c = Paged(96, [400, 333, 290], hq=16, hkv=2, page=page, cols=cols)
    q = c.q()
    put_infinite(c, 1, 0, [5, 130, 7, 300])
    want = oracle_attend(q, c.k, c.v, c.table, all_keys(c), c.sink, scale=0.125)
    out, lse = decode_shared(c, q, [0, 1, 2, 3], [0, 0, 0])
    infinite(out, lse, want, slice(1, 2), slice(0, 8))
    k, v, table, lens = c.gpu()
    sel = torch.arange(cols, dtype=torch.int32).expand(3, 2, cols).contiguous()
    have = torch.tensor([-(-n // page) for n in c.lens])[:, None, None]
    sel = torch.where(sel < have, sel, -1).cuda()
    out, lse = binding.decode_pages(q.cuda(), k, v, table, lens, sel, c.sink.cuda())
    infinite(out, lse, want, slice(1, 2), slice(0, 8))
