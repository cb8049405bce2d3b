"""extend where the table holds few keys (1280, or 2560 with many tiles): no tile is
cut, so up to 128 sequences (of tiles for a few rounds of CTAs) are one launch whose
CTAs find their tiles, and more have a schedule but no join.  A wider table with the same pages takes the general
way: tiles of four blocks of keys are not cut there either and give the same bits."""
import math

import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.step import oracle_extend
from test_gpu_step import BF, DEV, _check_extend, _clean, _code, _extend_case, _run_extend

pytestmark = pytest.mark.gpu


def _wide(c, page):
    """The same call with a table of more than 2560 keys."""
    more = torch.full((len(c[4]), 2560 // page + 1), -1, dtype=torch.int32)
    return (*c[:3], torch.cat([c[3], more], 1), *c[4:])


def _launches(run):
    n = binding.attn_sink_launch_count()
    r = run()
    return r, binding.attn_sink_launch_count() - n


CASES = [  # new, lens, page, hq, hkv, window
    ([1], [1], 16, 8, 1, 0),
    ([3, 0, 5, 1], [512, 7, 5, 0], 16, 8, 2, 0),
    ([130, 2, 64], [300, 2, 512], 1, 8, 8, 0),
    ([20, 11], [256, 129], 4, 10, 2, 40),
    ([17] * 32, [16 * i + 15 for i in range(32)], 16, 16, 2, 0),
    ([17] * 33, [min(512, 16 * i + 15) for i in range(33)], 16, 16, 2, 0),
    ([0] * 31 + [9], [0] * 31 + [9], 8, 8, 1, 0),
    ([2, 1] * 40, [400, 90] * 40, 32, 64, 8, 0),
    ([3, 0, 20] * 42 + [1, 17], [400, 5, 90] * 42 + [1, 512], 32, 16, 2, 0),
    ([3, 0, 20] * 43, [400, 5, 90] * 43, 32, 16, 2, 0),
    ([0] * 70 + [40] + [0] * 30, [3] * 70 + [500] + [0] * 30, 16, 8, 1, 0),
    ([5, 17, 1], [1280, 1153, 1025], 16, 8, 2, 0),
    ([1, 33], [1200, 1270], 8, 8, 1, 1000),
    ([256] * 8, [2400 + 20 * i for i in range(8)], 64, 8, 2, 0),
    ([10] * 50, [100 + 49 * i for i in range(50)], 16, 32, 4, 0),
    ([10] * 130, [100 + 18 * i for i in range(130)], 16, 4, 4, 0),
    ([300] * 8, [320 + 20 * i for i in range(8)], 32, 64, 8, 0),
    ([5, 3], [640, 600], 1, 8, 2, 0),
    ([5, 3], [640, 513], 20, 8, 2, 0),
]


@pytest.mark.parametrize("new,lens,page,hq,hkv,window", CASES)
def test_small_tables(new, lens, page, hq, hkv, window):
    c = _extend_case(page + len(new), new, lens, page, hq, hkv)
    got, n = _launches(lambda: _run_extend(c, window))
    general, m = _launches(lambda: _run_extend(_wide(c, page), window))
    # the windows here are narrow enough for whole tiles
    listed = len(new) > 128 or sum(new) >= 2400
    assert (n, m) == (2 if listed else 1, 1 if window else 3)
    if max(lens) <= 512:
        assert torch.equal(got[0], general[0]) and torch.equal(got[1], general[1])
    _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125,
                                     window=window), sum(new))
    _clean()


@pytest.mark.parametrize("page", [1, 2, 20])
def test_pages_copied_key_by_key(page):
    """Several blocks a tile and missing pages in the middle, at the ends of blocks
    and within them, where the copies' rings have come round."""
    new, lens = [33, 4, 70], [1400, 900, 333]
    c = _extend_case(page, new, lens, page, 16, 2, fill=0.0)
    got = _run_extend(c)
    _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125),
                  sum(new))
    _clean()
    holes = c[3].clone()
    for b, keys in enumerate([(5, 127, 128, 640, 1279), (0, 300, 700), (100,)]):
        for j in keys:
            holes[b, j // page] = -1
    got = _run_extend((*c[:3], holes, *c[4:]))
    assert _code() == 0x800
    _check_extend(got, oracle_extend(*c[:3], holes, c[4].tolist(), c[5].tolist(), c[6],
                                     scale=0.125), sum(new))


@pytest.mark.parametrize("wide", [False, True])
def test_bad_lists_of_sequences(wide):
    """Offsets that descend or lie outside q, lengths beyond the table: recorded,
    nothing outside the outputs is touched, and the next call is right."""
    c = _extend_case(3, [20, 30, 9], [100, 300, 9], 16, 8, 2, rows=64)
    c = _wide(c, 16) if wide else c
    for cu, lens in [([0, 20, 10, 59], [100, 300, 9]), ([0, 500, 600, 700], [100, 300, 9]),
                     ([-5, 20, 50, 59], [100, 300, 9]), ([0, 20, 50, 59], [100, 1 << 30, 9]),
                     ([0, 20, 50, 59], [-1, 300, 9]), ([0, 1 << 30, -(1 << 30), 59], [9, 9, 9])]:
        bad = (*c[:4], torch.tensor(lens, dtype=torch.int32), torch.tensor(cu, dtype=torch.int32),
               c[6])
        # the outputs lie in the middle of a larger buffer
        room = torch.full((3, 64, 8, 64), 7.0, dtype=BF, device=DEV)
        rest = torch.full((3, 8, 64), 7.0, device=DEV)
        _run_extend(bad, out=room[1], lse=rest[1])
        assert _code() == 0x800
        for x in (room, rest):
            assert (x[0] == 7).all() and (x[2] == 7).all()
    _check_extend(_run_extend(c), oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6],
                                                scale=0.125), 59)
    _clean()


def test_a_small_call_is_captured():
    c = [x.to(DEV) for x in _extend_case(9, [5, 1, 12], [90, 1, 300], 16, 8, 2)]
    want = binding.extend(*c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out, lse = binding.extend(*c)
    for shift in (0, 1):
        c[6].add_(shift)
        want = binding.extend(*c)
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    _clean()
