"""GPU parity of windowed attn_sink_extend calls, of few tiles (the general kernel)
and of many, whose keys are gathered for the band kernel.  Tolerances: P and the values are
fp16 there (2^-11 each) and the output bf16 (2^-8), so those of the general
kernel hold with room; the values' fp16 conversion is exact for bf16 numbers in
the fp16 normal range, and below it off by 2^-25 at most."""
import math

import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.step import oracle_extend
from test_gpu_step import BF, DEV, _check_extend, _clean, _code, _extend_case, _run_extend

pytestmark = pytest.mark.gpu

CASES = [  # name, new, lens, page, hq, hkv, window
    ("g8", [200, 65, 70], [900, 65, 4000], 16, 16, 2, 128),
    ("g1_w1", [300], [300], 8, 2, 2, 1),
    ("g4_page1", [64, 130], [500, 130], 1, 8, 2, 60),
    ("g2_page24", [129, 64, 63], [129, 1000, 70], 24, 4, 2, 100),
    ("g8_uneven", [700, 0, 5, 1], [3000, 50, 5, 0], 64, 8, 1, 129),
    ("more_new_than_keys", [150, 64], [20, 0], 16, 8, 1, 33),
    ("g128", [70], [200], 16, 128, 1, 176),
    ("g16_many", [64] * 40, list(range(64, 2064, 50)), 16, 32, 2, 17),
]


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("name,new,lens,page,hq,hkv,window", CASES, ids=[c[0] for c in CASES])
def test_windowed_chunks(name, new, lens, page, hq, hkv, window, many):
    if many:                               # more than 128 sequences
        n = 12 if hq // hkv > 2 else 130
        new, lens = new + [n] * 130, lens + [n + i * i % 1000 for i in range(130)]
    c = _extend_case(len(name) + page, new, lens, page, hq, hkv)
    got = _run_extend(c, window)
    _clean()
    _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125,
                                     window=window), sum(new))
    again = _run_extend(c, window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_both_ways_agree():
    """The same tokens as one call of many and as calls of few tokens a sequence."""
    c = _extend_case(3, [96], [1000], 16, 8, 2)
    whole = _run_extend(c, 100)
    q, kc, vc, table, _, _, sink = (x.to(DEV) for x in c)
    for at in range(0, 96, 32):
        cu = torch.tensor([0, 32], dtype=torch.int32, device=DEV)
        # padded with sequences of no tokens, so that few are new on average
        cu = torch.cat([cu, cu[-1:].expand(7)])
        lens = torch.tensor([904 + at + 32] + [0] * 7, dtype=torch.int32, device=DEV)
        out, lse = binding.extend(q[at:at + 32], kc, vc, table.expand(8, -1).contiguous(), lens, cu,
                                  sink, window=100)
        assert (out.double() - whole[0][at:at + 32].double()).abs().max() <= 2.0 ** -5
        assert (lse - whole[1][:, at:at + 32]).abs().max() <= 2.0 ** -12
    _clean()


@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("more", [0, 130])
def test_evicted_pages_and_rows_behind(page, more):
    c = _extend_case(6, [70, 130] + [9] * more, [900, 400] + [400] * more, page, 8, 2, rows=1536,
                     evict=130 + 64)
    out = torch.full((1536, 8, 64), 7.0, dtype=BF, device=DEV)
    lse = torch.full((8, 1536), 7.0, device=DEV)
    got = _run_extend(c, 64, out=out, lse=lse)
    _clean()
    n = 200 + 9 * more
    _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125,
                                     window=64), n)
    assert (out[n:] == 7).all() and (lse[:, n:] == 7).all()


@pytest.mark.parametrize("more", [0, 130])
def test_a_sequence_of_nan_keeps_to_itself(more):
    c = _extend_case(9, [70, 70, 70] + [9] * more, [300, 300, 300] + [9] * more, 16, 8, 2)
    held = c[3][1][c[3][1] >= 0].long()
    c[1][held], c[2][held] = math.nan, math.nan
    got = _run_extend(c, 100)
    ref = oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125, window=100)
    for a in (0, 140):
        part = (got[0][a:a + 70], got[1][:, a:a + 70])
        _check_extend(part, tuple(x[:, a:a + 70] if i == 1 else x[a:a + 70]
                                  for i, x in enumerate(ref)), 70)
    torch.cuda.synchronize()
    binding.attn_sink_device_error()          # NaN values lie outside the fp16 range


def test_inputs_out_of_range_are_reported():
    c = list(_extend_case(8, [70, 100] + [12] * 130, [200, 190] + [12] * 130, 16, 8, 2, fill=0.0))
    cu = c[5]
    good = c[3].clone()
    c[3] = good.clone()
    c[3][0, 12] = c[1].shape[0] + 5
    _run_extend(c, 100)
    assert _code() == 0x800
    c[3] = good
    c[2][int(good[1, 11])] = 1e6
    _run_extend(c, 100)
    assert _code() == 0x400
    for at, bad in ((2, 4000), (1, 300), (0, -4)):
        c[5] = cu.clone()
        c[5][at] = bad
        _run_extend(c, 100)
        assert _code() in (0x400, 0x800)
    c[2][int(good[1, 11])] = 0.0
    c[5] = cu
    _run_extend(c, 100)
    _clean()


@pytest.mark.parametrize("more", [0, 130])
def test_captured_and_replayed(more):
    cases = [_extend_case(20 + i, n + [9] * more, m + [9] * more, 16, 8, 2, rows=256 + 9 * more,
                          fill=0.0) for i, (n, m) in enumerate(
        [([100, 30], [300, 40]), ([128, 128], [2000, 128]), ([0, 200], [0, 1999])])]
    pages, cols = max(c[1].shape[0] for c in cases), max(c[3].shape[1] for c in cases)

    def padded(c):
        kc = torch.zeros(pages, 16, 2, 64, dtype=BF)
        vc, table = torch.zeros_like(kc), torch.full((2 + more, cols), -1, dtype=torch.int32)
        kc[:c[1].shape[0]], vc[:c[2].shape[0]], table[:, :c[3].shape[1]] = c[1], c[2], c[3]
        return (c[0], kc, vc, table, *c[4:])

    static = [x.to(DEV) for x in padded(cases[0])]
    binding.extend(*static, window=100)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.extend(*static, window=100)
    for c in cases[::-1]:
        for dst, src in zip(static, padded(c)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        _check_extend(out, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125,
                                         window=100), int(c[5][-1]))
    _clean()
