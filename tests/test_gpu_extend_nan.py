"""attn_sink_extend with scores that are not numbers, in whole and in cut tiles, and with
sinks of +inf, on the band kernel too."""
import math

import pytest
import torch

from oracle.step import oracle_extend
from test_gpu_step import _check_extend, _clean, _extend_case, _run_extend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("length", [60, 500, 9000])
def test_a_nan_score_gives_a_nan_lse(length, page):
    """-inf is the mark of a row without keys."""
    c = _extend_case(length, [20, 3], [length, 7], page, 8, 2, fill=0.0)
    for j in (length - 8, 11):             # one key in sight of the last tokens, one of all
        c[1][int(c[3][0, j // page]), j % page, 1] = math.nan
        out, lse = _run_extend(c)
        seen = torch.zeros(8, 23, dtype=torch.bool)
        seen[4:, max(0, 20 - (length - j)):20] = True
        assert torch.equal(lse.isnan().cpu(), seen)
        assert torch.equal(out.isnan().all(-1).cpu(), seen.T)
        assert torch.equal(out.isnan().any(-1).cpu(), seen.T)
    _clean()


@pytest.mark.parametrize("length", [60, 500, 9000])
def test_a_nan_query_gives_nan(length):
    """Every score of the row is NaN, in every part of its tile."""
    c = _extend_case(length, [20, 3], [length, 7], 16, 8, 2, fill=0.0)
    c[0][4, 5] = math.nan
    out, lse = _run_extend(c)
    seen = torch.zeros(8, 23, dtype=torch.bool)
    seen[5, 4] = True
    assert torch.equal(lse.isnan().cpu(), seen)
    assert torch.equal(out.isnan().all(-1).cpu(), seen.T)
    assert torch.equal(out.isnan().any(-1).cpu(), seen.T)
    _clean()


@pytest.mark.parametrize("length,window,more", [(60, 0, 0), (9000, 0, 0), (300, 100, 130)])
def test_a_sink_of_infinity_takes_all(length, window, more):
    """out = 0 and lse = inf; the other heads as ever."""
    c = list(_extend_case(length, [20, 3] + [12] * more, [length, 0] + [12] * more, 16, 8, 2))
    c[6] = torch.tensor([0.5, math.inf, 1.0, 0.0, math.inf, -1.0, -math.inf, 2.0])
    n = 23 + 12 * more
    out, lse = _run_extend(c, window)
    _clean()
    assert not out[:, [1, 4]].any() and (lse[[1, 4]] == math.inf).all()
    rest = [0, 2, 3, 5, 6, 7]
    ref = oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125, window=window)
    _check_extend((out[:, rest], lse[rest]), (ref[0][:, rest], ref[1][rest], ref[2][:, rest]), n)
