"""Windows wider than 32 bits are windows wider than any sequence."""
import pytest
import torch

from test_gpu_step import _clean, _extend_case, _run_extend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1, -2 ** 40])
def test_windows_past_32_bits(window):
    c = _extend_case(7, [5, 40], [300, 40], 16, 8, 2)
    a, b = _run_extend(c, window), _run_extend(c, 0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _clean()
