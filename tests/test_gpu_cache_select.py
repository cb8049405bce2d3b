"""The choice of pages where scores are far below the range of fp32: it is that of 64-bit
scores all the same."""
import pytest
import torch

from attention_learnable_head_gb300 import binding
from cache_cases import BF16, Paged
from test_gpu_cache import random_bounds, select_both

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert binding.attn_sink_device_error() == (0, 0)


def tiny(x, scale):
    """x times a power of two, in bf16 without a second rounding."""
    return (x.double() * 2.0 ** scale).to(BF16)


@pytest.mark.parametrize("q_exp,b_exp", [
    (-80, -80), (-100, -110), (-120, -3), (-3, -120), (-60, -70), (-45, -45), (-40, -40), (-30, -30)])
@pytest.mark.parametrize("lens,count", [([640, 333], 9), ([9000], 200)])
def test_small_scores(q_exp, b_exp, lens, count):
    """Products of 2^-60 to 2^-210: below 2^-149 fp32 has nothing left of them."""
    c = Paged(111, lens, page=8)
    select_both(c, tiny(c.q(), q_exp), tiny(random_bounds(c), b_exp), count)


def test_one_head_is_small():
    """The largest of a group's heads decides; a small one's scores beside zeros too."""
    c = Paged(112, [640, 333], hq=8, hkv=2)
    q = tiny(c.q(), -100)
    q[:, 1:4] = 0
    select_both(c, q, tiny(random_bounds(c), -60), 9)
    q = c.q()
    q[:, 0] = tiny(q[:, 0], -110)
    select_both(c, q, random_bounds(c), 9)


def test_zeros_are_ties():
    """Bounds or queries of zero: the lower columns, beside a sequence that has scores."""
    c = Paged(113, [640, 333])
    q, b = c.q(), random_bounds(c)
    q[0] = 0
    select_both(c, q, b, 9)
    select_both(c, c.q(), torch.zeros_like(b), 9)
    select_both(c, q, tiny(b, -100), 9)
