"""The weights of keys where some rows' lse is far from the others': each row is as exact as
its own lse and scores allow, whatever the rows next to it have.

Tolerances as in test_gpu_cache_edges.py: 2 SCORE for each weight and the additions of a
thread, here of at most 70 tokens x 4 heads / 8 and the lanes', below 300 steps of 2^-24."""
import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.cache import oracle_mass
from cache_cases import ints
from test_gpu_cache import SCORE, mass_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert binding.attn_sink_device_error() == (0, 0)


def both(c, cu, q, lse):
    k, _, table, lens = c.gpu()
    mass = torch.zeros(len(c.lens), c.hkv, c.cols * c.page, device="cuda")
    binding.key_mass(q.cuda(), k, table, lens, ints(cu), lse.cuda(), mass)
    want = oracle_mass(q, c.k, c.table, c.lens, cu, lse, torch.zeros(mass.shape), scale=0.125)
    assert (want > 0).any()
    err = (mass.double().cpu() - want).abs()
    assert (err <= (2 * SCORE + 300 * 2 ** -24) * want + 1e-30).all(), (err / (want + 1e-30)).max()


NEW = [[1, 1], [40, 70]]                                      # rows in registers, tiles of rows


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("far", [300.0, 3e3, 3e4, 1e6, 1e8, 1e10, 1e20, 9e29, 2e30, 3e38])
@pytest.mark.parametrize("head", [0, 3])
def test_a_head_that_is_switched_off(new, far, head):
    """A sink far above the scores leaves an lse of its size: that head gives no weight, the
    others theirs."""
    c, cu, q, lse = mass_case(97, new, [300, 513])
    lse[head] = far
    both(c, cu, q, lse)


@pytest.mark.parametrize("new", NEW)
def test_far_lse_of_single_tokens(new):
    c, cu, q, lse = mass_case(98, new, [300, 513])
    for t in range(0, cu[-1], 3):
        lse[:, t] = 10.0 ** (2 + t % 30)
    if cu[-1] == 2:
        lse[:3, 0] = 5.0
    both(c, cu, q, lse)


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("head", [0, 2])
def test_a_head_far_below(new, head):
    """Scores and lse of -8192 beside ones of a few: that head's weights are e^-25 of the
    others', its rounding (2^-24 of 8192, a few times) nothing of them."""
    c, cu, q, lse = mass_case(99, new, [300, 513])
    q[:, :, 0] = 0
    q[:, head] = 0
    q[:, head, 0] = -65536
    c.k[:, :, :, 0] = 1
    lse[head] = -8192 + 25
    both(c, cu, q, lse)


@pytest.mark.parametrize("new", NEW)
def test_all_far(new):
    """All lse and scores of 2048: a score's rounding, 2^-24 of 2048 a few times over, is what
    the weights are off by."""
    c, cu, q, lse = mass_case(100, new, [300, 513])
    q[:, :, 0] = 128
    c.k[:, :, :, 0] = 128
    lse += 2048
    k, _, table, lens = c.gpu()
    mass = torch.zeros(2, c.hkv, c.cols * c.page, device="cuda")
    binding.key_mass(q.cuda(), k, table, lens, ints(cu), lse.cuda(), mass)
    want = oracle_mass(q, c.k, c.table, c.lens, cu, lse, torch.zeros(mass.shape), scale=0.125)
    err = (mass.double().cpu() - want).abs()
    # 64 terms, cut at 2^-23 of what they add up to, and the lse's and the factor's roundings
    assert (err <= (64 + 8) * 2 ** -23 * 2048 * want + 1e-30).all()
