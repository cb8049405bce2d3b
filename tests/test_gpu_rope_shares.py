"""The head rotation and its gradient where a warp's share of a token is just small
enough to be copied as a whole (28 heads of q, k and v; the gradient 17, or 11 with
fp32 gradients), and just too large: the parity tests of test_gpu_step, at those
sizes, with one warp a token and with several."""
import pytest

import test_gpu_step as step

pytestmark = pytest.mark.gpu

SHARES = [  # tokens, query heads, key/value heads
    (3100, 24, 2), (3100, 25, 2), (3100, 27, 1), (7, 26, 1), (7, 27, 1),   # 28, 29
    (3100, 10, 2), (3100, 11, 2), (3100, 12, 1), (5, 6, 4), (5, 7, 4),      # 14, 15
    (3100, 4, 2), (3100, 5, 2), (3100, 6, 1), (2, 1, 1),                    # 8, 9
    (3100, 13, 2), (3100, 14, 2), (3100, 15, 1), (6, 9, 4), (6, 16, 1),     # 17, 18
    (3100, 7, 2), (3100, 8, 2), (3100, 9, 1), (4, 3, 4), (4, 10, 1),        # 11, 12
    (600, 64, 8), (800, 64, 8), (1600, 28, 4), (1500, 12, 2), (90, 64, 8),
]


@pytest.mark.parametrize("t,hq,hkv", SHARES)
def test_rope(t, hq, hkv):
    step.test_rope(t, hq, hkv, 64, 1, True, t % 2 == 1, 1.0, 4000)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("t,hq,hkv", SHARES)
def test_rope_backward(t, hq, hkv, fp32):
    step.test_rope_backward(t, hq, hkv, 64, 1, True, t % 2 == 1, 1.0, 4000, fp32)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("hq,hkv", [(24, 2), (25, 2)])
def test_without_norm_and_partly_rotated(hq, hkv, norm):
    step.test_rope(3100, hq, hkv, 48, 2, norm, False, 1.25, 4000)
    step.test_rope_backward(3100, hq, hkv, 48, 2, norm, False, 1.25, 4000, False)


@pytest.mark.parametrize("t,page", [(3100, 16), (64, 24)])
def test_rope_into_the_cache(t, page):
    step.test_rope_into_the_cache(t, page)
