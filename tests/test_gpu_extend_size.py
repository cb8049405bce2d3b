"""The size of attn_sink_extend's error as a whole, which the bound of each output (the
worst case) does not see.  Two roundings to bf16: of P, independent over the keys, and of
the output.  A rounding is off by at most 2^-8 of the value and evenly spread, 2^-8 /
sqrt(3) in the mean square, or less where the value lies higher in its binade.  For values
of random signs each moves the output by that part of it in the mean square, so together
sqrt(2 / 3) 2^-8 = 0.0032 of the outputs' norm; P's fp32 arithmetic (2^-11 at most) adds
its part, and the norm of thousands of outputs spreads by about a hundredth.  On the band
kernel P is fp16, off by 2^-11: sqrt(1 / 3) 2^-8 + 2^-11."""
import math

import pytest

from attention_learnable_head_gb300 import binding
from oracle.step import oracle_extend
from test_gpu_step import _clean, _extend_case, _run_extend

pytestmark = pytest.mark.gpu

ROUND = 2.0 ** -8 / math.sqrt(3)


@pytest.mark.parametrize("new,lens,page,hq,hkv,window,band", [
    ([5, 3, 4], [9000, 400, 3000], 16, 64, 8, 0, False),
    ([200, 300], [900, 300], 64, 16, 2, 0, False),
    ([17, 40], [2000, 5000], 1, 16, 2, 0, False),
    ([300, 7], [900, 513], 16, 8, 1, 128, False),
    ([70] * 140, [70 + 11 * i for i in range(140)], 16, 16, 2, 128, True),
])
def test_relative_norm(new, lens, page, hq, hkv, window, band):
    c = _extend_case(len(new) + page, new, lens, page, hq, hkv)
    before = binding.attn_sink_launch_count()
    out, _ = _run_extend(c, window)
    if band:
        assert binding.attn_sink_launch_count() - before == 3
    ref = oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125, window=window)[0]
    rel = ((out.cpu().double() - ref).norm() / ref.norm()).item()
    limit = (ROUND if band else math.sqrt(2) * ROUND) + 2.0 ** -11
    assert rel <= 1.01 * limit, rel
    _clean()
