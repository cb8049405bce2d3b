"""Decode steps over a cache whose unwritten rows hold NaN, as a cache that was
allocated and then filled by attn_sink_qkv_rope does: rows behind a sequence's
last key and before its window are no part of the result, and are not reported
as values outside the fp16 range."""
import math

import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.decode import oracle_decode
from parity import TOL_LSE, assert_close
from test_gpu_step import DEV, _clean, _extend_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,window", [(8, 0), (16, 0), (64, 0), (128, 0), (16, 40), (128, 100),
                                         (48, 0), (1, 7)])
def test_decode_over_unwritten_rows(page, window):
    lens = [1, 37, 64, 300, 1000]
    q, kc, vc, table, ln, _, sink = _extend_case(page, [1] * 5, lens, page, 16, 2, fill=math.nan)
    if window:
        # rows behind the window are gone too
        for b, n in enumerate(lens):
            for j in range(max(0, n - window)):
                kc[table[b, j // page], j % page] = math.nan
                vc[table[b, j // page], j % page] = math.inf
    out, lse, _ = binding.decode(*(x.to(DEV) for x in (q, kc, vc, table, ln, sink)), window=window)
    _clean()
    ref, ref_lse = oracle_decode(q, torch.nan_to_num(kc, 0.0, 0.0, 0.0),
                                 torch.nan_to_num(vc, 0.0, 0.0, 0.0), table, ln, sink, scale=0.125,
                                 window=window)
    assert_close(f"page {page} window {window} out", out.cpu(), ref)
    assert (lse.cpu().double() - ref_lse).abs().max().item() <= TOL_LSE
