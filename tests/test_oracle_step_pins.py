"""Pins of the oracles around the attention (CPU): the rotation against complex
arithmetic, its gradient against automatic differentiation and central
differences, the plan against its own invariants, the paged attention of
several tokens against the main attention oracle."""
import math

import pytest
import torch

from oracle import oracle_fwd
from oracle.step import (oracle_extend, oracle_plan, oracle_rope, oracle_rope_bwd, pair_dims,
                         rope_angles)

F64 = torch.float64


def _rope_case(seed, rotary, axes):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(5, 3, 64, generator=g, dtype=F64)
    w = 1 + 0.3 * torch.randn(64, generator=g, dtype=F64)
    pos = torch.randint(0, 1000, (axes, 5), generator=g)
    freq = 100.0 ** (-torch.arange(rotary // 2) / max(1, rotary // 2))
    return x, w, rope_angles(pos, freq, [i % axes for i in range(rotary // 2)])


@pytest.mark.parametrize("rotary,inter,axes", [(64, False, 1), (32, True, 2), (48, False, 3),
                                               (16, True, 1)])
def test_rotation_is_a_complex_product(rotary, inter, axes):
    x, _, ang = _rope_case(rotary, rotary, axes)
    y = oracle_rope(x, None, ang, eps=0.0, interleaved=inter, amplitude=1.5)
    a, b = pair_dims(rotary, inter)
    z = torch.complex(x[..., a], x[..., b]) * (1.5 * torch.exp(1j * ang))[:, None]
    assert torch.allclose(torch.complex(y[..., a], y[..., b]), z, atol=1e-12)
    assert torch.equal(y[..., rotary:], x[..., rotary:])


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_is_that_of_the_forward(inter):
    x, w, ang = _rope_case(3, 48, 2)
    kw = dict(eps=1e-3, interleaved=inter, amplitude=0.7)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(4), dtype=F64)
    xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
    ref = torch.autograd.grad(oracle_rope(xl, wl, ang, **kw), [xl, wl], dy)
    dx, dw = oracle_rope_bwd(x, w, ang, dy, **kw)
    assert torch.allclose(dx, ref[0], atol=1e-12) and torch.allclose(dw, ref[1], atol=1e-12)
    # central differences, independently of automatic differentiation
    h = 1e-6
    for t, hd, d in ((0, 0, 0), (2, 1, 40), (4, 2, 63)):
        e = torch.zeros_like(x)
        e[t, hd, d] = h
        num = ((oracle_rope(x + e, w, ang, **kw) - oracle_rope(x - e, w, ang, **kw)) * dy).sum()
        assert abs(num.item() / (2 * h) - dx[t, hd, d].item()) < 1e-7


def test_plan_gives_every_token_its_own_row():
    cached, new, page = [0, 5, 16, 17, 0, 3], [4, 0, 1, 40, 0, 13], 16
    table = [[100 * b + c if c < -(-cached[b] // page) else -9 for c in range(5)]
             for b in range(6)]
    slots, pos, cu, lens, needed = oracle_plan(cached, new, list(range(1000, 1020)), table, page, 64)
    real = slots[:sum(new)]
    assert len(set(real)) == len(real) and slots[sum(new):] == [-1] * (64 - sum(new))
    assert cu == [0, 4, 4, 5, 45, 45, 58] and lens == [4, 5, 17, 57, 0, 16]
    assert needed == 1 + 0 + 1 + 2 + 0 + 0 and table[5][0] == 500 and table[4][0] == -9
    assert pos[45:58] == list(range(3, 16)) and real[45] == 500 * 16 + 3
    assert table[3][2:4] == [1002, 1003]


@pytest.mark.parametrize("window", [0, 7])
def test_extend_is_the_attention_of_the_last_rows(window):
    g = torch.Generator().manual_seed(9)
    lens, new, page, hq, hkv = [20, 9, 0, 4, 13], [6, 9, 0, 1, 0], 4, 4, 2
    cu = [0, 6, 15, 15, 16, 16]
    count = [-(-n // page) for n in lens]
    perm = torch.randperm(sum(count) + 2, generator=g)
    kc = torch.randn(len(perm), page, hkv, 16, generator=g, dtype=F64)
    vc = torch.randn(len(perm), page, hkv, 16, generator=g, dtype=F64)
    table, at = torch.full((5, 5), -1), 0
    for b, c in enumerate(count):
        table[b, :c] = perm[at:at + c]
        at += c
    q = torch.randn(18, hq, 16, generator=g, dtype=F64)
    sink = torch.randn(hq, generator=g)
    out, lse, spread = oracle_extend(q, kc, vc, table, lens, cu, sink, scale=0.3, window=window)
    for b in range(5):
        rows = table[b, :count[b]]
        k, v = (c[rows].reshape(-1, hkv, 16)[:lens[b]] for c in (kc, vc))
        ref, ref_lse = oracle_fwd(q[cu[b]:cu[b + 1]], k, v, sink, scale=0.3, causal=True,
                                  window=window, cu_seqlens_q=[0, new[b]],
                                  cu_seqlens_k=[0, lens[b]])
        assert torch.allclose(out[cu[b]:cu[b + 1]], ref, atol=1e-12)
        assert torch.allclose(lse[:, cu[b]:cu[b + 1]], ref_lse, atol=1e-12)
    assert torch.isnan(out[16:]).all() and torch.isnan(lse[:, 16:]).all()
    assert (spread[:16] >= out[:16].abs() - 1e-12).all()
    # an entry outside the cache hides its keys
    table[0, 1] = 1000
    o2, l2, _ = oracle_extend(q, kc, vc, table, lens, cu, sink, scale=0.3)
    assert torch.isfinite(o2[:16]).all() and not torch.allclose(o2[:6], out[:6])
    assert math.isfinite(l2[0, 0].item())
