"""A serving loop whose lengths and free list stay on the device: every step is one
replay of a graph and nothing is read back between them."""
import math

import torch
import pytest

from attention_learnable_head_gb300 import binding
from oracle.step import oracle_extend
from test_gpu_step import BF, DEV, _check_extend, _clean

pytestmark = pytest.mark.gpu


def test_a_loop_without_reading_back():
    hq, hkv, page, pages, cols, room = 8, 2, 16, 40, 12, 64
    g = torch.Generator().manual_seed(6)
    total, steps = [120, 70, 33], [[40, 20, 0], [22, 1, 33], [1, 1, 0], [30, 21, 0], [27, 27, 0]]
    qkv = [torch.randn(n, hq + 2 * hkv, 64, generator=g).to(BF) for n in total]
    freq = (10000.0 ** (-torch.arange(32) / 32)).to(DEV)
    sink = torch.randn(hq, generator=g).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    cached, new = torch.zeros(3, **i32), torch.zeros(3, **i32)
    free = torch.randperm(pages, generator=g).int().to(DEV)
    table = torch.full((3, cols), -1, **i32)
    kc = torch.full((pages, page, hkv, 64), math.nan, dtype=BF, device=DEV)
    vc = torch.full_like(kc, math.nan)
    x = torch.zeros(room, hq + 2 * hkv, 64, dtype=BF, device=DEV)
    place = torch.arange(pages, device=DEV)

    def step():
        p = binding.page_plan(cached, new, free, table, page_size=page, num_pages=pages,
                              max_tokens=room)
        q, _, _ = binding.qkv_rope(x, p.positions, freq, heads_q=hq, heads_kv=hkv, slots=p.slots,
                                   k_cache=kc, v_cache=vc)
        r = binding.extend(q, kc, vc, table, p.seq_lens, p.cu_seqlens_q, sink)
        cached.copy_(p.seq_lens)
        at = place + p.pages_needed                         # the list without the pages taken
        free.copy_(torch.where(at < pages, free[at.clamp(max=pages - 1)], -1))
        return r

    step()                                                  # of no tokens: changes nothing
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    refs = []
    for s in qkv:
        n = len(s)
        q, k, v = binding.qkv_rope(s.to(DEV), torch.arange(n, **i32), freq, heads_q=hq,
                                   heads_kv=hkv)
        refs.append(oracle_extend(q.cpu(), k.cpu()[None], v.cpu()[None],
                                  torch.zeros(1, 1, dtype=torch.int32), [n], [0, n], sink.cpu(),
                                  scale=0.125))
    have, got = [0, 0, 0], []
    for s in steps:
        new.copy_(torch.tensor(s))
        rows = torch.cat([t[h:h + n] for t, h, n in zip(qkv, have, s)])
        x.zero_()
        x[:len(rows)].copy_(rows)
        graph.replay()
        got.append((out.clone(), lse.clone(), list(have)))
        have = [h + n for h, n in zip(have, s)]
    _clean()
    assert have == total and cached.tolist() == total
    for (o, z, start), s in zip(got, steps):
        at = 0
        for b, n in enumerate(s):
            part = slice(start[b], start[b] + n)
            _check_extend((o[at:at + n], z[:, at:at + n]),
                          (refs[b][0][part], refs[b][1][:, part], refs[b][2][part]), n)
            at += n
