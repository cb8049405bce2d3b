"""Calls of attn_sink_step.h that the parity tests do not make: caches whose
offsets pass 32 bits, empty caches and batches, a whole serving step captured into
one graph, two calls at once, windows wider than any sequence."""
import math

import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.step import oracle_extend
from test_gpu_step import BF, DEV, _check_extend, _clean, _dev, _extend_case, _rope_case, _run_extend

pytestmark = pytest.mark.gpu


def test_rows_beyond_32_bits():
    """A cache of 2^32 + 2^24 elements each for K and V: the last pages are written
    by qkv_rope and read by extend (general and windowed), by decode, and equal
    the same rows in a small cache."""
    hq, hkv, page = 8, 8, 16
    pages = (1 << 32) // (page * hkv * 64) + 2048
    kc = torch.empty(pages, page, hkv, 64, dtype=BF, device=DEV)
    vc = torch.empty_like(kc)
    assert kc.numel() > 1 << 32
    n = 40
    s = {k: _dev(v) for k, v in _rope_case(3, n, hq, hkv, 64, 1, True).items()}
    far = torch.arange(pages - 3, pages, dtype=torch.int32, device=DEV)
    slots = far.long()[torch.arange(n, device=DEV) // page] * page + torch.arange(n, device=DEV) % page
    assert slots[0].item() * hkv * 64 > 1 << 32
    q, _, _ = binding.qkv_rope(**s, heads_q=hq, heads_kv=hkv, slots=slots, k_cache=kc, v_cache=vc)
    near = [torch.zeros(3, page, hkv, 64, dtype=BF, device=DEV) for _ in range(2)]
    binding.qkv_rope(**s, heads_q=hq, heads_kv=hkv, slots=torch.arange(n, device=DEV),
                     k_cache=near[0], v_cache=near[1])
    i32 = dict(dtype=torch.int32, device=DEV)
    lens, cu = torch.tensor([n], **i32), torch.tensor([0, n], **i32)
    sink = torch.zeros(hq, device=DEV)
    for window in (0, 20):
        a = binding.extend(q, kc, vc, far[None], lens, cu, sink, window=window)
        b = binding.extend(q, *near, torch.arange(3, **i32)[None], lens, cu, sink, window=window)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = binding.decode(q[-1:].contiguous(), kc, vc, far[None], lens, sink)
    b = binding.decode(q[-1:].contiguous(), *near, torch.arange(3, **i32)[None], lens, sink)
    assert torch.equal(a[0], b[0])
    _clean()


def test_empty_caches_and_batches():
    i32 = dict(dtype=torch.int32, device=DEV)
    none = torch.zeros(0, 16, 2, 64, dtype=BF, device=DEV)
    q, sink = torch.randn(5, 8, 64, device=DEV).to(BF), torch.randn(8, device=DEV)
    for window in (0, 50):
        out, lse = binding.extend(q, none, none, torch.zeros(1, 0, **i32), torch.zeros(1, **i32),
                                  torch.tensor([0, 5], **i32), sink, window=window)
        assert not out.any() and torch.equal(lse, sink[:, None].expand(8, 5))
    out, lse = binding.extend(q[:0], none, none, torch.zeros(0, 3, **i32), torch.zeros(0, **i32),
                              torch.zeros(1, **i32), sink)
    assert out.shape == (0, 8, 64) and lse.shape == (8, 0)
    qkv = torch.randn(3, 12, 64, device=DEV).to(BF)
    args = (qkv, torch.zeros(3, **i32), torch.ones(32, device=DEV))
    binding.qkv_rope(*args, heads_q=8, heads_kv=2, k_cache=none, v_cache=none,
                     slots=torch.full((3,), -1, device=DEV))
    _clean()
    binding.qkv_rope(*args, heads_q=8, heads_kv=2, k_cache=none, v_cache=none,
                     slots=torch.zeros(3, dtype=torch.int64, device=DEV))
    assert binding.attn_sink_device_error() == (0, 0x800)


@pytest.mark.parametrize("new,window", [([5, 40], 1 << 30), ([5, 40], 2 ** 31 - 1), ([20, 3], 1000)])
def test_windows_wider_than_the_sequences(new, window):
    c = _extend_case(7, new, [300, 40], 16, 8, 2)
    a, b = _run_extend(c, window), _run_extend(c, 0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _clean()


@pytest.mark.parametrize("window", [0, 64])
def test_a_captured_serving_step(window):
    """plan, rope into the pages and extend in one graph, replayed as the sequences
    grow: only lengths, tokens and the free list change between replays."""
    hq, hkv, page, pages, cols, room = 8, 2, 16, 80, 24, 96
    g = torch.Generator().manual_seed(5)
    total, steps = [150, 70, 33], [[40, 20, 0], [22, 1, 33], [1, 1, 0], [60, 0, 0], [27, 48, 0]]
    qkv = [torch.randn(n, hq + 2 * hkv, 64, generator=g).to(BF) for n in total]
    freq, sink = (10000.0 ** (-torch.arange(32) / 32)).to(DEV), torch.randn(hq, generator=g)
    i32 = dict(dtype=torch.int32, device=DEV)
    cached, new = torch.zeros(3, **i32), torch.zeros(3, **i32)
    free, table = torch.zeros(pages, **i32), torch.full((3, cols), -1, **i32)
    kc = torch.full((pages, page, hkv, 64), math.nan, dtype=BF, device=DEV)
    vc = torch.full_like(kc, math.nan)
    x = torch.zeros(room, hq + 2 * hkv, 64, dtype=BF, device=DEV)

    def step():
        p = binding.page_plan(cached, new, free, table, page_size=page, num_pages=pages,
                              max_tokens=room)
        q, _, _ = binding.qkv_rope(x, p.positions, freq, heads_q=hq, heads_kv=hkv, slots=p.slots,
                                   k_cache=kc, v_cache=vc)
        return p, binding.extend(q, kc, vc, table, p.seq_lens, p.cu_seqlens_q, sink.to(DEV),
                                 window=window)

    step()
    graph = torch.cuda.CUDAGraph()
    sink = sink.to(DEV)
    with torch.cuda.graph(graph):
        p, (out, lse) = step()
    refs = []
    for s in qkv:
        n = len(s)
        q, k, v = binding.qkv_rope(s.to(DEV), torch.arange(n, **i32), freq, heads_q=hq,
                                   heads_kv=hkv)
        refs.append(oracle_extend(q.cpu(), k.cpu()[None], v.cpu()[None],
                                  torch.zeros(1, 1, dtype=torch.int32), [n], [0, n], sink.cpu(),
                                  scale=0.125, window=window))
    order = torch.randperm(pages, generator=g).int()
    table.fill_(-1)
    have, taken = [0, 0, 0], 0
    for s in steps:
        cached.copy_(torch.tensor(have))
        new.copy_(torch.tensor(s))
        free[:pages - taken].copy_(order[taken:])
        rows = torch.cat([t[h:h + n] for t, h, n in zip(qkv, have, s)])
        x.zero_()
        x[:len(rows)].copy_(rows)
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(s):
            part = slice(have[b], have[b] + n)
            _check_extend((out[at:at + n], lse[:, at:at + n]),
                          (refs[b][0][part], refs[b][1][:, part], refs[b][2][part]), n)
            at += n
        taken += p.pages_needed.item()
        have = [h + n for h, n in zip(have, s)]
    assert have == total
    _clean()


def test_two_gradients_at_once():
    """Calls on two streams have workspaces of their own."""
    cases = [{k: _dev(v) for k, v in _rope_case(i, 3000, 8, 2, 64, 1, True).items()} for i in (1, 2)]
    grads = [[torch.randn(3000, h, 64, device=DEV).to(BF) for h in (8, 2, 2)] for _ in cases]

    def run(i, stream=None):
        s = cases[i]
        return binding.qkv_rope_backward(
            s["qkv"], s["positions"], s["inv_freq"], *grads[i], heads_q=8, heads_kv=2,
            q_weight=s["q_weight"], k_weight=s["k_weight"], pair_axis=s["pair_axis"], stream=stream)

    alone = [run(0), run(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [run(i, st) for i, st in enumerate(streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    _clean()


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_of_extreme_positions(interleaved):
    """x = (1, 0) in every pair gives (cos, sin).  The angle is off by 2^-32 turns,
    and by inv_freq / 2 pi in fp64 (2^-52, as the product of two roundings) times a
    position of up to 2^31: 2^-21 turns, 2^-18 radians with the reference's own; the
    sine and cosine by 2^-22, the result by half a bf16 step: eps / 2 = 2^-8 of it."""
    pos = torch.tensor([0, 1, -1, 4097, 1_000_003, -99_999_999, 2 ** 31 - 1, -2 ** 31])
    freq = torch.tensor([1.0, -1.0, 0.75, 2.0 ** -30, 1e-9, -0.3, 0.0, 3.0] + [0.5 ** i for i in
                                                                                range(24)])
    bad = {5: math.nan, 9: math.inf}
    x = torch.zeros(len(pos), 3, 64)
    a = torch.arange(32) * 2 if interleaved else torch.arange(32)
    b = a + 1 if interleaved else a + 32
    x[:, :, a] = 1.0
    got = freq.clone()
    for i, f in bad.items():
        got[i] = f
    q, k, v = binding.qkv_rope(x.to(BF).to(DEV), pos.int().to(DEV), got.to(DEV), heads_q=1,
                               heads_kv=1, interleaved=interleaved)
    angle = pos.double()[:, None] * freq.double()
    keep = torch.tensor([i not in bad for i in range(32)])
    for y in (q[:, 0].cpu().double(), k[:, 0].cpu().double()):
        for d, ref in ((a, angle.cos()), (b, angle.sin())):
            err = (y[:, d] - ref).abs()[:, keep]
            assert (err <= 2.0 ** -8 * ref.abs()[:, keep] + 2.0 ** -17).all(), err.max()
            assert y[:, d][:, ~keep].isnan().all()
    assert torch.equal(v[:, 0].cpu(), x[:, 2].to(BF))
    _clean()
