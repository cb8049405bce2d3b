"""GPU parity of the entry points around the attention (attn_sink_step.h)
against the float64 oracles.

Tolerances, derived from the roundings (bf16 2^-8, fp32 2^-24 relative):
  plan      whole numbers: equal
  rope      one bf16 rounding of the result, 2^-8 |y|; the fp32 arithmetic before
            it (square root, three products, sine and cosine) is within 2^-20 of
            the terms' magnitudes |u_a| + |u_b|
  gradient  dx likewise: 2^-8 |dx| + 2^-19 of the terms' magnitudes; a weight's
            gradient is a sum of n fp32 terms: (2^-19 + n 2^-24) of the sum of
            their magnitudes at most
  extend    out: 2^-8 |out| for its rounding, and every P_ij moves by its bf16
            rounding 2^-8 and its fp32 arithmetic, below 2^-11 (a score of
            magnitude up to 30 summed from 64 fp32 products is off by less than
            64 * 30 * 2^-24 = 2^-13, exp2 by 2^-22): (2^-8 + 2^-11) sum_j P_ij |v_j|;
            lse: the scores' 2^-13 again, and a rounding of its own"""
import ctypes
import math
import time

import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.step import (oracle_extend, oracle_plan, oracle_rope, oracle_rope_bwd, pair_dims,
                         rope_angles)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def _clean():
    torch.cuda.synchronize()
    assert binding.attn_sink_device_error() == (0, 0)


def _code():
    st, code = binding.attn_sink_device_error()
    assert st == 0
    return code


# ----------------------------------------------------------------------------- plan
def _plan_case(seed, batch, page, most_cached, most_new, spare=3):
    r = torch.Generator().manual_seed(seed)
    cached = torch.randint(0, most_cached + 1, (batch,), generator=r).tolist()
    new = torch.randint(0, most_new + 1, (batch,), generator=r).tolist()
    if batch > 2:
        cached[1], new[2] = 0, 0
    cols = max([-(-(c + n) // page) for c, n in zip(cached, new)] + [0]) + 1
    held = sum(-(-c // page) for c in cached)
    need = sum(-(-(c + n) // page) + (-c // page) for c, n in zip(cached, new))
    perm = torch.randperm(held + need + spare, generator=r).tolist()
    table, at = [], 0
    for c in cached:
        n = -(-c // page)
        table.append(perm[at:at + n] + [-7] * (cols - n))
        at += n
    return cached, new, perm[held:], table, len(perm)


def _run_plan(cached, new, free, table, page, pages, tokens, cols=None):
    i32 = dict(dtype=torch.int32, device=DEV)
    t = torch.tensor(table, **i32).reshape(len(cached), -1 if cols is None else cols)
    p = binding.page_plan(torch.tensor(cached, **i32), torch.tensor(new, **i32),
                          torch.tensor(free, **i32), t, page_size=page, num_pages=pages,
                          max_tokens=tokens)
    torch.cuda.synchronize()
    return p, t


def _check_plan(p, t, ref, ref_table):
    slots, positions, cu, lens, needed = ref
    assert t.tolist() == ref_table
    assert p.slots.tolist() == slots and p.positions.tolist() == positions
    assert p.cu_seqlens_q.tolist() == cu and p.seq_lens.tolist() == lens
    assert p.pages_needed.item() == needed


@pytest.mark.parametrize("batch,page,cached,new,pad", [
    (1, 16, 0, 1, 0), (1, 16, 100, 5000, 7), (5, 1, 9, 4, 64), (7, 48, 200, 1, 1),
    (255, 16, 300, 3, 0), (256, 24, 40, 9, 5), (257, 16, 64, 2, 300), (1000, 128, 1000, 40, 11),
    (4, 16, 0, 0, 3)])
def test_plan(batch, page, cached, new, pad):
    c, n, free, table, pages = _plan_case(batch + page, batch, page, cached, new)
    tokens = sum(n) + pad
    ref_table = [list(r) for r in table]
    ref = oracle_plan(c, n, free, ref_table, page, tokens)
    p, t = _run_plan(c, n, free, table, page, pages, tokens)
    _check_plan(p, t, ref, ref_table)
    _clean()


def test_plan_of_no_sequences():
    p, t = _run_plan([], [], [3, 4], [], 16, 8, 5, cols=4)
    assert p.slots.tolist() == [-1] * 5 and p.cu_seqlens_q.tolist() == [0]
    assert p.pages_needed.item() == 0
    _clean()


def test_plan_reports_what_does_not_fit():
    # the free pages run out: the tokens without a page get no row
    c, n, free, table, pages = _plan_case(3, 6, 16, 40, 60, spare=0)
    few = free[:len(free) - 2]
    ref_table = [list(r) for r in table]
    ref = oracle_plan(c, n, few, ref_table, 16, sum(n))
    p, t = _run_plan(c, n, few, table, 16, pages, sum(n))
    _check_plan(p, t, ref, ref_table)
    assert _code() == 0x1000 and p.pages_needed.item() == len(free)
    # more tokens than there is room for
    p, t = _run_plan([3, 0], [4, 5], [1, 2], [[0, -1], [-1, -1]], 16, 8, 6)
    assert p.cu_seqlens_q.tolist() == [0, 4, 6] and p.slots.tolist() == [3, 4, 5, 6, 16, 17]
    assert _code() == 0x1000
    # lengths that are negative or beyond the table are clamped
    p, t = _run_plan([-3, 30], [2, 9], [1, 2, 3], [[-1, -1], [5, 6]], 16, 8, 16)
    assert p.seq_lens.tolist() == [2, 32] and p.cu_seqlens_q.tolist() == [0, 2, 4]
    assert _code() == 0x1000
    # pages outside the cache, listed free or held
    p, t = _run_plan([0, 4], [1, 1], [8, 3], [[-1, -1], [-2, -1]], 16, 8, 2)
    assert p.slots.tolist() == [-1, -1] and t[0, 0].item() == -1
    assert _code() == 0x1000


# ----------------------------------------------------------------------------- rope
def _rope_case(seed, t, hq, hkv, rotary, axes, norm, weight=torch.float32, far=2000, wide=0):
    g = torch.Generator().manual_seed(seed)
    rows = hq + 2 * hkv
    qkv = torch.randn(t, rows + wide, 64, generator=g).to(BF)[:, :rows]
    pairs = rotary // 2
    s = dict(qkv=qkv, positions=torch.randint(0, far, (axes, t), generator=g).int(),
             inv_freq=10000.0 ** (-torch.arange(pairs) / max(1, pairs)),
             pair_axis=[(i * axes) // max(1, pairs) for i in range(pairs)], q_weight=None,
             k_weight=None)
    if norm:
        s["q_weight"] = (1 + 0.2 * torch.randn(64, generator=g)).to(weight)
        s["k_weight"] = (1 + 0.2 * torch.randn(64, generator=g)).to(weight)
    return s


def _dev(x):
    if torch.is_tensor(x):
        # a strided view stays one
        return x.to(DEV) if x.is_contiguous() else torch.cat(
            [x, x[:, :1]], 1).to(DEV)[:, :x.shape[1]]
    return x


def _rope_refs(s, hq, hkv, inter, amp, eps):
    """Results and the magnitudes of the terms that make them."""
    ang = rope_angles(s["positions"], s["inv_freq"], s["pair_axis"])
    kw = dict(eps=eps, interleaved=inter, amplitude=amp)
    out = []
    for x, w in ((s["qkv"][:, :hq], s["q_weight"]), (s["qkv"][:, hq:hq + hkv], s["k_weight"])):
        y = oracle_rope(x, w, ang, **kw)
        u = oracle_rope(x, w, ang * 0, eps=eps, interleaved=inter, amplitude=1.0).abs()
        a, b = pair_dims(s["inv_freq"].shape[0] * 2, inter)
        size = u.clone()
        size[..., a] = size[..., b] = max(abs(amp), 1.0) * (u[..., a] + u[..., b])
        out.append((y, size))
    return out


ROPE = [  # t, hq, hkv, rotary, axes, norm, inter, amp, far
    (1, 64, 8, 64, 1, True, False, 1.0, 131072),
    (3, 5, 1, 48, 1, True, False, 1.0, 100),
    (129, 8, 8, 32, 2, True, True, 1.0, 4000),
    (130, 6, 2, 64, 3, True, False, 1.0, 4000),
    (37, 16, 2, 64, 1, False, False, 1.34, 2000000000),
    (64, 2, 1, 16, 4, False, True, 0.5, 100),
    (40, 4, 2, 0, 1, True, False, 1.0, 100),
    (2500, 3, 1, 64, 1, True, True, 1.0, 5000),
]


@pytest.mark.parametrize("t,hq,hkv,rotary,axes,norm,inter,amp,far", ROPE)
def test_rope(t, hq, hkv, rotary, axes, norm, inter, amp, far):
    s = _rope_case(t + hq, t, hq, hkv, rotary, axes, norm, far=far, wide=t % 3)
    got = binding.qkv_rope(**{k: _dev(v) for k, v in s.items()}, heads_q=hq, heads_kv=hkv,
                           interleaved=inter, amplitude=amp, eps=1e-5)
    _clean()
    refs = _rope_refs(s, hq, hkv, inter, amp, 1e-5)
    for g, (ref, size) in zip(got, refs):
        err = (g.cpu().double() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * size).all(), err.max()
    assert torch.equal(got[2].cpu(), s["qkv"][:, hq + hkv:])


def test_rope_bf16_weights_and_one_axis_vector():
    s = _rope_case(5, 50, 8, 2, 64, 1, True, weight=BF)
    s["positions"], s["pair_axis"] = s["positions"][0], None
    kw = {k: _dev(v) for k, v in s.items()}
    got = binding.qkv_rope(**kw, heads_q=8, heads_kv=2)
    kw["q_weight"], kw["k_weight"] = kw["q_weight"].float(), kw["k_weight"].float()
    for a, b in zip(got, binding.qkv_rope(**kw, heads_q=8, heads_kv=2)):
        assert torch.equal(a, b)
    _clean()


@pytest.mark.parametrize("t,page", [(1, 16), (33, 1), (200, 48)])
def test_rope_into_the_cache(t, page):
    """k and v land in their slots, every other row of the cache stays as it was;
    a slot of -1 writes nothing, one outside the cache is reported."""
    hq, hkv = 8, 2
    s = {k: _dev(v) for k, v in _rope_case(t, t, hq, hkv, 64, 1, True).items()}
    pages = t // page + 3
    kc = torch.randn(pages, page, hkv, 64, device=DEV).to(BF)
    vc = torch.randn(pages, page, hkv, 64, device=DEV).to(BF)
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.randperm(pages * page, device=DEV)[:t]
    plain = binding.qkv_rope(**s, heads_q=hq, heads_kv=hkv)
    q, k, v = binding.qkv_rope(**s, heads_q=hq, heads_kv=hkv, slots=slots, k_cache=kc, v_cache=vc)
    assert k is None and v is None and torch.equal(q, plain[0])
    k0.view(-1, hkv, 64)[slots], v0.view(-1, hkv, 64)[slots] = plain[1], plain[2]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    got = binding.qkv_rope(**s, heads_q=hq, heads_kv=hkv, slots=torch.full_like(slots, -1),
                           k_cache=kc, v_cache=vc, keep_kv=True)
    assert all(torch.equal(a, b) for a, b in zip(got, plain))
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    _clean()
    for bad in (pages * page, -2, 1 << 40):
        slots = torch.full_like(slots, bad)
        binding.qkv_rope(**s, heads_q=hq, heads_kv=hkv, slots=slots, k_cache=kc, v_cache=vc)
        assert _code() == 0x800
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_rope_of_no_tokens():
    s = {k: _dev(v) for k, v in _rope_case(1, 0, 4, 2, 64, 1, True).items()}
    q, k, v = binding.qkv_rope(**s, heads_q=4, heads_kv=2)
    assert q.shape == (0, 4, 64) and k.shape == v.shape == (0, 2, 64)
    dqkv, dwq, dwk = binding.qkv_rope_backward(s.pop("qkv"), s.pop("positions"),
                                               s.pop("inv_freq"), q, k, v, heads_q=4, heads_kv=2,
                                               **s)
    assert dqkv.shape == (0, 8, 64) and not dwq.any() and not dwk.any()
    _clean()


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("t,hq,hkv,rotary,axes,norm,inter,amp,far", ROPE)
def test_rope_backward(t, hq, hkv, rotary, axes, norm, inter, amp, far, fp32):
    s = _rope_case(t + hq, t, hq, hkv, rotary, axes, norm, far=far, wide=t % 3)
    g = torch.Generator().manual_seed(t)
    dys = [torch.randn(t, h, 64, generator=g) for h in (hq, hkv, hkv)]
    if not fp32:
        dys = [d.to(BF) for d in dys]
    d = {k: _dev(v) for k, v in s.items()}
    kw = dict(q_weight=d["q_weight"], k_weight=d["k_weight"], pair_axis=d["pair_axis"], heads_q=hq,
              heads_kv=hkv, interleaved=inter, amplitude=amp, eps=1e-5)
    args = (d["qkv"], d["positions"], d["inv_freq"], *(y.to(DEV) for y in dys))
    got, dwq, dwk = binding.qkv_rope_backward(*args, **kw)
    again = binding.qkv_rope_backward(*args, **kw)
    assert torch.equal(got, again[0])
    _clean()
    got = got.cpu().double()
    ang = rope_angles(s["positions"], s["inv_freq"], s["pair_axis"])
    at = 0
    for h, w, dy, dw, dw2 in ((hq, s["q_weight"], dys[0], dwq, again[1]),
                              (hkv, s["k_weight"], dys[1], dwk, again[2])):
        x = s["qkv"][:, at:at + h].double()
        okw = dict(eps=1e-5, interleaved=inter, amplitude=amp)
        ref, ref_w = oracle_rope_bwd(x, w, ang, dy, **okw)
        # magnitudes: |g| from |dy| of the pair, then the two terms of dx
        a, b = pair_dims(rotary, inter)
        mag = dy.double().abs()
        both = max(abs(amp), 1.0) * (mag[..., a] + mag[..., b])
        mag[..., a] = mag[..., b] = both
        size = mag
        if norm:
            inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)
            hm = mag * w.double().abs()
            size = inv * (hm + x.abs() * inv * inv * (hm * x.abs()).mean(-1, keepdim=True))
            bound = (2.0 ** -19 + t * h * 2.0 ** -24) * (mag * x.abs() * inv).sum((0, 1))
            assert ((dw.cpu().double() - ref_w).abs() <= bound).all()
            assert torch.equal(dw, dw2)
        err = (got[:, at:at + h] - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -19 * size).all(), err.max()
        at += h
    if not norm:
        assert dwq is None and dwk is None
    assert torch.equal(got[:, at:], dys[2].to(BF).double())


def test_rope_backward_against_differences():
    """Directional central differences of the kernel's own forward: L = <c, y>
    in 64 bits over bf16 results.  Each y is off by 2^-8 |y|, independently over
    1536 values of size 1, so L is off by about 2^-9 sqrt(1536) = 0.08 (rms),
    and a difference over 2h = 1 by sqrt(2) of that; eight of it are allowed."""
    hq, hkv, t = 4, 2, 4
    s = {k: _dev(v) for k, v in _rope_case(8, t, hq, hkv, 64, 1, True).items()}
    kw = dict(positions=s["positions"], inv_freq=s["inv_freq"], pair_axis=s["pair_axis"],
              heads_q=hq, heads_kv=hkv)
    c = [torch.randn(t, h, 64, device=DEV).to(BF) for h in (hq, hkv, hkv)]
    wq, wk = s["q_weight"], s["k_weight"]
    _, dwq, dwk = binding.qkv_rope_backward(s["qkv"], kw["positions"], kw["inv_freq"], *c,
                                            q_weight=wq, k_weight=wk, heads_q=hq, heads_kv=hkv,
                                            pair_axis=s["pair_axis"])

    def loss(a, b):
        ys = binding.qkv_rope(s["qkv"], q_weight=a, k_weight=b, **kw)
        return sum((y.double() * d.double()).sum().item() for y, d in zip(ys, c))

    for _ in range(3):
        da, db = torch.randn(64, device=DEV), torch.randn(64, device=DEV)
        num = loss(wq + 0.5 * da, wk + 0.5 * db) - loss(wq - 0.5 * da, wk - 0.5 * db)
        want = ((da * dwq).sum() + (db * dwk).sum()).item()
        assert abs(num - want) <= 8 * math.sqrt(2) * 0.08


def test_rope_autograd_and_broadcast_gradients():
    """Gradients reach the packed projection and both weights, through the
    attention as well, and a broadcast output gradient (sum().backward()) is
    taken as it is."""
    t, hq, hkv = 96, 4, 2
    s = {k: _dev(v) for k, v in _rope_case(2, t, hq, hkv, 64, 1, True, weight=BF).items()}
    leaves = [s[k].contiguous().requires_grad_() for k in ("qkv", "q_weight", "k_weight")]
    kw = dict(heads_q=hq, heads_kv=hkv, pair_axis=s["pair_axis"])
    q, k, v = binding.qkv_rope_autograd(leaves[0], s["positions"], s["inv_freq"],
                                        q_weight=leaves[1], k_weight=leaves[2], **kw)
    (q.sum() + v.sum()).backward()                      # k unused: zeros come in
    one = [torch.ones_like(q), torch.zeros_like(k), torch.ones_like(v)]
    ref = binding.qkv_rope_backward(leaves[0].detach(), s["positions"], s["inv_freq"], *one,
                                    q_weight=s["q_weight"], k_weight=s["k_weight"], **kw)
    assert torch.equal(leaves[0].grad, ref[0]) and torch.equal(leaves[1].grad, ref[1].to(BF))
    assert not leaves[2].grad.any()
    for x in leaves:
        x.grad = None
    q, k, v = binding.qkv_rope_autograd(leaves[0], s["positions"], s["inv_freq"],
                                        q_weight=leaves[1], k_weight=leaves[2], **kw)
    sink = torch.zeros(hq, device=DEV, requires_grad=True)
    out = binding.attn_sink(q[None], k[None], v[None], sink)
    out.float().square().sum().backward()
    for x in leaves + [sink]:
        assert torch.isfinite(x.grad.float()).all() and x.grad.float().abs().sum() > 0
    _clean()


# ----------------------------------------------------------------------------- extend
def _extend_case(seed, new, lens, page, hq, hkv, rows=None, fill=math.nan, evict=0):
    """Everything of the cache that no sequence holds is `fill`; `evict`: table
    entries of the first pages of each sequence are invalid (behind a window)."""
    g = torch.Generator().manual_seed(seed)
    count = [-(-n // page) for n in lens]
    perm = torch.randperm(sum(count) + 3, generator=g)
    shape = (len(perm), page, hkv, 64)
    kc, vc = torch.full(shape, fill).to(BF), torch.full(shape, fill).to(BF)
    table, at = torch.full((len(lens), max(count + [1])), -1, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        for p in range(count[b]):
            pg, m = int(perm[at + p]), min(page, n - p * page)
            table[b, p] = pg
            kc[pg, :m] = torch.randn(m, hkv, 64, generator=g).to(BF)
            vc[pg, :m] = torch.randn(m, hkv, 64, generator=g).to(BF)
        at += count[b]
        if evict:
            table[b, :max(0, (n - evict) // page)] = -1
    cu = torch.tensor([0] + new).cumsum(0).int()
    t = sum(new) if rows is None else rows
    q = torch.randn(t, hq, 64, generator=g).to(BF)
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32), cu, torch.randn(hq, generator=g)


def _check_extend(got, ref, used):
    out, lse = got[0].cpu().double(), got[1].cpu().double()
    ro, rl, spread = ref
    err = (out - ro).abs()[:used]
    bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -11) * spread
    assert (err <= bound[:used]).all(), (err - bound[:used]).max()
    assert torch.equal(torch.isneginf(lse[:, :used]), torch.isneginf(rl[:, :used]))
    fin = torch.isfinite(rl[:, :used])
    e = (lse[:, :used] - rl[:, :used])[fin].abs()
    assert (e <= 2.0 ** -13 + 2.0 ** -22 * rl[:, :used][fin].abs()).all(), e.max()


def _run_extend(c, window=0, scale=0.125, **kw):
    return binding.extend(*(x.to(DEV) for x in c), window=window, softmax_scale=scale, **kw)


EXTEND = [  # name, new, lens, page, hq, hkv, window
    ("one_token", [1], [1], 16, 8, 1, 0),
    ("ragged", [5, 1, 0, 17, 33], [300, 1, 40, 17, 1000], 16, 16, 2, 0),
    ("prompts", [130, 257], [130, 257], 64, 8, 2, 0),
    ("g1_page8", [200, 3], [700, 90], 8, 2, 2, 0),
    ("g3_page24", [43, 90], [500, 91], 24, 6, 2, 0),
    ("g5_page128", [25, 26, 51], [129, 128, 127], 128, 10, 2, 0),
    ("g128", [3, 1], [70, 200], 16, 128, 1, 0),
    ("g100", [2, 1], [70, 200], 16, 100, 1, 0),
    ("page1", [9, 40], [150, 333], 1, 8, 1, 0),
    ("page20_window", [9, 40], [150, 333], 20, 8, 2, 60),
    ("window1", [20, 3], [200, 3], 16, 8, 2, 1),
    ("window", [300, 7, 1], [900, 513, 129], 16, 8, 1, 128),
    ("window_long", [64], [3000], 32, 16, 2, 1000),
    ("more_new_than_keys", [40, 5, 3], [8, 0, 3], 16, 8, 2, 0),
    ("split", [2, 19], [6000, 9000], 16, 16, 2, 0),
    ("split_page4", [3], [5000], 4, 8, 1, 0),
    ("split_many_heads", [1, 1, 1], [4000, 100, 5000], 64, 64, 64, 0),
]


@pytest.mark.parametrize("name,new,lens,page,hq,hkv,window", EXTEND, ids=[c[0] for c in EXTEND])
def test_extend(name, new, lens, page, hq, hkv, window):
    c = _extend_case(len(name) + page, new, lens, page, hq, hkv)
    got = _run_extend(c, window)
    _clean()
    _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125,
                                     window=window), sum(new))
    again = _run_extend(c, window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_extend_leaves_the_rows_behind_the_last_sequence():
    c = _extend_case(4, [5, 20], [90, 20], 16, 8, 1, rows=64)
    out = torch.full((64, 8, 64), 7.0, dtype=BF, device=DEV)
    lse = torch.full((8, 64), 7.0, device=DEV)
    got = _run_extend(c, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert (out[25:] == 7).all() and (lse[:, 25:] == 7).all()
    _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125), 25)
    _clean()


@pytest.mark.parametrize("page", [16, 12])
def test_extend_window_does_not_need_evicted_pages(page):
    """Pages that lie behind every token's window may be gone."""
    c = _extend_case(6, [10, 3], [900, 400], page, 8, 2, evict=10 + 64)
    got = _run_extend(c, window=64)
    _clean()
    _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125,
                                     window=64), 13)


def test_extend_infinite_and_extreme_sinks():
    c = list(_extend_case(7, [4, 2], [50, 0], 16, 8, 2))
    c[6] = torch.tensor([-math.inf, -math.inf, 80.0, -80.0, 0.0, -30.0, 8.0, 30.0])
    got = _run_extend(c)
    _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125), 6)
    _clean()


@pytest.mark.parametrize("page", [16, 6])
def test_extend_bad_entries_are_reported_and_skipped(page):
    c = list(_extend_case(8, [9, 4], [200, 90], page, 8, 2))
    c[3] = c[3].clone()
    c[3][0, 2], c[3][1, 1] = c[1].shape[0] + 5, -3
    got = _run_extend(c)
    assert _code() == 0x800
    _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125), 13)
    # a length beyond the table is clamped to it, a negative one to 0
    cap = c[3].shape[1] * page
    c[4] = torch.tensor([cap + 999, -5], dtype=torch.int32)
    got = _run_extend(c)
    assert _code() == 0x800 and torch.equal(got[1][:, 9:].cpu(), c[6][:, None].expand(8, 4))
    # offsets beyond the rows of q, and descending ones
    for cu in ([0, 9, 400], [0, 30, 13], [-4, 3, 13]):
        c[5] = torch.tensor(cu, dtype=torch.int32)
        _run_extend(c)
        assert _code() == 0x800


def test_extend_agrees_with_decode():
    """One new token per sequence: the same attention as attn_sink_decode."""
    lens = [257, 64, 1, 3000]
    c = _extend_case(11, [1] * 4, lens, 16, 16, 2, fill=0.0)
    out, lse = _run_extend(c)
    q, kc, vc, table, ln, _, sink = (x.to(DEV) for x in c)
    od, ld, _ = binding.decode(q, kc, vc, table, ln, sink)
    assert (lse - ld).abs().max().item() <= 2.0 ** -12
    spread = oracle_extend(*c[:4], lens, c[5].tolist(), c[6], scale=0.125)[2]
    err = (out.double() - od.double()).abs().cpu()
    assert (err <= 2.0 ** -7 * od.double().abs().cpu() + 2.0 ** -7 * spread).all()
    _clean()


def test_extend_captured_and_replayed_with_other_lengths():
    """A captured step follows the lengths, tables and offsets that are in device
    memory at each replay; two graphs of their own workspaces run side by side."""
    cases = [_extend_case(20 + i, n, m, 16, 8, 2, rows=48) for i, (n, m) in enumerate(
        [([5, 1, 0], [300, 40, 9]), ([16, 16, 16], [16, 2000, 77]), ([0, 1, 47], [0, 5000, 47])])]
    pages = max(c[1].shape[0] for c in cases)
    cols = max(c[3].shape[1] for c in cases)

    def padded(c):
        kc = torch.zeros(pages, 16, 2, 64, dtype=BF)
        vc, table = torch.zeros_like(kc), torch.full((3, cols), -1, dtype=torch.int32)
        kc[:c[1].shape[0]], vc[:c[2].shape[0]], table[:, :c[3].shape[1]] = c[1], c[2], c[3]
        return (c[0], kc, vc, table, *c[4:])

    static = [[x.to(DEV) for x in padded(cases[0])] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for st, stream in zip(static, streams):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            binding.extend(*st)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs.append(binding.extend(*st))
            graphs.append(graph)
    torch.cuda.synchronize()
    for pick in ([1, 2], [2, 0], [0, 1]):
        for st, i in zip(static, pick):
            for dst, src in zip(st, padded(cases[i])):
                dst.copy_(src)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for got, i in zip(outs, pick):
            c = cases[i]
            _check_extend(got, oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6],
                                             scale=0.125), int(c[5][-1]))
    _clean()


def test_extend_on_a_stream_of_its_own():
    c = _extend_case(30, [7, 9], [500, 60], 16, 8, 2)
    ref = _run_extend(c)
    args = [x.to(DEV) for x in c]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for s in (stream, stream.cuda_stream, 0):
        got = binding.extend(*args, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    _clean()


@pytest.mark.parametrize("page", [16, 4])
def test_extend_wait_that_runs_out(page):
    """The test build withholds a key block: the call comes back with a timeout
    code, and later calls are clean."""
    from attention_learnable_head_gb300.build import build
    L = binding.load_library(build(test=True))
    c = [x.to(DEV) for x in _extend_case(31, [5, 40], [600, 700], page, 8, 2)]
    p = binding.AttnSinkExtendParams(2, 45, 8, 2, 64, page, c[1].shape[0], c[3].shape[1], 0, 0.125)
    out, lse = torch.zeros(45, 8, 64, dtype=BF, device=DEV), torch.zeros(8, 45, device=DEV)
    ws = torch.empty(L.attn_sink_extend_workspace_size(ctypes.byref(p)), dtype=torch.uint8,
                     device=DEV)
    stream = torch.cuda.current_stream().cuda_stream

    def run():
        return L.attn_sink_extend(ctypes.byref(p), *(x.data_ptr() for x in c), out.data_ptr(),
                                  lse.data_ptr(), ws.data_ptr(), ws.numel(), stream)

    def error():
        code = ctypes.c_int(0)
        return L.attn_sink_device_error(stream, ctypes.byref(code)), code.value

    assert run() == 0 and error() == (0, 0)
    ref = out.clone()
    L.attn_sink_test_withhold(1, -1)
    try:
        t0 = time.monotonic()
        assert run() == 0
        st, code = error()
        assert time.monotonic() - t0 < 2.0 and st == 5 and code & 0xF00 == 0x100
    finally:
        L.attn_sink_test_withhold(-1, -1)
    out.zero_()
    assert run() == 0 and error() == (0, 0) and torch.equal(out, ref)


# ----------------------------------------------------------------------------- together
def test_a_serving_run_gives_the_attention_of_the_whole_sequences():
    """Prompts in two chunks, then single tokens: plan, rope into the pages, and
    extend or decode; every output against the attention of the oracle over the
    whole sequence's rotated keys."""
    hq, hkv, page, pages, cols = 16, 2, 16, 64, 12
    g = torch.Generator().manual_seed(50)
    total, steps = [90, 41, 130], [[60, 0, 100], [28, 39, 29], [1, 1, 1], [1, 1, 0]]
    qkv = [torch.randn(n, hq + 2 * hkv, 64, generator=g).to(BF) for n in total]
    freq = 10000.0 ** (-torch.arange(32) / 32)
    wq, wk = (1 + 0.2 * torch.randn(64, generator=g) for _ in range(2))
    sink = torch.randn(hq, generator=g)
    free = torch.randperm(pages, generator=g).int().to(DEV)
    kc = torch.full((pages, page, hkv, 64), math.nan, dtype=BF, device=DEV)
    vc = torch.full_like(kc, math.nan)
    table = torch.full((3, cols), -1, dtype=torch.int32, device=DEV)
    cached = [0, 0, 0]
    # the keys as the kernel rounds them, from one pass over each whole sequence
    refs = []
    for x in qkv:
        q, k, v = binding.qkv_rope(x.to(DEV), torch.arange(len(x), dtype=torch.int32, device=DEV),
                                   freq.to(DEV), heads_q=hq, heads_kv=hkv, q_weight=wq.to(DEV),
                                   k_weight=wk.to(DEV))
        n = len(x)
        refs.append(oracle_extend(q.cpu(), k.cpu().view(1, n, hkv, 64), v.cpu().view(1, n, hkv, 64),
                                  torch.zeros(1, 1, dtype=torch.int32), [n], [0, n], sink,
                                  scale=0.125))
    for new in steps:
        pad = 5
        p = binding.page_plan(torch.tensor(cached, dtype=torch.int32, device=DEV),
                              torch.tensor(new, dtype=torch.int32, device=DEV), free, table,
                              page_size=page, num_pages=pages, max_tokens=sum(new) + pad)
        x = torch.cat([x[c:c + n] for x, c, n in zip(qkv, cached, new)] +
                      [torch.zeros(pad, hq + 2 * hkv, 64, dtype=BF)]).to(DEV)
        q, _, _ = binding.qkv_rope(x, p.positions, freq.to(DEV), heads_q=hq, heads_kv=hkv,
                                   q_weight=wq.to(DEV), k_weight=wk.to(DEV), slots=p.slots,
                                   k_cache=kc, v_cache=vc)
        out, lse = binding.extend(q, kc, vc, table, p.seq_lens, p.cu_seqlens_q, sink.to(DEV))
        at = 0
        for b, n in enumerate(new):
            rows = slice(cached[b], cached[b] + n)
            ref = (refs[b][0][rows], refs[b][1][:, rows], refs[b][2][rows])
            _check_extend((out[at:at + n], lse[:, at:at + n]), ref, n)
            at += n
        if new == [1, 1, 1]:
            kz, vz = torch.nan_to_num(kc), torch.nan_to_num(vc)
            od, _, _ = binding.decode(q[:3], kz, vz, table, p.seq_lens, sink.to(DEV))
            for b in range(3):
                ro, sp = refs[b][0][cached[b]], refs[b][2][cached[b]]
                e = (od[b].cpu().double() - ro).abs()
                assert (e <= 2.0 ** -8 * ro.abs() + 2.0 ** -10 * sp).all()
        free = free[p.pages_needed.item():].contiguous()
        cached = [c + n for c, n in zip(cached, new)]
        _clean()
    assert cached == total
