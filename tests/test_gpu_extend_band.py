"""Windowed attn_sink_extend calls on the band kernel (three launches: regions and
tiles, gather, band kernel), each padded with sequences so that it is taken.
Tolerances as in test_gpu_extend_window.py."""
import math

import pytest
import torch

from attention_learnable_head_gb300 import binding
from oracle.step import oracle_extend
from test_gpu_step import BF, DEV, _check_extend, _clean, _code, _extend_case, _run_extend

pytestmark = pytest.mark.gpu


def _band(run):
    """What `run` returns; it has to be a call on the band kernel."""
    n = binding.attn_sink_launch_count()
    r = run()
    assert binding.attn_sink_launch_count() - n == 3
    return r


def _oracle(c, window):
    return oracle_extend(*c[:4], c[4].tolist(), c[5].tolist(), c[6], scale=0.125, window=window)


def test_lse_of_partial_tiles_is_the_same_every_time():
    """Every tile is partial and every CTA has several: the sums of a row's halves
    must not be overwritten by the next tile's before both have been read, also in a
    CTA's last pass."""
    new = [8 + i % 7 for i in range(420)]
    c = _extend_case(1, new, [n + i * 37 % 300 for i, n in enumerate(new)], 16, 16, 2)
    d = [x.to(DEV) for x in c]
    first = _band(lambda: binding.extend(*d, window=128))
    _check_extend(first, _oracle(c, 128), sum(new))
    for _ in range(300):
        out, lse = binding.extend(*d, window=128)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    _clean()


def test_extreme_sinks():
    """A sink far above the scores leaves the probabilities their bits: out is small, not
    zero."""
    c = list(_extend_case(2, [40] + [12] * 130, [300] + [12 + i for i in range(130)], 16, 8, 2))
    c[6] = torch.tensor([-math.inf, 80.0, 30.0, 17.0, 12.0, 8.0, -30.0, 0.0])
    got = _band(lambda: _run_extend(c, 100))
    ref = _oracle(c, 100)
    _check_extend(got, ref, 40 + 12 * 130)
    assert got[0][:, 2].any() and got[0][:, 3].any() and (ref[0][:, 1].abs().max() > 0)
    _clean()


@pytest.mark.parametrize("window", [100, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf, 1e6])
def test_values_behind_a_tile_do_not_reach_it(window, value):
    """The box of a tile's keys is rounded up to 16: the rows behind its last key hold
    values of later tokens, which no token of the tile sees."""
    new, lens = [40] + [12] * 130, [300] + [12] * 130
    c = _extend_case(3, new, lens, 16, 16, 2, fill=0.0)
    j = 300 - 40 + 16                      # the first token of the second tile of 16
    ref = _oracle(c, window)               # (in sums of the oracle 0 * inf is not 0 either)
    page = int(c[3][0, j // 16])
    c[1][page, j % 16], c[2][page, j % 16] = value, value
    got = _band(lambda: _run_extend(c, window))
    assert _code() == (0 if math.isnan(value) else 0x400)
    for a, b in ((0, 16), (40, sum(new))):
        _check_extend((got[0][a:b], got[1][:, a:b]),
                      (ref[0][a:b], ref[1][:, a:b], ref[2][a:b]), b - a)


def test_a_nan_score_gives_a_nan_lse():
    """-inf is the mark of a row without keys."""
    c = _extend_case(6, [40] + [12] * 130, [300] + [12] * 130, 16, 8, 2, fill=0.0)
    j = 300 - 20
    c[1][int(c[3][0, j // 16]), j % 16, 1] = math.nan
    out, lse = _band(lambda: _run_extend(c, 100))
    seen = torch.zeros(8, 40 + 12 * 130, dtype=torch.bool)
    seen[4:, 20:40] = True                 # tokens from that key on, heads of kv head 1
    assert torch.equal(lse.isnan().cpu(), seen)
    assert torch.equal(out.isnan().all(-1).cpu(), seen.T)
    assert torch.equal(out.isnan().any(-1).cpu(), seen.T)
    _clean()


@pytest.mark.parametrize("page", [16, 12])
def test_keys_without_a_page_are_skipped(page):
    """As on the general kernel: such a key takes no weight."""
    new, lens = [70, 40] + [12] * 130, [200, 190] + [12 + i for i in range(130)]
    c = list(_extend_case(4, new, lens, page, 8, 2))
    c[3] = c[3].clone()
    for b, j in ((0, 199), (0, 120), (1, 150), (1, 151 + page), (9, 3), (50, 40)):
        c[3][b, j // page] = -1
    c[3][0, 140 // page] = c[1].shape[0]
    got = _band(lambda: _run_extend(c, 100))
    assert _code() == 0x800
    _check_extend(got, _oracle(c, 100), sum(new))
    # none of the keys of a token is left
    c[3][:] = -1
    got = _band(lambda: _run_extend(c, 100))
    assert _code() == 0x800 and not got[0].any()
    _check_extend(got, _oracle(c, 100), sum(new))
    c = _extend_case(5, new, lens, page, 8, 2)
    _check_extend(_band(lambda: _run_extend(c, 100)), _oracle(c, 100), sum(new))
    _clean()


def test_both_ways_agree_on_the_same_tokens():
    """The same sequences in one call on the band kernel and alone on the general one."""
    new, lens = [96, 41, 130] + [12] * 130, [1000, 41, 777] + [12 + 5 * i for i in range(130)]
    c = _extend_case(7, new, lens, 16, 8, 2)
    d = [x.to(DEV) for x in c]
    out, lse = _band(lambda: binding.extend(*d, window=100))
    ref = _oracle(c, 100)
    for b in (0, 1, 2, 80):
        a, e = int(c[5][b]), int(c[5][b + 1])
        before = binding.attn_sink_launch_count()
        one = binding.extend(d[0][a:e], d[1], d[2], d[3][b:b + 1].contiguous(), d[4][b:b + 1],
                             torch.tensor([0, e - a], dtype=torch.int32, device=DEV), d[6], window=100)
        assert binding.attn_sink_launch_count() - before == 1
        # P in fp16 and in bf16, the output in bf16 twice
        spread = ref[2][a:e]
        err = (out[a:e].double() - one[0].double()).abs().cpu()
        assert (err <= 2.0 ** -7 * ref[0][a:e].abs() + (2.0 ** -8 + 2.0 ** -10) * spread).all()
        assert (lse[:, a:e] - one[1]).abs().max() <= 2.0 ** -12
    _clean()


def test_far_rows_are_gathered():
    """Pages whose offsets pass 32 bits, shared by all sequences."""
    hkv, page, n = 8, 16, 40
    pages = (1 << 32) // (page * hkv * 64) + 2048
    kc = torch.empty(pages, page, hkv, 64, dtype=BF, device=DEV)
    vc = torch.empty_like(kc)
    near = [torch.randn(3, page, hkv, 64, device=DEV).to(BF) for _ in range(2)]
    kc[-3:], vc[-3:] = near[0], near[1]
    i32 = dict(dtype=torch.int32, device=DEV)
    lens, cu = torch.full((131,), n, **i32), torch.arange(132, **i32) * n
    q = torch.randn(131 * n, 64, 64, device=DEV).to(BF)
    sink = torch.randn(64, device=DEV)
    far = torch.arange(pages - 3, pages, **i32).expand(131, 3).contiguous()
    a = _band(lambda: binding.extend(q, kc, vc, far, lens, cu, sink, window=100))
    b = _band(lambda: binding.extend(q, *near, torch.arange(3, **i32).expand(131, 3).contiguous(),
                                     lens, cu, sink, window=100))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = (q, *near, torch.arange(3, **i32)[None].expand(131, 3), lens, cu, sink)
    c = [x.cpu() for x in c]
    part = oracle_extend(c[0][:n], c[1], c[2], c[3][:1], [n], [0, n], c[6], scale=0.125, window=100)
    _check_extend((a[0][:n], a[1][:, :n]), part, n)
    _clean()


@pytest.mark.parametrize("cu", [{2: 4000}, {1: 300}, {0: -4}, {3: 0, 60: 10 ** 6}, {131: 1 << 30}])
def test_bad_lists_of_sequences(cu):
    """Offsets that descend or lie outside q are recorded as such, nothing outside the
    outputs is touched, and the next call is right."""
    new, lens = [70, 100] + [12] * 130, [200, 190] + [12] * 130
    n = sum(new)
    c = list(_extend_case(8, new, lens, 16, 8, 2))
    good = c[5]
    c[5] = good.clone()
    for at, x in cu.items():
        c[5][at] = x
    room = torch.full((3, n, 8, 64), 7.0, dtype=BF, device=DEV)
    rest = torch.full((3, 8, n), 7.0, device=DEV)
    _band(lambda: _run_extend(c, 100, out=room[1], lse=rest[1]))
    assert _code() == 0x800
    for x in (room, rest):
        assert (x[0] == 7).all() and (x[2] == 7).all()
    c[5] = good
    _check_extend(_band(lambda: _run_extend(c, 100)), _oracle(c, 100), n)
    _clean()


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -20, 2.0 ** -30])
def test_small_values(size):
    """Values below 2^-14 are rounded to multiples of 2^-24 here: off by 2^-25."""
    new, lens = [40] + [12] * 130, [300] + [12 + i for i in range(130)]
    c = list(_extend_case(9, new, lens, 16, 8, 2, fill=0.0))
    c[2] = (c[2].float() * size).to(BF)
    got = _band(lambda: _run_extend(c, 100))
    ref = _oracle(c, 100)
    err = (got[0].cpu().double() - ref[0]).abs()
    assert (err <= 2.0 ** -8 * ref[0].abs() + (2.0 ** -8 + 2.0 ** -11) * ref[2] + 2.0 ** -25).all()
    _clean()


def test_a_wait_that_runs_out():
    """The test build withholds a tile's keys: the call comes back with a timeout code,
    and later calls are clean."""
    import ctypes
    import time

    from attention_learnable_head_gb300.build import build
    L = binding.load_library(build(test=True))
    new, lens = [40] * 140, [60 + i for i in range(140)]
    c = [x.to(DEV) for x in _extend_case(31, new, lens, 16, 16, 2)]
    n = sum(new)
    p = binding.AttnSinkExtendParams(140, n, 16, 2, 64, 16, c[1].shape[0], c[3].shape[1], 100, 0.125)
    out, lse = torch.zeros(n, 16, 64, dtype=BF, device=DEV), torch.zeros(16, n, device=DEV)
    ws = torch.empty(L.attn_sink_extend_workspace_size(ctypes.byref(p)), dtype=torch.uint8,
                     device=DEV)
    stream = torch.cuda.current_stream().cuda_stream

    def run():
        before = L.attn_sink_launch_count()
        st = L.attn_sink_extend(ctypes.byref(p), *(x.data_ptr() for x in c), out.data_ptr(),
                                lse.data_ptr(), ws.data_ptr(), ws.numel(), stream)
        assert L.attn_sink_launch_count() - before == 3
        return st

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
