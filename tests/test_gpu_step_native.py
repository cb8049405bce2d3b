"""The conveniences of attn_sink_step.h take a plain call through the native module
(csrc/fast_calls.cpp) and any other through Python; both have to give the same."""
import pytest
import torch

from attention_learnable_head_gb300 import binding
from test_gpu_step import BF, DEV, _clean, _dev, _rope_case

pytestmark = pytest.mark.gpu

PLAIN = dict(page_plan=5, qkv_rope=3, qkv_rope_backward=3, extend=2)   # results of each


def _same(name, run):
    """The call with no stream given (native) and with the current one given
    (Python): equal results, and only the first asks the native module."""
    native, asked = binding._fast(), []

    class Spy:
        def __getattr__(self, attr):
            def call(*args):
                r = getattr(native, attr)(*args)
                asked.append((attr, r))
                return r
            return call
    binding._FAST = Spy()
    try:
        a, b = run(None), run(torch.cuda.current_stream())
    finally:
        binding._FAST = native
    assert [n for n, _ in asked] == [name] and len(asked[0][1]) == PLAIN[name]
    assert len(a) == len(b) == PLAIN[name]
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype == y.dtype and x.is_contiguous() and torch.equal(x, y)
    _clean()


@pytest.mark.parametrize("batch", [0, 1, 300])
def test_page_plan(batch):
    i32 = dict(dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(batch)
    cached = torch.randint(0, 90, (batch,), generator=g).int().to(DEV)
    new = torch.randint(0, 40, (batch,), generator=g).int().to(DEV)
    table = torch.arange(batch * 9, **i32).view(batch, 9)
    free = torch.arange(batch * 9, batch * 18, **i32)
    tables = []

    def run(stream):
        tables.append(table.clone())
        return binding.page_plan(cached, new, free, tables[-1], page_size=16,
                                 num_pages=max(batch, 1) * 18, max_tokens=batch * 40 + 3,
                                 stream=stream)
    _same("page_plan", run)
    assert torch.equal(*tables)


@pytest.mark.parametrize("weight", [torch.float32, BF, None])
@pytest.mark.parametrize("tokens,axes,rows,interleaved", [
    (0, 1, 10, False), (1, 1, 10, True), (37, 3, 13, False), (200, 2, 10, True)])
def test_rope(tokens, axes, rows, interleaved, weight):
    s = {k: _dev(v) for k, v in _rope_case(tokens, tokens, 6, 2, 64, axes, True).items()}
    wide = torch.randn(tokens, rows, 64, device=DEV).to(BF)
    qkv = wide[:, :10]                                     # rows of tokens further apart
    w = dict.fromkeys(("q_weight", "k_weight"))
    if weight is not None:
        w = {k: s[k].to(weight) for k in w}
    pair_axis = None if axes == 1 else [i % axes for i in range(32)]
    kw = dict(heads_q=6, heads_kv=2, pair_axis=pair_axis, interleaved=interleaved, amplitude=1.25,
              eps=1e-5, **w)
    args = (qkv, s["positions"], s["inv_freq"])
    _same("qkv_rope", lambda st: binding.qkv_rope(*args, **kw, stream=st))
    slots = torch.randperm(256, device=DEV)[:tokens]
    for keep in (None, True):
        caches = []

        def run(stream):
            caches.append([torch.zeros(16, 16, 2, 64, dtype=BF, device=DEV) for _ in "kv"])
            return binding.qkv_rope(*args, **kw, slots=slots, k_cache=caches[-1][0],
                                    v_cache=caches[-1][1], keep_kv=keep, stream=stream)
        _same("qkv_rope", run)
        assert all(torch.equal(x, y) for x, y in zip(*caches))
    for kind in (BF, torch.float32):
        d = [torch.randn(tokens, h, 64, device=DEV).to(kind) for h in (6, 2, 2)]
        _same("qkv_rope_backward", lambda st: binding.qkv_rope_backward(*args, *d, **kw, stream=st))


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("window", [0, 40])
def test_extend(window, given):
    i32 = dict(dtype=torch.int32, device=DEV)
    q = torch.randn(70, 8, 64, device=DEV).to(BF)
    kc, vc = (torch.randn(20, 16, 2, 64, device=DEV).to(BF) for _ in "kv")
    args = (q, kc, vc, torch.arange(20, **i32).view(2, 10), torch.tensor([150, 31], **i32),
            torch.tensor([0, 50, 70], **i32), torch.randn(8, device=DEV))

    def run(stream):
        room = {}
        if given:
            room = dict(out=torch.zeros(70, 8, 64, dtype=BF, device=DEV),
                        lse=torch.zeros(8, 70, device=DEV))
        r = binding.extend(*args, window=window, softmax_scale=0.2, stream=stream, **room)
        assert not given or (r[0].data_ptr() == room["out"].data_ptr()
                             and r[1].data_ptr() == room["lse"].data_ptr())
        return r
    _same("extend", run)


def test_errors_name_the_argument_or_the_status():
    """A refusal by the library comes back as its exception, and what the native
    module does not take is named by the Python checks."""
    i32 = dict(dtype=torch.int32, device=DEV)
    one = torch.ones(1, **i32)
    with pytest.raises(RuntimeError, match="attn_sink_page_plan"):
        binding.page_plan(one, one, one, one.view(1, 1), page_size=0, num_pages=4, max_tokens=1)
    with pytest.raises(ValueError, match="new_lens"):
        binding.page_plan(one, one.long(), one, one.view(1, 1), page_size=16, num_pages=4,
                          max_tokens=1)
    qkv, freq = torch.zeros(1, 3, 64, dtype=BF, device=DEV), torch.ones(32, device=DEV)
    with pytest.raises(ValueError, match="pair_axis"):
        binding.qkv_rope(qkv, one, freq, heads_q=1, heads_kv=1, pair_axis=[1] * 32)
    with pytest.raises(ValueError, match="k_cache"):
        binding.qkv_rope(qkv, one, freq, heads_q=1, heads_kv=1, slots=one.long())
    with pytest.raises(RuntimeError, match="attn_sink_extend"):
        binding.extend(qkv[:, :1].contiguous(), qkv[None], qkv[None], one.view(1, 1), one,
                       torch.tensor([0, 1], **i32), torch.zeros(1, device=DEV), window=-1)
    _clean()


def test_another_stream_is_used():
    """Inside torch.cuda.stream the call goes to that stream: its outputs are those
    of inputs that the stream wrote just before."""
    i32 = dict(dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    qkv = torch.zeros(4096, 48, 64, dtype=BF, device=DEV)
    freq, pos = torch.ones(32, device=DEV), torch.zeros(4096, **i32)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.randn(8192, 8192, device=DEV)
        for _ in range(4):
            big = big @ big * 1e-2                        # keeps the stream busy
        qkv.fill_(1.0)
        q, _, _ = binding.qkv_rope(qkv, pos, freq, heads_q=32, heads_kv=8)
    side.synchronize()
    assert (q == 1).all()
    _clean()


def test_out_of_memory_is_an_exception():
    """An allocation that fails in the native module raises torch's own error, and
    the next call works."""
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    kw = dict(page_size=16, num_pages=4)
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.01)
    try:
        with pytest.raises(torch.cuda.OutOfMemoryError):
            binding.page_plan(one, one, one, one.view(1, 1), max_tokens=1 << 30, **kw)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert binding.page_plan(one, one, one, one.view(1, 1), max_tokens=1, **kw).slots.tolist() == [17]
    _clean()


def test_threads_share_the_module():
    """Calls from several threads, each on a stream of its own."""
    import threading

    s = {k: _dev(v) for k, v in _rope_case(5, 400, 8, 2, 64, 1, True).items()}
    want = binding.qkv_rope(**s, heads_q=8, heads_kv=2)
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = binding.qkv_rope(**s, heads_q=8, heads_kv=2)
            torch.cuda.current_stream().synchronize()
            bad.extend(not torch.equal(a, b) for a, b in zip(got, want))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(bad) == 12 and not any(bad)
    _clean()
