"""The entry points of attn_sink_cache.h without a GPU: exported, mirrored, and refusing
bad arguments on the host with the documented status and no launch."""
import ctypes
import math

import pytest
import torch

from attention_learnable_head_gb300 import binding
from attention_learnable_head_gb300.build import build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x7F0000000000       # never dereferenced: validation fails first

PARAMS = dict(
    decode_shared=(binding.AttnSinkSharedParams,
                   dict(batch=4, num_groups=2, heads_q=16, heads_kv=2, head_dim=64, page_size=16,
                        num_pages=64, max_pages=8, softmax_scale=0.125)),
    page_bounds=(binding.AttnSinkBoundsParams,
                 dict(batch=4, heads_kv=2, head_dim=64, page_size=16, num_pages=64, max_pages=8)),
    select_pages=(binding.AttnSinkSelectParams,
                  dict(batch=4, heads_q=16, heads_kv=2, head_dim=64, page_size=16, num_pages=64,
                       max_pages=8, count=4, keep_first=1, keep_last=1)),
    decode_pages=(binding.AttnSinkPagesParams,
                  dict(batch=4, heads_q=16, heads_kv=2, head_dim=64, page_size=16, num_pages=64,
                       max_pages=8, count=4, softmax_scale=0.125)),
    key_mass=(binding.AttnSinkMassParams,
              dict(batch=4, total_q=9, heads_q=16, heads_kv=2, head_dim=64, page_size=16,
                   num_pages=64, max_pages=8, max_keys=128, accumulate=1, softmax_scale=0.125)),
    evict=(binding.AttnSinkEvictParams,
           dict(batch=4, heads_kv=2, head_dim=64, page_size=16, num_pages=64, max_pages=8,
                max_keys=128, budget=50, keep_first=2, keep_last=8, max_freed=32)))
POINTERS = dict(
    decode_shared=["q", "k", "v", "table", "lens", "groups", "prefix", "sink", "out", "lse"],
    page_bounds=["k", "table", "cached", "lens", "bounds"],
    select_pages=["q", "bounds", "table", "lens", "selected"],
    decode_pages=["q", "k", "v", "table", "lens", "selected", "sink", "out", "lse"],
    key_mass=["q", "k", "table", "lens", "cu", "lse", "mass"],
    evict=["k", "v", "table", "lens", "mass", "mass_out", "new_lens", "freed", "count"])
WORK = {"decode_shared", "select_pages", "decode_pages", "evict"}
ALIGNED = {"q", "k", "v", "out", "bounds"}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    return binding.lib()


@pytest.fixture(autouse=True)
def _no_launch():
    n0 = binding.attn_sink_launch_count()
    yield
    assert binding.attn_sink_launch_count() == n0


def _params(name, **kw):
    kind, fields = PARAMS[name]
    return kind(*{**fields, **kw}.values())


def _call(name, params, ws=FAKE, ws_bytes=1 << 40, **kw):
    at = {p: FAKE + 4096 * i for i, p in enumerate(POINTERS[name])}
    at.update(kw)
    work = [ws, ws_bytes] if name in WORK else []
    return getattr(binding, "attn_sink_" + name)(params, *at.values(), *work, stream=0)


def _workspace(name, params):
    return getattr(binding, f"attn_sink_{name}_workspace_size")(params) if name in WORK else 0


def test_exports_every_declared_symbol():
    names = binding.header_functions("attn_sink_cache.h")
    assert set(names) == ({"attn_sink_" + n for n in PARAMS} |
                          {f"attn_sink_{n}_workspace_size" for n in WORK})
    for n in names:
        assert hasattr(binding.lib(), n) and hasattr(binding, n), n


def test_struct_layouts():
    for name, (kind, fields) in PARAMS.items():
        assert ctypes.sizeof(kind) == 4 * len(fields)
        assert [f for f, _ in kind._fields_] == list(fields)


COMMON = [("batch", -1, INVALID), ("batch", (1 << 24) + 1, UNSUPPORTED), ("heads_kv", 0, INVALID),
          ("head_dim", 128, UNSUPPORTED), ("page_size", 0, INVALID), ("num_pages", -1, INVALID),
          ("num_pages", 1 << 27, UNSUPPORTED), ("max_pages", -1, INVALID),
          ("max_pages", 1 << 27, INVALID)]
GROUP = [("heads_q", 15, INVALID), ("heads_q", 0, INVALID), ("heads_q", 6, UNSUPPORTED),
         ("heads_q", 32, UNSUPPORTED)]
SCALE = [("softmax_scale", x, INVALID) for x in (0.0, -1.0, math.inf, math.nan)]


@pytest.mark.parametrize("name,field,value,status", [
    *[(n, *c) for n in PARAMS for c in COMMON],
    *[(n, *c) for n in ("decode_shared", "select_pages", "decode_pages") for c in GROUP],
    *[(n, *c) for n in ("decode_shared", "decode_pages", "key_mass") for c in SCALE],
    ("decode_shared", "num_groups", 5, INVALID), ("decode_shared", "num_groups", 0, INVALID),
    ("decode_shared", "num_groups", -1, INVALID), ("decode_shared", "batch", 65536, UNSUPPORTED),
    ("select_pages", "count", 0, INVALID), ("select_pages", "keep_first", -1, INVALID),
    ("select_pages", "keep_last", -1, INVALID), ("select_pages", "keep_first", 4, INVALID),
    ("select_pages", "keep_last", 2 ** 31 - 1, INVALID),
    ("decode_pages", "count", -1, INVALID), ("decode_pages", "count", 1 << 27, INVALID),
    ("key_mass", "total_q", -1, INVALID), ("key_mass", "total_q", (1 << 30) + 1, UNSUPPORTED),
    ("key_mass", "heads_q", 2 * 129, UNSUPPORTED), ("key_mass", "heads_q", 3, INVALID),
    ("key_mass", "max_keys", -1, INVALID), ("key_mass", "max_keys", (1 << 30) + 1, UNSUPPORTED),
    ("key_mass", "accumulate", 2, INVALID),
    ("evict", "budget", -1, INVALID), ("evict", "budget", 9, INVALID),
    ("evict", "keep_first", -1, INVALID), ("evict", "keep_last", -1, INVALID),
    ("evict", "keep_last", 2 ** 31 - 1, INVALID), ("evict", "max_freed", -1, INVALID),
    ("evict", "max_keys", -1, INVALID), ("evict", "max_keys", (1 << 30) + 1, UNSUPPORTED)])
def test_rejects_bad_params(name, field, value, status):
    p = _params(name, **{field: value})
    assert _call(name, p) == status
    assert _workspace(name, p) == 0


@pytest.mark.parametrize("name", PARAMS)
def test_rejects_null_and_misaligned_pointers(name):
    for p in POINTERS[name]:
        assert _call(name, _params(name), **{p: None}) == INVALID, p
    for p in ALIGNED & set(POINTERS[name]):
        assert _call(name, _params(name), **{p: FAKE + 8}) == INVALID, p
    assert _call(name, None) == INVALID


@pytest.mark.parametrize("name", sorted(WORK))
def test_rejects_a_bad_workspace(name):
    p = _params(name)
    need = _workspace(name, p)
    assert need > 0
    assert _call(name, p, ws=None) == WORKSPACE
    assert _call(name, p, ws=FAKE + 16) == WORKSPACE
    assert _call(name, p, ws_bytes=need - 1) == WORKSPACE


def test_evict_rejects_outputs_in_place():
    p = _params("evict")
    assert _call("evict", p, mass_out=FAKE, mass=FAKE) == INVALID
    assert _call("evict", p, new_lens=FAKE, lens=FAKE) == INVALID


@pytest.mark.parametrize("name", [n for n in PARAMS if n != "evict"])
def test_no_sequence_is_nothing_to_do(name):
    p = _params(name, batch=0, **({"num_groups": 0} if name == "decode_shared" else {}))
    assert _call(name, p) == OK
    assert _workspace(name, p) == 0


def test_conveniences_name_what_is_wrong():
    """The Python checks, on tensors that are on no GPU."""
    bf16 = torch.bfloat16
    q, k = torch.zeros(2, 8, 64, dtype=bf16), torch.zeros(4, 16, 2, 64, dtype=bf16)
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cu, sink = torch.zeros(2, dtype=torch.int32), torch.zeros(8)
    bounds = torch.zeros(4, 2, 2, 64, dtype=bf16)
    sel = torch.zeros(2, 2, 4, dtype=torch.int32)
    mass, lse = torch.zeros(2, 2, 48), torch.zeros(8, 2)
    cu3 = torch.zeros(3, dtype=torch.int32)
    calls = [
        (lambda **kw: binding.decode_shared(**{**dict(
            q=q, k_cache=k, v_cache=k, block_table=table, seq_lens=lens, cu_groups=cu,
            prefix_lens=cu[:1], sink=sink), **kw}),
         dict(q=q.float(), k_cache=k[:, :, :1], v_cache=k[:1], block_table=table.long(),
              seq_lens=lens[:1], cu_groups=cu3, prefix_lens=cu.float(), sink=sink.to(bf16),
              out=q[:1], lse=lse[:1])),
        (lambda **kw: binding.page_bounds(**{**dict(
            k_cache=k, block_table=table, cached_lens=lens, seq_lens=lens, bounds=bounds), **kw}),
         dict(k_cache=k.float(), cached_lens=lens[:1], bounds=bounds[:, :1], seq_lens=table)),
        (lambda **kw: binding.select_pages(**{**dict(
            q=q, bounds=bounds, block_table=table, seq_lens=lens, count=4, page_size=16), **kw}),
         dict(q=q[:1], bounds=bounds[:, :, :1], block_table=table[:1], count=0,
              page_size=2 ** 31)),
        (lambda **kw: binding.decode_pages(**{**dict(
            q=q, k_cache=k, v_cache=k, block_table=table, seq_lens=lens, selected=sel,
            sink=sink), **kw}),
         dict(q=q[0], selected=sel[:, :1], sink=sink[:4], out=q.float(), lse=lse.double())),
        (lambda **kw: binding.key_mass(**{**dict(
            q=q, k_cache=k, block_table=table, seq_lens=lens, cu_seqlens_q=cu3, lse=lse,
            mass=mass), **kw}),
         dict(q=q.float(), cu_seqlens_q=cu, lse=lse[:, :1], mass=mass[:, :1])),
        (lambda **kw: binding.evict(**{**dict(
            k_cache=k, v_cache=k, block_table=table, seq_lens=lens, mass=mass, budget=16), **kw}),
         dict(v_cache=k[:1], mass=mass.double(), budget=2 ** 31))]
    for call, wrong in calls:
        for name, value in wrong.items():
            with pytest.raises(ValueError):
                call(**{name: value})
        with pytest.raises(ValueError, match="CUDA device"):
            call()
