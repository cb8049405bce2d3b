"""The entry points of attn_sink_step.h without a GPU: exported, mirrored, and
refusing bad arguments on the host with the documented status and no launch."""
import ctypes
import math

import pytest
import torch

from attention_learnable_head_gb300 import binding
from attention_learnable_head_gb300.build import build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x7F0000000000       # never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    return binding.lib()


@pytest.fixture(autouse=True)
def _no_launch():
    n0 = binding.attn_sink_launch_count()
    yield
    assert binding.attn_sink_launch_count() == n0


def test_exports_every_declared_symbol():
    names = binding.header_functions("attn_sink_step.h")
    assert set(names) == {"attn_sink_page_plan", "attn_sink_qkv_rope",
                          "attn_sink_qkv_rope_bwd_workspace_size", "attn_sink_qkv_rope_bwd",
                          "attn_sink_extend_workspace_size", "attn_sink_extend"}
    for n in names:
        assert hasattr(binding.lib(), n) and hasattr(binding, n), n


def test_struct_layouts():
    assert ctypes.sizeof(binding.AttnSinkPlanParams) == 24
    assert ctypes.sizeof(binding.AttnSinkRopeParams) == 24 + 7 * 4 + 32 + 7 * 4
    assert ctypes.sizeof(binding.AttnSinkExtendParams) == 40


# ----------------------------------------------------------------------------- plan
def _plan(p=(), **kw):
    f = dict(batch=4, page_size=16, num_pages=64, max_pages=8, num_free=10, max_tokens=32)
    f.update(p)
    a = dict(cached=FAKE, new=FAKE, free=FAKE, table=FAKE, slots=FAKE, pos=FAKE, cu=FAKE,
             lens=FAKE + 4096, needed=FAKE)
    a.update(kw)
    return binding.attn_sink_page_plan(binding.AttnSinkPlanParams(*f.values()), *a.values(),
                                       stream=0)


@pytest.mark.parametrize("field,value", [
    ("batch", -1), ("page_size", 0), ("num_pages", -1), ("max_pages", -1), ("num_free", -1),
    ("max_tokens", -1), ("max_pages", 1 << 27)])
def test_plan_rejects_bad_params(field, value):
    assert _plan({field: value}) == INVALID


@pytest.mark.parametrize("name", ["cached", "new", "free", "table", "slots", "pos", "cu", "lens",
                                  "needed"])
def test_plan_rejects_null_pointers(name):
    assert _plan(**{name: None}) == INVALID


def test_plan_rejects_misaligned_slots_and_null_params():
    assert _plan(slots=FAKE + 4) == INVALID
    assert binding.attn_sink_page_plan(None, *[FAKE] * 9, stream=0) == INVALID


@pytest.mark.parametrize("name", ["cached", "new"])
def test_plan_rejects_lengths_in_place(name):
    assert _plan(**{name: FAKE + 4096}) == INVALID


# ----------------------------------------------------------------------------- rope
def _rope_params(**kw):
    p = binding.make_rope_params(16, 8, 2, rotary_dim=64, row_stride=12 * 64, norm=True)
    for k, v in kw.items():
        if k == "axis":
            p.pair_axis[5] = v
        else:
            setattr(p, k, v)
    return p


def _rope(p, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, pos=FAKE, freq=FAKE, qw=FAKE, kw=FAKE, slots=None, qo=FAKE,
             ko=FAKE, vo=FAKE, kc=None, vc=None)
    a.update(kw)
    return binding.attn_sink_qkv_rope(p, *a.values(), stream=0)


def _rope_bwd(p, strides=(768, 768, 768), ws=FAKE, ws_bytes=1 << 30, **kw):
    a = dict(q=FAKE, k=FAKE, pos=FAKE, freq=FAKE, qw=FAKE, kw=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
             dqi=FAKE, dki=FAKE, dvi=FAKE)
    b = dict(dqw=FAKE, dkw=FAKE)
    for k, v in kw.items():
        (b if k in b else a)[k] = v
    return binding.attn_sink_qkv_rope_bwd(p, *a.values(), *strides, *b.values(), ws, ws_bytes,
                                          stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=128), UNSUPPORTED), (dict(rotary_dim=8), UNSUPPORTED),
    (dict(rotary_dim=50), UNSUPPORTED), (dict(rotary_dim=80), INVALID),
    (dict(rotary_dim=-16), INVALID), (dict(tokens=-1), INVALID), (dict(heads_q=0), INVALID),
    (dict(heads_kv=0), INVALID), (dict(interleaved=2), INVALID), (dict(norm=2), INVALID),
    (dict(weight_bf16=-1), INVALID), (dict(num_axes=0), INVALID), (dict(num_axes=5), INVALID),
    (dict(axis=1), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.nan), INVALID),
    (dict(amplitude=math.inf), INVALID)])
def test_rope_rejects_bad_params(kw, status):
    p = _rope_params(**kw)
    assert _rope(p) == status
    assert _rope_bwd(p) == status
    assert binding.attn_sink_qkv_rope_bwd_workspace_size(p) == 0


def test_rope_rejects_bad_strides_and_pointers():
    for kw in (dict(q_stride=768 + 4), dict(q_stride=448), dict(k_stride=64), dict(v_stride=0),
               dict(q_stride=-768)):
        assert _rope(_rope_params(**kw)) == INVALID, kw
    for name in ("q", "k", "v", "pos", "freq", "qw", "kw", "qo"):
        assert _rope(_rope_params(), **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "qo", "ko", "vo"):
        assert _rope(_rope_params(), **{name: FAKE + 8}) == INVALID, name
    assert _rope(None) == INVALID
    assert _rope(_rope_params(tokens=0), q=None, k=None, v=None, qo=None) == OK
    # a cache needs its sizes and its tensors
    assert _rope(_rope_params(), slots=FAKE, kc=FAKE, vc=FAKE) == INVALID
    paged = _rope_params(page_size=16, num_pages=4)
    assert _rope(paged, slots=FAKE, kc=None, vc=FAKE) == INVALID
    assert _rope(paged, slots=FAKE, kc=FAKE, vc=FAKE + 8) == INVALID
    assert _rope(paged, slots=FAKE + 4, kc=FAKE, vc=FAKE) == INVALID


def test_rope_bwd_rejects_bad_arguments():
    p = _rope_params()
    assert _rope_bwd(None) == INVALID
    assert _rope_bwd(_rope_params(grad_dtype=2)) == INVALID
    for s in ((770, 768, 768), (768, 64, 768), (768, 768, 0)):
        assert _rope_bwd(p, strides=s) == INVALID, s
    for name in ("q", "k", "pos", "freq", "qw", "kw", "dq", "dk", "dqi", "dki", "dv", "dvi",
                 "dqw", "dkw"):
        assert _rope_bwd(p, **{name: None}) == INVALID, name
    for name in ("q", "k", "dq", "dk", "dv", "dqi", "dki", "dvi"):
        assert _rope_bwd(p, **{name: FAKE + 8}) == INVALID, name


# ----------------------------------------------------------------------------- extend
def _ext_params(**kw):
    p = binding.AttnSinkExtendParams(4, 20, 16, 2, 64, 16, 64, 8, 0, 0.125)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _extend(p, ws=FAKE, ws_bytes=1 << 40, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, lens=FAKE, cu=FAKE, sink=FAKE, out=FAKE,
             lse=FAKE)
    a.update(kw)
    return binding.attn_sink_extend(p, *a.values(), ws, ws_bytes, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=32), UNSUPPORTED), (dict(heads_q=258), UNSUPPORTED),
    (dict(heads_q=15), INVALID), (dict(heads_q=0), INVALID), (dict(heads_kv=0), INVALID),
    (dict(batch=-1), INVALID), (dict(total_q=-1), INVALID), (dict(page_size=0), INVALID),
    (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(max_pages=1 << 27), INVALID), (dict(softmax_scale=0.0), INVALID),
    (dict(softmax_scale=math.nan), INVALID), (dict(softmax_scale=math.inf), INVALID),
    (dict(heads_q=1 << 24, heads_kv=1 << 24, total_q=1 << 20), UNSUPPORTED)])
def test_extend_rejects_bad_params(kw, status):
    assert _extend(_ext_params(**kw)) == status
    assert binding.attn_sink_extend_workspace_size(_ext_params(**kw)) == 0


def test_extend_rejects_bad_pointers_and_workspaces():
    p = _ext_params()
    assert _extend(None) == INVALID
    assert binding.attn_sink_extend_workspace_size(None) == 0
    for name in ("q", "kc", "vc", "table", "lens", "cu", "sink", "out", "lse"):
        assert _extend(p, **{name: None}) == INVALID, name
    for name in ("q", "kc", "vc", "out"):
        assert _extend(p, **{name: FAKE + 8}) == INVALID, name
    n = binding.attn_sink_extend_workspace_size(p)
    assert n > 0 and n % 256 == 0
    for ws, nbytes in ((None, n), (FAKE + 16, n), (FAKE, n - 1)):
        assert _extend(p, ws=ws, ws_bytes=nbytes) == WORKSPACE
    for kw in (dict(batch=0), dict(total_q=0)):           # nothing to do
        assert _extend(_ext_params(**kw), ws=None, ws_bytes=0) == OK
        assert binding.attn_sink_extend_workspace_size(_ext_params(**kw)) == 0


@pytest.mark.parametrize("pages,page,heads,status", [
    (1 << 27, 16, 2, UNSUPPORTED), ((1 << 31) - 1, 1, 3, UNSUPPORTED),
    ((1 << 27) - 1, 16, 2, OK), ((1 << 31) - 1, 1, 2, OK), (1 << 31 - 4, 7, 4, OK)])
def test_extend_counts_the_cache_rows_of_all_heads_in_32_bits(pages, page, heads, status):
    p = _ext_params(num_pages=pages, page_size=page, heads_kv=heads, heads_q=heads)
    assert (binding.attn_sink_extend_workspace_size(p) > 0) == (status == OK)
    # without room in the workspace nothing is launched
    assert _extend(p, ws=None, ws_bytes=0) == (WORKSPACE if status == OK else status)


# ----------------------------------------------------------------------------- conveniences
def test_conveniences_reject_bad_tensors():
    i32, bf16 = torch.int32, torch.bfloat16
    lens = torch.zeros(3, dtype=i32)
    plan = dict(page_size=16, num_pages=4, max_tokens=8)
    table = torch.zeros(3, 4, dtype=i32)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.page_plan(lens, lens, lens, table, **plan)
    with pytest.raises(ValueError, match="cached_lens"):
        binding.page_plan(lens.long(), lens, lens, table, **plan)
    with pytest.raises(ValueError, match="block_table"):
        binding.page_plan(lens, lens, lens, table.T.contiguous().T, **plan)
    with pytest.raises(ValueError, match="new_lens"):
        binding.page_plan(lens, lens[:2], lens, table, **plan)
    with pytest.raises(ValueError, match="max_tokens"):
        binding.page_plan(lens, lens, lens, table, page_size=16, num_pages=4, max_tokens=-1)

    qkv, pos, freq = torch.zeros(3, 6, 64, dtype=bf16), torch.zeros(3, dtype=i32), torch.zeros(32)
    heads = dict(heads_q=4, heads_kv=1)
    w = torch.ones(64)
    bad = [
        ((qkv, pos, freq), {}, "CUDA device"), ((qkv.float(), pos, freq), {}, "qkv"),
        ((qkv[:, :5], pos, freq), {}, "qkv"), ((qkv[:, :, ::2], pos, freq), {}, "qkv"),
        ((qkv.transpose(0, 1).contiguous().transpose(0, 1), pos, freq), {}, "qkv"),
        ((qkv, pos.long(), freq), {}, "positions"), ((qkv, pos[:2], freq), {}, "positions"),
        ((qkv, pos, freq.double()), {}, "inv_freq"), ((qkv, pos, torch.zeros(33)), {}, "inv_freq"),
        ((qkv, pos.expand(2, 3).contiguous(), freq), {}, "pair_axis"),
        ((qkv, pos, freq), dict(pair_axis=[0] * 31), "pair_axis"),
        ((qkv, pos, freq), dict(pair_axis=[1] * 32), "pair_axis"),
        ((qkv, pos, freq), dict(q_weight=w), "go together"),
        ((qkv, pos, freq), dict(q_weight=w.half(), k_weight=w.half()), "q_weight"),
        ((qkv, pos, freq), dict(q_weight=w, k_weight=w.bfloat16()), "k_weight"),
        ((qkv, pos, freq), dict(k_cache=qkv), "slots"),
        ((qkv, pos, freq), dict(slots=pos.long()), "k_cache"),
    ]
    for args, kw, match in bad:
        with pytest.raises(ValueError, match=match):
            binding.qkv_rope(*args, **heads, **kw)
    dq, dk = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 1, 64, dtype=bf16)
    with pytest.raises(ValueError, match="dk"):
        binding.qkv_rope_backward(qkv, pos, freq, dq, dk.float(), dk, **heads)
    with pytest.raises(ValueError, match="dq"):
        binding.qkv_rope_backward(qkv, pos, freq, dq.half(), dk, dk, **heads)
    with pytest.raises(ValueError, match="inv_freq"):
        binding.qkv_rope_autograd(qkv, pos, freq.clone().requires_grad_(), **heads)
    with pytest.raises(binding.AttnSinkError, match="UNSUPPORTED"):
        p = binding._rope_params(qkv, pos, torch.zeros(4), 4, 1, None, None, None)
        binding._check(binding.attn_sink_qkv_rope(p, *[FAKE] * 13, stream=0), "rope")

    cache, sink = torch.zeros(4, 16, 1, 64, dtype=bf16), torch.zeros(4)
    cu = torch.zeros(4, dtype=i32)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.extend(dq, cache, cache, table, lens, cu, sink)
    with pytest.raises(ValueError, match="sink"):
        binding.extend(dq, cache, cache, table, lens, cu, sink.bfloat16())
    with pytest.raises(ValueError, match="cu_seqlens_q"):
        binding.extend(dq, cache, cache, table, lens, cu[:3], sink)
    with pytest.raises(ValueError, match="v_cache"):
        binding.extend(dq, cache, cache[:3], table, lens, cu, sink)
    with pytest.raises(ValueError, match="lse"):
        binding.extend(dq, cache, cache, table, lens, cu, sink, lse=torch.zeros(4, 2))


def test_axis_sections():
    assert binding.axis_sections(2, 1, 3) == [0, 0, 1, 2, 2, 2]
