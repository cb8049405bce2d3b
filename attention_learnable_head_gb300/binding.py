"""ctypes binding of libattn_sink.so.

``attn_sink_fwd``, ``attn_sink_bwd``, ``attn_sink_fwd_workspace_size``,
``attn_sink_bwd_workspace_size``,
``attn_sink_status_string``, ``attn_sink_device_error``,
``attn_sink_launch_count``, ``attn_sink_last_cuda_error``,
``attn_sink_kernel_timing``, ``attn_sink_kernel_time``, ``attn_sink_fwd_chunk``,
``attn_sink_merge``, ``attn_sink_bwd_deterministic``, ``attn_sink_decode``,
``attn_sink_decode_workspace_size``, ``attn_sink_fwd_ex``, ``attn_sink_bwd_ex`` and
``attn_sink_fwd_noalloc`` mirror the C entry
points of ``include/attn_sink.h`` one to one: they only turn tensors into
device pointers and return the library's status.  ``forward``, ``backward``
and ``attn_sink`` (autograd) are conveniences on top that allocate outputs and
the workspace with torch and raise on a non-zero status.  The entry points of
``include/attn_sink_step.h`` (``attn_sink_page_plan``, ``attn_sink_qkv_rope``,
``attn_sink_qkv_rope_bwd``, ``attn_sink_extend`` and their workspace sizes) and
their conveniences ``page_plan``, ``qkv_rope``, ``qkv_rope_backward``,
``qkv_rope_autograd`` and ``extend`` come after them; a plain call of these goes
through the native module ``attn_sink_fast`` (``csrc/fast_calls.cpp``) to the same
entry points; so do those of ``include/attn_sink_cache.h`` (``decode_shared``,
``page_bounds``, ``select_pages``, ``decode_pages``, ``key_mass``, ``evict``).  Every step of the
computation runs in the library's CUDA kernels; there is no other code path,
and loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib.util
import math
import os
import re
from typing import NamedTuple

import torch

from .build import FAST_PATH, INCLUDE, LIB_PATH, fast_built_for, fast_target

c_int, c_float, c_void_p, c_size_t = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
c_longlong = ctypes.c_longlong

ATTN_SINK_OK = 0
STATUS_NAMES = {0: "ATTN_SINK_OK", 1: "ATTN_SINK_ERR_INVALID_ARG", 2: "ATTN_SINK_ERR_UNSUPPORTED",
                3: "ATTN_SINK_ERR_WORKSPACE", 4: "ATTN_SINK_ERR_CUDA", 5: "ATTN_SINK_ERR_TIMEOUT"}


class AttnSinkParams(ctypes.Structure):
    """Mirror of ``attn_sink_params`` in include/attn_sink.h (field order matters)."""
    _fields_ = [
        ("batch", c_int), ("seqlen_q", c_int), ("seqlen_k", c_int),
        ("num_seqs", c_int), ("total_q", c_int), ("total_k", c_int),
        ("max_seqlen_q", c_int), ("max_seqlen_k", c_int),
        ("heads_q", c_int), ("heads_kv", c_int), ("head_dim", c_int),
        ("causal", c_int), ("window", c_int), ("softmax_scale", c_float),
        ("grad_dtype", c_int),
    ]


class AttnSinkDecodeParams(ctypes.Structure):
    """Mirror of ``attn_sink_decode_params`` in include/attn_sink.h."""
    _fields_ = [
        ("batch", c_int), ("heads_q", c_int), ("heads_kv", c_int), ("head_dim", c_int),
        ("page_size", c_int), ("num_pages", c_int), ("max_pages", c_int), ("window", c_int),
        ("softmax_scale", c_float),
    ]


class AttnSinkPlanParams(ctypes.Structure):
    """Mirror of ``attn_sink_plan_params`` in include/attn_sink_step.h."""
    _fields_ = [
        ("batch", c_int), ("page_size", c_int), ("num_pages", c_int), ("max_pages", c_int),
        ("num_free", c_int), ("max_tokens", c_int),
    ]


class AttnSinkRopeParams(ctypes.Structure):
    """Mirror of ``attn_sink_rope_params`` in include/attn_sink_step.h."""
    _fields_ = [
        ("q_stride", c_longlong), ("k_stride", c_longlong), ("v_stride", c_longlong),
        ("tokens", c_int), ("heads_q", c_int), ("heads_kv", c_int), ("head_dim", c_int),
        ("rotary_dim", c_int), ("interleaved", c_int), ("num_axes", c_int),
        ("pair_axis", ctypes.c_ubyte * 32), ("norm", c_int), ("weight_bf16", c_int),
        ("eps", c_float), ("amplitude", c_float), ("page_size", c_int), ("num_pages", c_int),
        ("grad_dtype", c_int),
    ]


class AttnSinkExtendParams(ctypes.Structure):
    """Mirror of ``attn_sink_extend_params`` in include/attn_sink_step.h."""
    _fields_ = [
        ("batch", c_int), ("total_q", c_int), ("heads_q", c_int), ("heads_kv", c_int),
        ("head_dim", c_int), ("page_size", c_int), ("num_pages", c_int), ("max_pages", c_int),
        ("window", c_int), ("softmax_scale", c_float),
    ]


class AttnSinkSharedParams(ctypes.Structure):
    """Mirror of ``attn_sink_shared_params`` in include/attn_sink_cache.h."""
    _fields_ = [
        ("batch", c_int), ("num_groups", c_int), ("heads_q", c_int), ("heads_kv", c_int),
        ("head_dim", c_int), ("page_size", c_int), ("num_pages", c_int), ("max_pages", c_int),
        ("softmax_scale", c_float),
    ]


class AttnSinkBoundsParams(ctypes.Structure):
    """Mirror of ``attn_sink_bounds_params`` in include/attn_sink_cache.h."""
    _fields_ = [
        ("batch", c_int), ("heads_kv", c_int), ("head_dim", c_int), ("page_size", c_int),
        ("num_pages", c_int), ("max_pages", c_int),
    ]


class AttnSinkSelectParams(ctypes.Structure):
    """Mirror of ``attn_sink_select_params`` in include/attn_sink_cache.h."""
    _fields_ = [
        ("batch", c_int), ("heads_q", c_int), ("heads_kv", c_int), ("head_dim", c_int),
        ("page_size", c_int), ("num_pages", c_int), ("max_pages", c_int), ("count", c_int),
        ("keep_first", c_int), ("keep_last", c_int),
    ]


class AttnSinkPagesParams(ctypes.Structure):
    """Mirror of ``attn_sink_pages_params`` in include/attn_sink_cache.h."""
    _fields_ = [
        ("batch", c_int), ("heads_q", c_int), ("heads_kv", c_int), ("head_dim", c_int),
        ("page_size", c_int), ("num_pages", c_int), ("max_pages", c_int), ("count", c_int),
        ("softmax_scale", c_float),
    ]


class AttnSinkMassParams(ctypes.Structure):
    """Mirror of ``attn_sink_mass_params`` in include/attn_sink_cache.h."""
    _fields_ = [
        ("batch", c_int), ("total_q", c_int), ("heads_q", c_int), ("heads_kv", c_int),
        ("head_dim", c_int), ("page_size", c_int), ("num_pages", c_int), ("max_pages", c_int),
        ("max_keys", c_int), ("accumulate", c_int), ("softmax_scale", c_float),
    ]


class AttnSinkEvictParams(ctypes.Structure):
    """Mirror of ``attn_sink_evict_params`` in include/attn_sink_cache.h."""
    _fields_ = [
        ("batch", c_int), ("heads_kv", c_int), ("head_dim", c_int), ("page_size", c_int),
        ("num_pages", c_int), ("max_pages", c_int), ("max_keys", c_int), ("budget", c_int),
        ("keep_first", c_int), ("keep_last", c_int), ("max_freed", c_int),
    ]


class AttnSinkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        extra = ""
        if status == 4:
            extra = f", last CUDA error {attn_sink_last_cuda_error()}"
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({attn_sink_status_string(status)}{extra})")


_LIB = None


def header_functions(header: str = "attn_sink.h") -> list[str]:
    """Names of the functions a header under include/ declares."""
    text = open(os.path.join(INCLUDE, header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^(?:[A-Za-z_]\w*[\s*]+)+(attn_sink_\w+)\s*\(", text, flags=re.M)


def lib():
    """Load libattn_sink.so (built in-tree by ``build.build()``)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (nvcc, sm_103a)")
    _LIB = load_library(LIB_PATH)
    return _LIB


def load_library(path: str):
    """A ctypes handle on a build of the library at `path` with the C
    signatures of the headers under include/ attached (the product library, or the
    test build that also exports attn_sink_test_withhold)."""
    L = ctypes.CDLL(path)
    P = ctypes.POINTER(AttnSinkParams)
    L.attn_sink_fwd.argtypes = [P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
    L.attn_sink_fwd_workspace_size.argtypes = [P]
    L.attn_sink_fwd_workspace_size.restype = c_size_t
    L.attn_sink_fwd_noalloc.argtypes = [P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    L.attn_sink_fwd_noalloc.restype = c_int
    L.attn_sink_fwd.restype = c_int
    L.attn_sink_fwd_chunk.argtypes = [P, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                      c_void_p]
    L.attn_sink_fwd_chunk.restype = c_int
    L.attn_sink_merge.argtypes = [c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    L.attn_sink_merge.restype = c_int
    PD = ctypes.POINTER(AttnSinkDecodeParams)
    L.attn_sink_decode_workspace_size.argtypes = [PD]
    L.attn_sink_decode_workspace_size.restype = c_size_t
    L.attn_sink_decode.argtypes = [PD, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                   c_void_p]
    L.attn_sink_decode.restype = c_int
    L.attn_sink_bwd_workspace_size.argtypes = [P]
    L.attn_sink_bwd_workspace_size.restype = c_size_t
    L.attn_sink_bwd.argtypes = [P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
    L.attn_sink_bwd.restype = c_int
    L.attn_sink_bwd_deterministic.argtypes = L.attn_sink_bwd.argtypes
    L.attn_sink_bwd_deterministic.restype = c_int
    L.attn_sink_fwd_ex.argtypes = [P, c_int] + L.attn_sink_fwd.argtypes[1:]
    L.attn_sink_fwd_ex.restype = c_int
    L.attn_sink_bwd_ex.argtypes = [P, c_int] + L.attn_sink_bwd.argtypes[1:]
    L.attn_sink_bwd_ex.restype = c_int
    L.attn_sink_status_string.argtypes = [c_int]
    L.attn_sink_status_string.restype = ctypes.c_char_p
    L.attn_sink_device_error.argtypes = [c_void_p, ctypes.POINTER(c_int)]
    L.attn_sink_device_error.restype = c_int
    L.attn_sink_last_cuda_error.argtypes = []
    L.attn_sink_last_cuda_error.restype = c_int
    L.attn_sink_launch_count.argtypes = []
    L.attn_sink_launch_count.restype = ctypes.c_ulonglong
    L.attn_sink_kernel_timing.argtypes = [c_int]
    L.attn_sink_kernel_timing.restype = c_int
    L.attn_sink_kernel_time.argtypes = [c_int, ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_ulonglong)]
    L.attn_sink_kernel_time.restype = c_int
    L.attn_sink_page_plan.argtypes = [ctypes.POINTER(AttnSinkPlanParams)] + [c_void_p] * 10
    L.attn_sink_page_plan.restype = c_int
    PR = ctypes.POINTER(AttnSinkRopeParams)
    L.attn_sink_qkv_rope.argtypes = [PR] + [c_void_p] * 14
    L.attn_sink_qkv_rope.restype = c_int
    L.attn_sink_qkv_rope_bwd_workspace_size.argtypes = [PR]
    L.attn_sink_qkv_rope_bwd_workspace_size.restype = c_size_t
    L.attn_sink_qkv_rope_bwd.argtypes = ([PR] + [c_void_p] * 12 + [c_longlong] * 3 +
                                         [c_void_p] * 3 + [c_size_t, c_void_p])
    L.attn_sink_qkv_rope_bwd.restype = c_int
    PE = ctypes.POINTER(AttnSinkExtendParams)
    L.attn_sink_extend_workspace_size.argtypes = [PE]
    L.attn_sink_extend_workspace_size.restype = c_size_t
    L.attn_sink_extend.argtypes = [PE] + [c_void_p] * 10 + [c_size_t, c_void_p]
    L.attn_sink_extend.restype = c_int
    for name, params, pointers, work in (
            ("decode_shared", AttnSinkSharedParams, 10, True),
            ("page_bounds", AttnSinkBoundsParams, 5, False),
            ("select_pages", AttnSinkSelectParams, 5, True),
            ("decode_pages", AttnSinkPagesParams, 9, True),
            ("key_mass", AttnSinkMassParams, 7, False),
            ("evict", AttnSinkEvictParams, 9, True)):
        f = getattr(L, "attn_sink_" + name)
        f.argtypes = ([ctypes.POINTER(params)] + [c_void_p] * pointers +
                      ([c_void_p, c_size_t] if work else []) + [c_void_p])
        f.restype = c_int
        if work:
            f = getattr(L, f"attn_sink_{name}_workspace_size")
            f.argtypes = [ctypes.POINTER(params)]
            f.restype = c_size_t
    if hasattr(L, "attn_sink_test_withhold"):
        L.attn_sink_test_withhold.argtypes = [c_int, c_int]
        L.attn_sink_test_withhold.restype = c_int
    return L


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _pref(params):
    return None if params is None else ctypes.byref(params)


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ----------------------------------------------------------------------------- C entry points
def attn_sink_fwd(params: AttnSinkParams, q, k, v, sink, cu_seqlens_q, cu_seqlens_k, out,
                  out_residual, lse, workspace, workspace_bytes: int, stream=None) -> int:
    return lib().attn_sink_fwd(_pref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(sink),
                               _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(out),
                               _ptr(out_residual), _ptr(lse), _ptr(workspace),
                               int(workspace_bytes), _stream(stream))


ATTN_SINK_FLAG_SINK_BF16 = 1
ATTN_SINK_FLAG_ACCUMULATE_DSINK = 2
ATTN_SINK_FLAG_DETERMINISTIC = 4


def attn_sink_fwd_ex(params: AttnSinkParams, flags: int, q, k, v, sink, cu_seqlens_q,
                     cu_seqlens_k, out, out_residual, lse, workspace, workspace_bytes: int,
                     stream=None) -> int:
    return lib().attn_sink_fwd_ex(_pref(params), int(flags), _ptr(q), _ptr(k), _ptr(v),
                                  _ptr(sink), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(out),
                                  _ptr(out_residual), _ptr(lse), _ptr(workspace),
                                  int(workspace_bytes), _stream(stream))


def attn_sink_bwd_ex(params: AttnSinkParams, flags: int, q, k, v, sink, cu_seqlens_q,
                     cu_seqlens_k, out, out_residual, lse, dout, dq, dk, dv, dsink, workspace,
                     workspace_bytes: int, stream=None) -> int:
    return lib().attn_sink_bwd_ex(_pref(params), int(flags), _ptr(q), _ptr(k), _ptr(v),
                                  _ptr(sink), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(out),
                                  _ptr(out_residual), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                                  _ptr(dv), _ptr(dsink), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream))


def attn_sink_fwd_chunk(params: AttnSinkParams, q_pos0: int, q, k, v, cu_seqlens_q,
                        cu_seqlens_k, out, out_residual, lse, workspace, workspace_bytes: int,
                        stream=None) -> int:
    return lib().attn_sink_fwd_chunk(_pref(params), int(q_pos0), _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(out),
                                     _ptr(out_residual), _ptr(lse), _ptr(workspace),
                                     int(workspace_bytes), _stream(stream))


def attn_sink_merge(num_chunks: int, total_q: int, heads_q: int, head_dim: int, o_parts,
                    o_residual_parts, lse_parts, sink, out, out_residual, lse,
                    stream=None) -> int:
    return lib().attn_sink_merge(int(num_chunks), int(total_q), int(heads_q), int(head_dim),
                                 _ptr(o_parts), _ptr(o_residual_parts), _ptr(lse_parts),
                                 _ptr(sink), _ptr(out), _ptr(out_residual), _ptr(lse),
                                 _stream(stream))


def attn_sink_decode_workspace_size(params: AttnSinkDecodeParams) -> int:
    return int(lib().attn_sink_decode_workspace_size(
        None if params is None else ctypes.byref(params)))


def attn_sink_decode(params: AttnSinkDecodeParams, q, k_cache, v_cache, block_table, seq_lens,
                     sink, out, out_residual, lse, workspace, workspace_bytes: int,
                     stream=None) -> int:
    return lib().attn_sink_decode(None if params is None else ctypes.byref(params), _ptr(q),
                                  _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                  _ptr(seq_lens), _ptr(sink), _ptr(out), _ptr(out_residual),
                                  _ptr(lse), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream))


def make_decode_params(q_shape, cache_shape, max_pages: int, *, window: int = 0,
                       softmax_scale: float | None = None) -> AttnSinkDecodeParams:
    """Params from q [B, H_q, d] and a cache [num_pages, page_size, H_kv, d]."""
    p = AttnSinkDecodeParams()
    p.batch, p.heads_q, p.head_dim = int(q_shape[0]), int(q_shape[1]), int(q_shape[2])
    p.num_pages, p.page_size, p.heads_kv = (int(cache_shape[0]), int(cache_shape[1]),
                                            int(cache_shape[2]))
    p.max_pages = int(max_pages)
    p.window = int(window)
    p.softmax_scale = float(softmax_scale if softmax_scale is not None
                            else 1.0 / math.sqrt(p.head_dim))
    return p


def decode(q, k_cache, v_cache, block_table, seq_lens, sink, *, window: int = 0,
           softmax_scale: float | None = None, residual: bool = False, stream=None):
    """(out, lse, out_residual) of one decode step over a paged cache
    (attn_sink_decode): q [B, H_q, 64], caches [pages, page_size, H_kv, 64],
    block_table [B, max_pages] int32, seq_lens [B] int32."""
    p = make_decode_params(q.shape, k_cache.shape, block_table.shape[1], window=window,
                           softmax_scale=softmax_scale)
    out = torch.empty_like(q)
    res = torch.empty_like(q) if residual else None
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    nbytes = attn_sink_decode_workspace_size(p)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check(attn_sink_decode(p, q, k_cache, v_cache, block_table, seq_lens, sink, out, res, lse,
                            ws, ws.numel(), stream), "attn_sink_decode")
    return out, lse, res


# Bytes of the static scratch behind attn_sink_fwd_noalloc (the header's
# ATTN_SINK_NOALLOC_SCRATCH_BYTES).
ATTN_SINK_NOALLOC_SCRATCH_BYTES = 16 << 20


def attn_sink_fwd_noalloc(params: AttnSinkParams, q, k, v, sink, cu_seqlens_q, cu_seqlens_k, out,
                          out_residual, lse, stream=None) -> int:
    """Forward for callers that cannot allocate device memory: the library's
    own static scratch replaces the workspace (see include/attn_sink.h)."""
    return lib().attn_sink_fwd_noalloc(_pref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(sink),
                                       _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(out),
                                       _ptr(out_residual), _ptr(lse), _stream(stream))


def attn_sink_fwd_workspace_size(params: AttnSinkParams) -> int:
    return int(lib().attn_sink_fwd_workspace_size(_pref(params)))


def attn_sink_bwd_workspace_size(params: AttnSinkParams) -> int:
    return int(lib().attn_sink_bwd_workspace_size(_pref(params)))


def attn_sink_bwd(params: AttnSinkParams, q, k, v, sink, cu_seqlens_q, cu_seqlens_k, out,
                  out_residual, lse, dout, dq, dk, dv, dsink, workspace, workspace_bytes: int,
                  stream=None) -> int:
    return lib().attn_sink_bwd(_pref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(sink),
                               _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(out),
                               _ptr(out_residual), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                               _ptr(dv), _ptr(dsink), _ptr(workspace), int(workspace_bytes),
                               _stream(stream))


def attn_sink_bwd_deterministic(params: AttnSinkParams, q, k, v, sink, cu_seqlens_q, cu_seqlens_k, out,
                  out_residual, lse, dout, dq, dk, dv, dsink, workspace, workspace_bytes: int,
                  stream=None) -> int:
    return lib().attn_sink_bwd_deterministic(_pref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(sink),
                               _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(out),
                               _ptr(out_residual), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                               _ptr(dv), _ptr(dsink), _ptr(workspace), int(workspace_bytes),
                               _stream(stream))


def attn_sink_status_string(status: int) -> str:
    return lib().attn_sink_status_string(int(status)).decode()


def attn_sink_last_cuda_error() -> int:
    return int(lib().attn_sink_last_cuda_error())


def attn_sink_launch_count() -> int:
    return int(lib().attn_sink_launch_count())


ATTN_SINK_KERNEL_FWD = 0
ATTN_SINK_KERNEL_BWD_MAIN = 1
ATTN_SINK_KERNEL_BWD_DQ = 2
ATTN_SINK_KERNEL_MERGE = 3


def attn_sink_kernel_timing(on: bool) -> int:
    return int(lib().attn_sink_kernel_timing(1 if on else 0))


def attn_sink_kernel_time(kernel: int) -> tuple[int, float, int]:
    """(status, summed milliseconds, launches) of `kernel` since its last read."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_ulonglong(0)
    st = lib().attn_sink_kernel_time(int(kernel), ctypes.byref(ms), ctypes.byref(n))
    return int(st), float(ms.value), int(n.value)


def attn_sink_device_error(stream=None) -> tuple[int, int]:
    code = c_int(0)
    st = lib().attn_sink_device_error(_stream(stream), ctypes.byref(code))
    return st, code.value


# ----------------------------------------------------------------------------- conveniences
def make_params(q_shape, k_shape, *, causal: bool, window: int, softmax_scale: float | None,
                num_seqs: int | None = None, max_seqlen_q: int | None = None,
                max_seqlen_k: int | None = None, grad_dtype: int = 0) -> AttnSinkParams:
    """Params from tensor shapes: q [B, N, H, d] (dense) or [T, H, d] (packed;
    then num_seqs and max_seqlen_* are required)."""
    p = AttnSinkParams()
    d = int(q_shape[-1])
    p.head_dim = d
    p.heads_q = int(q_shape[-2])
    p.heads_kv = int(k_shape[-2])
    p.causal = int(bool(causal))
    p.window = int(window)
    p.softmax_scale = float(softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(d))
    p.grad_dtype = int(grad_dtype)
    if len(q_shape) == 4:
        p.batch, p.seqlen_q, p.seqlen_k = int(q_shape[0]), int(q_shape[1]), int(k_shape[1])
    else:
        if num_seqs is None or max_seqlen_q is None or max_seqlen_k is None:
            raise ValueError("packed inputs need num_seqs and max_seqlen_q / max_seqlen_k")
        p.num_seqs = int(num_seqs)
        p.total_q, p.total_k = int(q_shape[0]), int(k_shape[0])
        p.max_seqlen_q, p.max_seqlen_k = int(max_seqlen_q), int(max_seqlen_k)
    return p


def _check(status: int, where: str):
    if status != ATTN_SINK_OK:
        raise AttnSinkError(status, where)


def _lse_len(q) -> int:
    return q.shape[0] * q.shape[1] if q.dim() == 4 else q.shape[0]


def forward(q, k, v, sink, *, causal: bool = True, window: int = 0,
            softmax_scale: float | None = None, cu_seqlens_q=None, cu_seqlens_k=None,
            max_seqlen_q: int | None = None, max_seqlen_k: int | None = None,
            residual: bool = True, stream=None):
    """(out, lse, out_residual): out like q (bf16), lse [H_q, T_q] fp32, and the
    bf16 rounding residual of out (None when residual=False)."""
    num_seqs = None if cu_seqlens_q is None else cu_seqlens_q.numel() - 1
    p = make_params(q.shape, k.shape, causal=causal, window=window, softmax_scale=softmax_scale,
                    num_seqs=num_seqs, max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k)
    out = torch.empty_like(q)
    res = torch.empty_like(q) if residual else None
    lse = torch.empty((q.shape[-2], _lse_len(q)), dtype=torch.float32, device=q.device)
    nbytes = attn_sink_fwd_workspace_size(p)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    if sink.dtype == torch.bfloat16:      # a bf16 sink parameter, read exactly
        _check(attn_sink_fwd_ex(p, ATTN_SINK_FLAG_SINK_BF16, q, k, v, sink, cu_seqlens_q,
                                cu_seqlens_k, out, res, lse, ws, ws.numel(), stream),
               "attn_sink_fwd_ex")
    else:
        _check(attn_sink_fwd(p, q, k, v, sink, cu_seqlens_q, cu_seqlens_k, out, res, lse, ws,
                             ws.numel(), stream), "attn_sink_fwd")
    return out, lse, res


def forward_chunk(q, k, v, q_pos0: int, *, causal: bool = True, window: int = 0,
                  softmax_scale: float | None = None, cu_seqlens_q=None, cu_seqlens_k=None,
                  max_seqlen_q: int | None = None, max_seqlen_k: int | None = None,
                  residual: bool = True, stream=None):
    """(out, lse, out_residual) of the queries over one key chunk, without the
    sink (attn_sink_fwd_chunk); k, v hold the chunk's keys."""
    num_seqs = None if cu_seqlens_q is None else cu_seqlens_q.numel() - 1
    p = make_params(q.shape, k.shape, causal=causal, window=window, softmax_scale=softmax_scale,
                    num_seqs=num_seqs, max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k)
    out = torch.empty_like(q)
    res = torch.empty_like(q) if residual else None
    lse = torch.empty((q.shape[-2], _lse_len(q)), dtype=torch.float32, device=q.device)
    nbytes = attn_sink_fwd_workspace_size(p)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check(attn_sink_fwd_chunk(p, q_pos0, q, k, v, cu_seqlens_q, cu_seqlens_k, out, res, lse,
                               ws, ws.numel(), stream), "attn_sink_fwd_chunk")
    return out, lse, res


def merge(outs, lses, sink, *, residuals=None, stream=None):
    """(out, lse, out_residual) of the whole key sequence from the chunks'
    results (attn_sink_merge): outs like q, lses [H_q, T_q], residuals optional."""
    o = torch.stack(list(outs)).contiguous()
    ls = torch.stack(list(lses)).contiguous()
    r = None if residuals is None else torch.stack(list(residuals)).contiguous()
    out = torch.empty_like(o[0])
    res = torch.empty_like(o[0])
    lse = torch.empty_like(ls[0])
    heads, d = o.shape[-2], o.shape[-1]
    _check(attn_sink_merge(o.shape[0], ls.shape[-1], heads, d, o, r, ls, sink, out, res, lse,
                           stream), "attn_sink_merge")
    return out, lse, res


def backward(q, k, v, sink, out, lse, dout, *, out_residual=None, causal: bool = True,
             window: int = 0, softmax_scale: float | None = None, cu_seqlens_q=None,
             cu_seqlens_k=None, max_seqlen_q: int | None = None,
             max_seqlen_k: int | None = None, grad_dtype: int = 0, workspace=None,
             deterministic: bool = False, dsink=None, accumulate_dsink: bool = False,
             stream=None):
    """dq, dk, dv (bf16, or fp32 when grad_dtype = 1) and dsink ([H_q], the
    sink's dtype: fp32, or bf16 for a bf16 sink).
    deterministic=True: bitwise reproducible (attn_sink_bwd_deterministic);
    accumulate_dsink=True: the gradient is added into the given `dsink`."""
    num_seqs = None if cu_seqlens_q is None else cu_seqlens_q.numel() - 1
    p = make_params(q.shape, k.shape, causal=causal, window=window, softmax_scale=softmax_scale,
                    num_seqs=num_seqs, max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k,
                    grad_dtype=grad_dtype)
    gd = torch.float32 if grad_dtype == 1 else torch.bfloat16
    dq = torch.empty(q.shape, dtype=gd, device=q.device)
    dk = torch.empty(k.shape, dtype=gd, device=q.device)
    dv = torch.empty(v.shape, dtype=gd, device=q.device)
    if accumulate_dsink and dsink is None:
        raise ValueError("accumulate_dsink needs the dsink tensor to add into")
    if dsink is None:
        dsink = torch.empty_like(sink)
    nbytes = attn_sink_bwd_workspace_size(p)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    flags = ((ATTN_SINK_FLAG_SINK_BF16 if sink.dtype == torch.bfloat16 else 0)
             | (ATTN_SINK_FLAG_ACCUMULATE_DSINK if accumulate_dsink else 0)
             | (ATTN_SINK_FLAG_DETERMINISTIC if deterministic else 0))
    if flags & (ATTN_SINK_FLAG_SINK_BF16 | ATTN_SINK_FLAG_ACCUMULATE_DSINK):
        _check(attn_sink_bwd_ex(p, flags, q, k, v, sink, cu_seqlens_q, cu_seqlens_k, out,
                                out_residual, lse, dout, dq, dk, dv, dsink, workspace,
                                workspace.numel(), stream), "attn_sink_bwd_ex")
    else:
        fn = attn_sink_bwd_deterministic if deterministic else attn_sink_bwd
        _check(fn(p, q, k, v, sink, cu_seqlens_q, cu_seqlens_k, out, out_residual, lse,
                  dout, dq, dk, dv, dsink, workspace, workspace.numel(), stream), fn.__name__)
    return dq, dk, dv, dsink


class AttnSinkFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run in libattn_sink.so."""

    @staticmethod
    def forward(ctx, q, k, v, sink, causal, window, softmax_scale, cu_seqlens_q, cu_seqlens_k,
                max_seqlen_q, max_seqlen_k):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        sink32 = sink.detach().float().contiguous()
        out, lse, res = forward(q, k, v, sink32, causal=causal, window=window,
                                softmax_scale=softmax_scale, cu_seqlens_q=cu_seqlens_q,
                                cu_seqlens_k=cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                                max_seqlen_k=max_seqlen_k)
        ctx.save_for_backward(q, k, v, sink32, out, res, lse, cu_seqlens_q, cu_seqlens_k)
        ctx.cfg = (causal, window, softmax_scale, max_seqlen_q, max_seqlen_k, sink.dtype)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, sink32, out, res, lse, cu_q, cu_k = ctx.saved_tensors
        causal, window, scale, mq, mk, sink_dtype = ctx.cfg
        dq, dk, dv, dsink = backward(q, k, v, sink32, out, lse, dout.contiguous(),
                                     out_residual=res, causal=causal,
                                     window=window, softmax_scale=scale, cu_seqlens_q=cu_q,
                                     cu_seqlens_k=cu_k, max_seqlen_q=mq, max_seqlen_k=mk)
        return dq, dk, dv, dsink.to(sink_dtype), None, None, None, None, None, None, None


def attn_sink(q, k, v, sink, *, causal: bool = True, window: int = 0,
              softmax_scale: float | None = None, cu_seqlens_q=None, cu_seqlens_k=None,
              max_seqlen_q: int | None = None, max_seqlen_k: int | None = None):
    """Differentiable attention with a learnable per-head sink (bf16 q/k/v)."""
    return AttnSinkFunction.apply(q, k, v, sink, causal, window, softmax_scale, cu_seqlens_q,
                                  cu_seqlens_k, max_seqlen_q, max_seqlen_k)


# ----------------------------------------------------------------------------- include/attn_sink_step.h
def attn_sink_page_plan(params: AttnSinkPlanParams, cached_lens, new_lens, free_pages, block_table,
                        slots, positions, cu_seqlens, seq_lens, pages_needed, stream=None) -> int:
    return lib().attn_sink_page_plan(_pref(params), _ptr(cached_lens), _ptr(new_lens),
                                     _ptr(free_pages), _ptr(block_table), _ptr(slots),
                                     _ptr(positions), _ptr(cu_seqlens), _ptr(seq_lens),
                                     _ptr(pages_needed), _stream(stream))


def attn_sink_qkv_rope(params: AttnSinkRopeParams, q, k, v, positions, inv_freq, q_weight,
                       k_weight, slots, q_out, k_out, v_out, k_cache, v_cache,
                       stream=None) -> int:
    return lib().attn_sink_qkv_rope(_pref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(positions),
                                    _ptr(inv_freq), _ptr(q_weight), _ptr(k_weight), _ptr(slots),
                                    _ptr(q_out), _ptr(k_out), _ptr(v_out), _ptr(k_cache),
                                    _ptr(v_cache), _stream(stream))


def attn_sink_qkv_rope_bwd_workspace_size(params: AttnSinkRopeParams) -> int:
    return int(lib().attn_sink_qkv_rope_bwd_workspace_size(_pref(params)))


def attn_sink_qkv_rope_bwd(params: AttnSinkRopeParams, q, k, positions, inv_freq, q_weight,
                           k_weight, dq, dk, dv, dq_in, dk_in, dv_in, dq_in_stride: int,
                           dk_in_stride: int, dv_in_stride: int, dq_weight, dk_weight, workspace,
                           workspace_bytes: int, stream=None) -> int:
    return lib().attn_sink_qkv_rope_bwd(_pref(params), _ptr(q), _ptr(k), _ptr(positions),
                                        _ptr(inv_freq), _ptr(q_weight), _ptr(k_weight), _ptr(dq),
                                        _ptr(dk), _ptr(dv), _ptr(dq_in), _ptr(dk_in),
                                        _ptr(dv_in), int(dq_in_stride), int(dk_in_stride),
                                        int(dv_in_stride), _ptr(dq_weight), _ptr(dk_weight),
                                        _ptr(workspace), int(workspace_bytes), _stream(stream))


def attn_sink_extend_workspace_size(params: AttnSinkExtendParams) -> int:
    return int(lib().attn_sink_extend_workspace_size(_pref(params)))


def attn_sink_extend(params: AttnSinkExtendParams, q, k_cache, v_cache, block_table, seq_lens,
                     cu_seqlens_q, sink, out, lse, workspace, workspace_bytes: int,
                     stream=None) -> int:
    return lib().attn_sink_extend(_pref(params), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(block_table), _ptr(seq_lens), _ptr(cu_seqlens_q),
                                  _ptr(sink), _ptr(out), _ptr(lse), _ptr(workspace),
                                  int(workspace_bytes), _stream(stream))


_FAST = None


def _fast():
    """The native module attn_sink_fast (csrc/fast_calls.cpp) on libattn_sink.so:
    the conveniences' checks, allocations and calls in the plain case.  Its
    functions return None where a call is anything else; the Python code behind
    each use then checks the arguments one by one."""
    global _FAST
    if _FAST is None:
        if not os.path.exists(FAST_PATH) or fast_built_for() != fast_target():
            raise RuntimeError(
                f"{FAST_PATH} is missing or not built for {fast_target()}: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = lib()
        spec = importlib.util.spec_from_file_location("attn_sink_fast", FAST_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.init(*(ctypes.cast(f, c_void_p).value for f in (
            L.attn_sink_page_plan, L.attn_sink_qkv_rope, L.attn_sink_qkv_rope_bwd_workspace_size,
            L.attn_sink_qkv_rope_bwd, L.attn_sink_extend_workspace_size, L.attn_sink_extend,
            L.attn_sink_decode_shared_workspace_size, L.attn_sink_decode_shared,
            L.attn_sink_page_bounds, L.attn_sink_select_pages_workspace_size,
            L.attn_sink_select_pages, L.attn_sink_decode_pages_workspace_size,
            L.attn_sink_decode_pages, L.attn_sink_key_mass, L.attn_sink_evict_workspace_size,
            L.attn_sink_evict)))
        _FAST = module
    return _FAST


_NOTHING = contextlib.nullcontext()
# The current stream of a device as an integer; Stream objects cost a few
# microseconds, which is what the smallest of these calls take.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device, stream):
    """Context in which `device` is current and `stream` (None: the device's
    current one) is its current stream, so that outputs and workspaces are
    allocated for the stream that uses them."""
    if device.type != "cuda":
        raise ValueError(f"the tensors have to be on a CUDA device, not on {device}")
    if stream is None:
        if device.index == torch.cuda.current_device():
            return _NOTHING
        return torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _want(name, t, dtype, device, shape):
    """Check one tensor argument: its type, device and shape, and that it is
    contiguous."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} has to be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError(f"{name} has to be contiguous")


def _dims(name, t, n):
    """The shape of a tensor that has to have n dimensions."""
    if t.dim() != n:
        raise ValueError(f"{name} has to have {n} dimensions, not shape {tuple(t.shape)}")
    return t.shape


def _in_32_bits(**sizes):
    """ctypes would cut an integer to 32 bits without a word."""
    for name, n in sizes.items():
        if not -2 ** 31 <= n < 2 ** 31:
            raise ValueError(f"{name} is {n}: it has to fit 32 bits")


class PagePlan(NamedTuple):
    """What a serving step needs to know of its tokens (see page_plan)."""
    slots: torch.Tensor          # [max_tokens] int64: cache row of each new token, -1: none
    positions: torch.Tensor      # [max_tokens] int32
    cu_seqlens_q: torch.Tensor   # [B + 1] int32
    seq_lens: torch.Tensor       # [B] int32: cached + new
    pages_needed: torch.Tensor   # [1] int32: entries of free_pages that are now taken


def page_plan(cached_lens, new_lens, free_pages, block_table, *, page_size: int, num_pages: int,
              max_tokens: int, stream=None) -> PagePlan:
    """Plan a serving step on the GPU (attn_sink_page_plan): sequence b has
    cached_lens[b] keys and gets new_lens[b] new tokens; new pages are taken from
    free_pages in order and written into block_table [B, max_pages] in place.
    Nothing is read back: max_tokens bounds the tokens of the step."""
    if stream is None:
        r = (_FAST or _fast()).page_plan(cached_lens, new_lens, free_pages, block_table,
                                         page_size, num_pages, max_tokens)
        if r is not None:
            if type(r) is int:
                _check(r, "attn_sink_page_plan")
            return PagePlan(*r)
    dev, i32 = block_table.device, torch.int32
    b, = _dims("cached_lens", cached_lens, 1)
    cols, free = _dims("block_table", block_table, 2)[1], _dims("free_pages", free_pages, 1)[0]
    _want("cached_lens", cached_lens, i32, dev, (b,))
    _want("new_lens", new_lens, i32, dev, (b,))
    _want("free_pages", free_pages, i32, dev, (free,))
    _want("block_table", block_table, i32, dev, (b, cols))
    if max_tokens < 0:
        raise ValueError(f"max_tokens is {max_tokens}")
    _in_32_bits(page_size=page_size, num_pages=num_pages, max_tokens=max_tokens, cached_lens=b,
                block_table=cols, free_pages=free)
    with _on(dev, stream):
        slots = torch.empty(max_tokens, dtype=torch.int64, device=dev)
        positions = torch.empty(max_tokens, dtype=i32, device=dev)
        small = torch.empty(2 * b + 2, dtype=i32, device=dev)
        at = small.data_ptr()
        p = AttnSinkPlanParams(b, page_size, num_pages, cols, free, max_tokens)
        _check(lib().attn_sink_page_plan(
            ctypes.byref(p), cached_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(),
            block_table.data_ptr(), slots.data_ptr(), positions.data_ptr(), at, at + 4 * (b + 1),
            at + 4 * (2 * b + 1), _raw_stream(dev.index)), "attn_sink_page_plan")
        return PagePlan(slots, positions, *small.split_with_sizes((b + 1, b, 1)))


def axis_sections(*sections: int) -> list[int]:
    """pair_axis of qkv_rope for whole sections of pairs: the first sections[0]
    pairs turn with axis 0, the next sections[1] with axis 1, and so on."""
    return [axis for axis, n in enumerate(sections) for _ in range(n)]


def make_rope_params(tokens: int, heads_q: int, heads_kv: int, *, rotary_dim: int,
                     row_stride: int, num_axes: int = 1, pair_axis=None,
                     interleaved: bool = False, norm: bool = False, weight_bf16: bool = False,
                     eps: float = 1e-6, amplitude: float = 1.0, page_size: int = 0,
                     num_pages: int = 0, grad_dtype: int = 0,
                     head_dim: int = 64) -> AttnSinkRopeParams:
    """Params of attn_sink_qkv_rope / _bwd for a packed projection whose tokens
    are row_stride elements apart."""
    p = AttnSinkRopeParams()
    _in_32_bits(tokens=tokens, heads_q=heads_q, heads_kv=heads_kv, num_axes=num_axes,
                page_size=page_size, num_pages=num_pages)
    p.q_stride = p.k_stride = p.v_stride = row_stride
    p.tokens, p.heads_q, p.heads_kv, p.head_dim = tokens, heads_q, heads_kv, head_dim
    p.rotary_dim, p.interleaved, p.num_axes = rotary_dim, int(interleaved), num_axes
    if pair_axis is not None:
        ctypes.memmove(p.pair_axis, bytes(pair_axis), len(pair_axis))
    p.norm, p.weight_bf16, p.eps, p.amplitude = int(norm), int(weight_bf16), eps, amplitude
    p.page_size, p.num_pages, p.grad_dtype = page_size, num_pages, grad_dtype
    return p


@functools.lru_cache(maxsize=256)
def _rope_params_of(t, heads_q, heads_kv, pairs, stride, axes, pair_axis, norm, weight_bf16, eps,
                    interleaved, amplitude, page_size, num_pages, grad_dtype):
    """The params of a shape, kept for its next call (they are only read)."""
    if pairs > 32:
        raise ValueError(f"inv_freq has {pairs} entries: a head has 32 pairs")
    if pair_axis is None:
        if axes > 1:
            raise ValueError("positions with several axes need pair_axis")
    elif len(pair_axis) != pairs or max(pair_axis, default=0) >= axes:
        raise ValueError(f"pair_axis needs {pairs} entries in [0, {axes}), one per pair")
    return make_rope_params(t, heads_q, heads_kv, rotary_dim=2 * pairs, row_stride=stride,
                            num_axes=axes, pair_axis=pair_axis, interleaved=interleaved, norm=norm,
                            weight_bf16=weight_bf16, eps=eps, amplitude=amplitude,
                            page_size=page_size, num_pages=num_pages, grad_dtype=grad_dtype)


def _rope_params(qkv, positions, inv_freq, heads_q, heads_kv, q_weight, k_weight, pair_axis,
                 eps=1e-6, interleaved=False, amplitude=1.0, page_size=0, num_pages=0,
                 grad_dtype=0) -> AttnSinkRopeParams:
    """Checks of qkv_rope and its backward, and their params."""
    dev, rows = qkv.device, heads_q + 2 * heads_kv
    t = _dims("qkv", qkv, 3)[0]
    if qkv.dtype is not torch.bfloat16 or qkv.shape != (t, rows, 64):
        raise ValueError(f"qkv has to be bfloat16 [T, {rows}, 64], not {qkv.dtype} "
                         f"{tuple(qkv.shape)}")
    stride, head, one = qkv.stride()
    if t and (one != 1 or head != 64 or stride < rows * 64 or stride % 8):
        if t > 1 or one != 1 or head != 64:
            raise ValueError("qkv: the heads of a token have to be contiguous and the tokens a "
                             f"multiple of 8 elements apart (strides {tuple(qkv.stride())})")
        stride = rows * 64                  # a single token: its stride means nothing
    elif t == 0:
        stride = rows * 64
    axes = positions.shape[0] if positions.dim() == 2 else 1
    _want("positions", positions, torch.int32, dev, (axes, t) if positions.dim() == 2 else (t,))
    pairs, = _dims("inv_freq", inv_freq, 1)
    _want("inv_freq", inv_freq, torch.float32, dev, (pairs,))
    norm = q_weight is not None
    if norm != (k_weight is not None):
        raise ValueError("q_weight and k_weight go together")
    if norm:
        kind = q_weight.dtype
        if kind is not torch.float32 and kind is not torch.bfloat16:
            raise ValueError(f"q_weight has to be float32 or bfloat16, not {kind}")
        _want("q_weight", q_weight, kind, dev, (64,))
        _want("k_weight", k_weight, kind, dev, (64,))
    if pair_axis is not None:
        try:
            pair_axis = bytes(pair_axis)
        except ValueError:
            raise ValueError(f"pair_axis: entries in [0, {axes})") from None
    return _rope_params_of(t, heads_q, heads_kv, pairs, stride, axes, pair_axis, norm,
                           norm and kind is torch.bfloat16, eps, interleaved, amplitude, page_size,
                           num_pages, grad_dtype)


def _at(t):
    return None if t is None else t.data_ptr()


def qkv_rope(qkv, positions, inv_freq, *, heads_q: int, heads_kv: int, q_weight=None,
             k_weight=None, eps: float = 1e-6, pair_axis=None, interleaved: bool = False,
             amplitude: float = 1.0, slots=None, k_cache=None, v_cache=None,
             keep_kv: bool | None = None, stream=None):
    """(q, k, v) of a packed projection qkv [T, heads_q + 2 heads_kv, 64] bf16
    (attn_sink_qkv_rope): q and k normalised per head (with q_weight and k_weight
    [64], fp32 or bf16; None: no norm) and rotated by positions [T] or [axes, T]
    int32, inv_freq [rotary_dim / 2] fp32.  Pair i turns with the axis
    pair_axis[i] (see axis_sections); interleaved pairs are (2i, 2i + 1), the
    others (i, i + rotary_dim / 2); amplitude multiplies the rotated dimensions.
    With slots [T] int64, k and v are written to those rows of k_cache and
    v_cache [pages, page_size, heads_kv, 64], and k and v are None unless
    keep_kv."""
    if stream is None:
        r = (_FAST or _fast()).qkv_rope(qkv, positions, inv_freq, heads_q, heads_kv, q_weight,
                                        k_weight, eps, pair_axis, interleaved, amplitude, slots,
                                        k_cache, v_cache, keep_kv)
        if r is not None:
            if type(r) is int:
                _check(r, "attn_sink_qkv_rope")
            return r
    paged = slots is not None
    pages = page = 0
    if paged:
        if k_cache is None or v_cache is None:
            raise ValueError("slots need k_cache and v_cache")
        pages, page = _dims("k_cache", k_cache, 4)[:2]
    elif k_cache is not None or v_cache is not None:
        raise ValueError("k_cache and v_cache need slots")
    p = _rope_params(qkv, positions, inv_freq, heads_q, heads_kv, q_weight, k_weight, pair_axis,
                     eps, interleaved, amplitude, page, pages)
    dev, t, bf16 = qkv.device, qkv.shape[0], torch.bfloat16
    if paged:
        _want("slots", slots, torch.int64, dev, (t,))
        _want("k_cache", k_cache, bf16, dev, (pages, page, heads_kv, 64))
        _want("v_cache", v_cache, bf16, dev, (pages, page, heads_kv, 64))
    keep = not paged if keep_kv is None else keep_kv
    with _on(dev, stream):
        q = torch.empty((t, heads_q, 64), dtype=bf16, device=dev)
        k = torch.empty((t, heads_kv, 64), dtype=bf16, device=dev) if keep else None
        v = torch.empty((t, heads_kv, 64), dtype=bf16, device=dev) if keep else None
        base = qkv.data_ptr()
        _check(lib().attn_sink_qkv_rope(
            ctypes.byref(p), base, base + 128 * heads_q, base + 128 * (heads_q + heads_kv),
            positions.data_ptr(), inv_freq.data_ptr(), _at(q_weight), _at(k_weight), _at(slots),
            q.data_ptr(), _at(k), _at(v), _at(k_cache), _at(v_cache), _raw_stream(dev.index)),
            "attn_sink_qkv_rope")
    return q, k, v


def qkv_rope_backward(qkv, positions, inv_freq, dq, dk, dv, *, heads_q: int, heads_kv: int,
                      q_weight=None, k_weight=None, eps: float = 1e-6, pair_axis=None,
                      interleaved: bool = False, amplitude: float = 1.0, stream=None):
    """(dqkv, dq_weight, dk_weight) of qkv_rope (attn_sink_qkv_rope_bwd): dq
    [T, heads_q, 64], dk and dv [T, heads_kv, 64], all bf16 or all fp32 (as
    backward gives them); dqkv [T, heads_q + 2 heads_kv, 64] bf16, the weights'
    gradients [64] fp32 (None without norm), bitwise reproducible."""
    if stream is None:
        r = (_FAST or _fast()).qkv_rope_backward(qkv, positions, inv_freq, heads_q, heads_kv,
                                                 q_weight, k_weight, eps, pair_axis, interleaved,
                                                 amplitude, dq, dk, dv)
        if r is not None:
            if type(r) is int:
                _check(r, "attn_sink_qkv_rope_bwd")
            return r
    kind = dq.dtype
    if kind is not torch.float32 and kind is not torch.bfloat16:
        raise ValueError(f"dq has to be float32 or bfloat16, not {kind}")
    p = _rope_params(qkv, positions, inv_freq, heads_q, heads_kv, q_weight, k_weight, pair_axis,
                     eps, interleaved, amplitude, 0, 0, int(kind is torch.float32))
    dev, t, rows = qkv.device, qkv.shape[0], heads_q + 2 * heads_kv
    _want("dq", dq, kind, dev, (t, heads_q, 64))
    _want("dk", dk, kind, dev, (t, heads_kv, 64))
    _want("dv", dv, kind, dev, (t, heads_kv, 64))
    with _on(dev, stream):
        dqkv = torch.empty((t, rows, 64), dtype=torch.bfloat16, device=dev)
        dwq = dwk = ws = None
        nbytes = 0
        if p.norm:
            dwq, dwk = torch.empty((2, 64), dtype=torch.float32, device=dev).unbind()
            nbytes = attn_sink_qkv_rope_bwd_workspace_size(p)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        src, dst, kq, kk = qkv.data_ptr(), dqkv.data_ptr(), 128 * heads_q, 128 * heads_kv
        _check(lib().attn_sink_qkv_rope_bwd(
            ctypes.byref(p), src, src + kq, positions.data_ptr(), inv_freq.data_ptr(),
            _at(q_weight), _at(k_weight), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dst,
            dst + kq, dst + kq + kk, rows * 64, rows * 64, rows * 64, _at(dwq), _at(dwk), _at(ws),
            nbytes, _raw_stream(dev.index)), "attn_sink_qkv_rope_bwd")
    return dqkv, dwq, dwk


class QkvRopeFunction(torch.autograd.Function):
    """Autograd wrapper of qkv_rope and qkv_rope_backward."""

    @staticmethod
    def forward(ctx, qkv, q_weight, k_weight, positions, inv_freq, cfg):
        ctx.save_for_backward(qkv, q_weight, k_weight, positions, inv_freq)
        ctx.cfg = cfg
        return qkv_rope(qkv, positions, inv_freq, q_weight=q_weight, k_weight=k_weight, **cfg)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk, dv):
        qkv, qw, kw, positions, inv_freq = ctx.saved_tensors
        dqkv, dqw, dkw = qkv_rope_backward(qkv, positions, inv_freq, dq.contiguous(),
                                           dk.contiguous(), dv.contiguous(), q_weight=qw,
                                           k_weight=kw, **ctx.cfg)
        if dqw is not None:
            dqw, dkw = dqw.to(qw.dtype), dkw.to(kw.dtype)
        return dqkv, dqw, dkw, None, None, None


def qkv_rope_autograd(qkv, positions, inv_freq, *, heads_q: int, heads_kv: int, q_weight=None,
                      k_weight=None, eps: float = 1e-6, pair_axis=None,
                      interleaved: bool = False, amplitude: float = 1.0):
    """qkv_rope with gradients to qkv, q_weight and k_weight (training).  inv_freq
    is a constant: one that requires a gradient is refused.  To capture a
    backward pass into a CUDA graph, call qkv_rope_backward itself."""
    if inv_freq.requires_grad:
        raise ValueError("inv_freq has no gradient here")
    cfg = dict(heads_q=heads_q, heads_kv=heads_kv, eps=eps, pair_axis=pair_axis,
               interleaved=interleaved, amplitude=amplitude)
    return QkvRopeFunction.apply(qkv, q_weight, k_weight, positions, inv_freq, cfg)


def extend(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, sink, *, window: int = 0,
           softmax_scale: float | None = None, out=None, lse=None, stream=None):
    """(out, lse) of several new tokens per sequence over a paged cache
    (attn_sink_extend): q [T, H_q, 64] packed by cu_seqlens_q [B + 1] int32,
    caches [pages, page_size, H_kv, 64] that hold the new tokens' keys too,
    block_table [B, max_pages] int32, seq_lens [B] int32 (cached + new), sink
    [H_q] fp32.  Rows of out and lse behind cu_seqlens_q[B] are not written:
    give out and lse to keep what they hold there."""
    if softmax_scale is None:
        softmax_scale = 0.125
    if stream is None:
        r = (_FAST or _fast()).extend(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q,
                                      sink, window, softmax_scale, out, lse)
        if r is not None:
            if type(r) is int:
                _check(r, "attn_sink_extend")
            return r
    dev, bf16, i32 = q.device, torch.bfloat16, torch.int32
    b, = _dims("seq_lens", seq_lens, 1)
    t, hq, _ = _dims("q", q, 3)
    pages, page, hkv, _ = _dims("k_cache", k_cache, 4)
    cols = _dims("block_table", block_table, 2)[1]
    _want("q", q, bf16, dev, (t, hq, 64))
    _want("k_cache", k_cache, bf16, dev, (pages, page, hkv, 64))
    _want("v_cache", v_cache, bf16, dev, (pages, page, hkv, 64))
    _want("block_table", block_table, i32, dev, (b, cols))
    _want("seq_lens", seq_lens, i32, dev, (b,))
    _want("cu_seqlens_q", cu_seqlens_q, i32, dev, (b + 1,))
    _want("sink", sink, torch.float32, dev, (hq,))
    if out is not None:
        _want("out", out, bf16, dev, (t, hq, 64))
    if lse is not None:
        _want("lse", lse, torch.float32, dev, (hq, t))
    _in_32_bits(seq_lens=b, q=max(t, hq), k_cache=max(pages, page, hkv), block_table=cols)
    window = min(max(window, 0), 2 ** 31 - 1)             # any length is below 2^30
    p = AttnSinkExtendParams(b, t, hq, hkv, 64, page, pages, cols, window, softmax_scale)
    with _on(dev, stream):
        if out is None:
            out = torch.empty((t, hq, 64), dtype=bf16, device=dev)
        if lse is None:
            lse = torch.empty((hq, t), dtype=torch.float32, device=dev)
        nbytes = lib().attn_sink_extend_workspace_size(ctypes.byref(p))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check(lib().attn_sink_extend(
            ctypes.byref(p), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens_q.data_ptr(), sink.data_ptr(),
            out.data_ptr(), lse.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(dev.index)),
            "attn_sink_extend")
    return out, lse


# ----------------------------------------------------------------------------- include/attn_sink_cache.h
def attn_sink_decode_shared_workspace_size(params: AttnSinkSharedParams) -> int:
    return int(lib().attn_sink_decode_shared_workspace_size(_pref(params)))


def attn_sink_decode_shared(params: AttnSinkSharedParams, q, k_cache, v_cache, block_table,
                            seq_lens, cu_groups, prefix_lens, sink, out, lse, workspace,
                            workspace_bytes: int, stream=None) -> int:
    return lib().attn_sink_decode_shared(_pref(params), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                         _ptr(block_table), _ptr(seq_lens), _ptr(cu_groups),
                                         _ptr(prefix_lens), _ptr(sink), _ptr(out), _ptr(lse),
                                         _ptr(workspace), int(workspace_bytes), _stream(stream))


def attn_sink_page_bounds(params: AttnSinkBoundsParams, k_cache, block_table, cached_lens,
                          seq_lens, bounds, stream=None) -> int:
    return lib().attn_sink_page_bounds(_pref(params), _ptr(k_cache), _ptr(block_table),
                                       _ptr(cached_lens), _ptr(seq_lens), _ptr(bounds),
                                       _stream(stream))


def attn_sink_select_pages_workspace_size(params: AttnSinkSelectParams) -> int:
    return int(lib().attn_sink_select_pages_workspace_size(_pref(params)))


def attn_sink_select_pages(params: AttnSinkSelectParams, q, bounds, block_table, seq_lens,
                           selected, workspace, workspace_bytes: int, stream=None) -> int:
    return lib().attn_sink_select_pages(_pref(params), _ptr(q), _ptr(bounds), _ptr(block_table),
                                        _ptr(seq_lens), _ptr(selected), _ptr(workspace),
                                        int(workspace_bytes), _stream(stream))


def attn_sink_decode_pages_workspace_size(params: AttnSinkPagesParams) -> int:
    return int(lib().attn_sink_decode_pages_workspace_size(_pref(params)))


def attn_sink_decode_pages(params: AttnSinkPagesParams, q, k_cache, v_cache, block_table,
                           seq_lens, selected, sink, out, lse, workspace, workspace_bytes: int,
                           stream=None) -> int:
    return lib().attn_sink_decode_pages(_pref(params), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(block_table), _ptr(seq_lens), _ptr(selected),
                                        _ptr(sink), _ptr(out), _ptr(lse), _ptr(workspace),
                                        int(workspace_bytes), _stream(stream))


def attn_sink_key_mass(params: AttnSinkMassParams, q, k_cache, block_table, seq_lens,
                       cu_seqlens_q, lse, mass, stream=None) -> int:
    return lib().attn_sink_key_mass(_pref(params), _ptr(q), _ptr(k_cache), _ptr(block_table),
                                    _ptr(seq_lens), _ptr(cu_seqlens_q), _ptr(lse), _ptr(mass),
                                    _stream(stream))


def attn_sink_evict_workspace_size(params: AttnSinkEvictParams) -> int:
    return int(lib().attn_sink_evict_workspace_size(_pref(params)))


def attn_sink_evict(params: AttnSinkEvictParams, k_cache, v_cache, block_table, seq_lens, mass,
                    mass_out, new_lens, freed_pages, num_freed, workspace, workspace_bytes: int,
                    stream=None) -> int:
    return lib().attn_sink_evict(_pref(params), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                 _ptr(seq_lens), _ptr(mass), _ptr(mass_out), _ptr(new_lens),
                                 _ptr(freed_pages), _ptr(num_freed), _ptr(workspace),
                                 int(workspace_bytes), _stream(stream))


def _paged(k_cache, v_cache, block_table, seq_lens, dev):
    """Checks of a paged cache and its tables; (batch, pages, page size, kv heads,
    columns).  v_cache may be None."""
    b, = _dims("seq_lens", seq_lens, 1)
    pages, page, hkv, _ = _dims("k_cache", k_cache, 4)
    cols = _dims("block_table", block_table, 2)[1]
    _want("k_cache", k_cache, torch.bfloat16, dev, (pages, page, hkv, 64))
    if v_cache is not None:
        _want("v_cache", v_cache, torch.bfloat16, dev, (pages, page, hkv, 64))
    _want("block_table", block_table, torch.int32, dev, (b, cols))
    _want("seq_lens", seq_lens, torch.int32, dev, (b,))
    _in_32_bits(seq_lens=b, k_cache=max(pages, page, hkv), block_table=cols)
    return b, pages, page, hkv, cols


def decode_shared(q, k_cache, v_cache, block_table, seq_lens, cu_groups, prefix_lens, sink, *,
                  softmax_scale: float | None = None, out=None, lse=None, stream=None):
    """(out, lse) of one decode step over a paged cache in which groups of sequences
    share their first keys (attn_sink_decode_shared): decode with, beside its
    arguments, cu_groups [P + 1] int32, the groups' first sequences from 0 to B, and
    prefix_lens [P] int32, how many keys each group shares.  Those are read through
    the block-table row of the group's first sequence, once for all of it."""
    if softmax_scale is None:
        softmax_scale = 0.125
    if stream is None:
        r = (_FAST or _fast()).decode_shared(q, k_cache, v_cache, block_table, seq_lens, cu_groups,
                                             prefix_lens, sink, softmax_scale, out, lse)
        if r is not None:
            if type(r) is int:
                _check(r, "attn_sink_decode_shared")
            return r
    dev, i32 = q.device, torch.int32
    b, pages, page, hkv, cols = _paged(k_cache, v_cache, block_table, seq_lens, dev)
    hq = _dims("q", q, 3)[1]
    groups, = _dims("prefix_lens", prefix_lens, 1)
    _want("q", q, torch.bfloat16, dev, (b, hq, 64))
    _want("cu_groups", cu_groups, i32, dev, (groups + 1,))
    _want("prefix_lens", prefix_lens, i32, dev, (groups,))
    _want("sink", sink, torch.float32, dev, (hq,))
    _in_32_bits(q=hq, prefix_lens=groups)
    out, lse = _results(out, lse, q, dev, stream)
    p = AttnSinkSharedParams(b, groups, hq, hkv, 64, page, pages, cols, softmax_scale)
    with _on(dev, stream):
        nbytes = attn_sink_decode_shared_workspace_size(p)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check(attn_sink_decode_shared(p, q, k_cache, v_cache, block_table, seq_lens, cu_groups,
                                       prefix_lens, sink, out, lse, ws, nbytes,
                                       _raw_stream(dev.index)), "attn_sink_decode_shared")
    return out, lse


def _results(out, lse, q, dev, stream):
    """out [T, H_q, 64] and lse [H_q, T] of a call with these queries: the caller's own,
    checked, or new ones."""
    t, hq, _ = q.shape
    if out is not None:
        _want("out", out, torch.bfloat16, dev, (t, hq, 64))
    if lse is not None:
        _want("lse", lse, torch.float32, dev, (hq, t))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((t, hq, 64), dtype=torch.bfloat16, device=dev)
        if lse is None:
            lse = torch.empty((hq, t), dtype=torch.float32, device=dev)
    return out, lse


def page_bounds(k_cache, block_table, cached_lens, seq_lens, bounds, *, stream=None) -> None:
    """Bring the bounds [pages, heads_kv, 2, 64] bf16 of a paged cache's keys (the
    elementwise minimum and maximum over each page) up to date after keys
    [cached_lens[b], seq_lens[b]) of every sequence were written
    (attn_sink_page_bounds); in place."""
    if stream is None:
        r = (_FAST or _fast()).page_bounds(k_cache, block_table, cached_lens, seq_lens, bounds)
        if r is not None:
            _check(r, "attn_sink_page_bounds")
            return
    dev = k_cache.device
    b, pages, page, hkv, cols = _paged(k_cache, None, block_table, seq_lens, dev)
    _want("cached_lens", cached_lens, torch.int32, dev, (b,))
    _want("bounds", bounds, torch.bfloat16, dev, (pages, hkv, 2, 64))
    p = AttnSinkBoundsParams(b, hkv, 64, page, pages, cols)
    with _on(dev, stream):
        _check(attn_sink_page_bounds(p, k_cache, block_table, cached_lens, seq_lens, bounds,
                                     _raw_stream(dev.index)), "attn_sink_page_bounds")


def select_pages(q, bounds, block_table, seq_lens, *, count: int, page_size: int,
                 keep_first: int = 1, keep_last: int = 1, stream=None):
    """The pages of each sequence and kv head whose bounds promise the largest scores
    for the new token's queries q [B, H_q, 64] (attn_sink_select_pages): selected
    [B, heads_kv, count] int32, columns of the block table in ascending order, -1
    behind the last.  The first keep_first and the last keep_last pages are always
    there."""
    if stream is None:
        r = (_FAST or _fast()).select_pages(q, bounds, block_table, seq_lens, count, page_size,
                                            keep_first, keep_last)
        if r is not None:
            if type(r) is int:
                _check(r, "attn_sink_select_pages")
            return r
    dev, i32 = q.device, torch.int32
    b, = _dims("seq_lens", seq_lens, 1)
    hq = _dims("q", q, 3)[1]
    pages, hkv = _dims("bounds", bounds, 4)[:2]
    cols = _dims("block_table", block_table, 2)[1]
    _want("q", q, torch.bfloat16, dev, (b, hq, 64))
    _want("bounds", bounds, torch.bfloat16, dev, (pages, hkv, 2, 64))
    _want("block_table", block_table, i32, dev, (b, cols))
    _want("seq_lens", seq_lens, i32, dev, (b,))
    if count < 1:
        raise ValueError(f"count is {count}")
    _in_32_bits(seq_lens=b, q=hq, bounds=max(pages, hkv), block_table=cols, count=count,
                page_size=page_size, keep_first=keep_first, keep_last=keep_last)
    p = AttnSinkSelectParams(b, hq, hkv, 64, page_size, pages, cols, count, keep_first, keep_last)
    with _on(dev, stream):
        selected = torch.empty((b, hkv, count), dtype=i32, device=dev)
        nbytes = attn_sink_select_pages_workspace_size(p)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check(attn_sink_select_pages(p, q, bounds, block_table, seq_lens, selected, ws, nbytes,
                                      _raw_stream(dev.index)), "attn_sink_select_pages")
    return selected


def decode_pages(q, k_cache, v_cache, block_table, seq_lens, selected, sink, *,
                 softmax_scale: float | None = None, out=None, lse=None, stream=None):
    """(out, lse) of one decode step over the selected pages alone
    (attn_sink_decode_pages): decode with, beside its arguments, selected [B,
    heads_kv, count] int32, the columns of the block table each kv head reads (as
    select_pages gives them; a negative entry is none)."""
    if softmax_scale is None:
        softmax_scale = 0.125
    if stream is None:
        r = (_FAST or _fast()).decode_pages(q, k_cache, v_cache, block_table, seq_lens, selected,
                                            sink, softmax_scale, out, lse)
        if r is not None:
            if type(r) is int:
                _check(r, "attn_sink_decode_pages")
            return r
    dev = q.device
    b, pages, page, hkv, cols = _paged(k_cache, v_cache, block_table, seq_lens, dev)
    hq = _dims("q", q, 3)[1]
    count = _dims("selected", selected, 3)[2]
    _want("q", q, torch.bfloat16, dev, (b, hq, 64))
    _want("selected", selected, torch.int32, dev, (b, hkv, count))
    _want("sink", sink, torch.float32, dev, (hq,))
    _in_32_bits(q=hq, selected=count)
    out, lse = _results(out, lse, q, dev, stream)
    p = AttnSinkPagesParams(b, hq, hkv, 64, page, pages, cols, count, softmax_scale)
    with _on(dev, stream):
        nbytes = attn_sink_decode_pages_workspace_size(p)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check(attn_sink_decode_pages(p, q, k_cache, v_cache, block_table, seq_lens, selected,
                                      sink, out, lse, ws, nbytes, _raw_stream(dev.index)),
               "attn_sink_decode_pages")
    return out, lse


def key_mass(q, k_cache, block_table, seq_lens, cu_seqlens_q, lse, mass, *,
             accumulate: bool = True, softmax_scale: float | None = None, stream=None):
    """The attention weight each cached key gets from the new tokens, summed over them
    and over the query heads of its kv head (attn_sink_key_mass): added to mass [B,
    heads_kv, C] fp32 in place (accumulate False: written, the rest of a row zero).
    q [T, H_q, 64] packed by cu_seqlens_q [B + 1] int32 and lse [H_q, T] as extend,
    decode and the calls above took and gave them.  Single tokens and chunks of prompts
    belong in calls of their own (attn_sink_cache.h says why).  Returns mass."""
    if softmax_scale is None:
        softmax_scale = 0.125
    if stream is None:
        r = (_FAST or _fast()).key_mass(q, k_cache, block_table, seq_lens, cu_seqlens_q, lse, mass,
                                        accumulate, softmax_scale)
        if r is not None:
            _check(r, "attn_sink_key_mass")
            return mass
    dev = q.device
    b, pages, page, hkv, cols = _paged(k_cache, None, block_table, seq_lens, dev)
    t, hq, _ = _dims("q", q, 3)
    keys = _dims("mass", mass, 3)[2]
    _want("q", q, torch.bfloat16, dev, (t, hq, 64))
    _want("cu_seqlens_q", cu_seqlens_q, torch.int32, dev, (b + 1,))
    _want("lse", lse, torch.float32, dev, (hq, t))
    _want("mass", mass, torch.float32, dev, (b, hkv, keys))
    _in_32_bits(q=max(t, hq), mass=keys)
    p = AttnSinkMassParams(b, t, hq, hkv, 64, page, pages, cols, keys, int(bool(accumulate)),
                           softmax_scale)
    with _on(dev, stream):
        _check(attn_sink_key_mass(p, q, k_cache, block_table, seq_lens, cu_seqlens_q, lse, mass,
                                  _raw_stream(dev.index)), "attn_sink_key_mass")
    return mass


class Evicted(NamedTuple):
    """What evict leaves beside the caches (see there)."""
    seq_lens: torch.Tensor       # [B] int32: min(length, budget)
    mass: torch.Tensor           # [B, heads_kv, C] fp32: the kept keys' at their new places
    freed_pages: torch.Tensor    # [B * max_pages] int32, -1 behind the last
    num_freed: torch.Tensor      # [1] int32


def evict(k_cache, v_cache, block_table, seq_lens, mass, *, budget: int, keep_first: int = 0,
          keep_last: int = 0, stream=None) -> Evicted:
    """Cut every sequence down to budget keys (attn_sink_evict): each kv head keeps its
    first keep_first, its last keep_last and otherwise those with the largest mass
    [B, heads_kv, C] fp32; the kept ones at positions >= budget move into the holes
    below, in k_cache and v_cache in place.  freed_pages are the pages that hold no
    key any more, a free list for page_plan.  A head's keys are then no longer in the
    order of their tokens: no windows on such a cache, bounds to be made anew
    (page_bounds with cached_lens = 0), and new tokens go on with positions of their
    own."""
    if stream is None:
        r = (_FAST or _fast()).evict(k_cache, v_cache, block_table, seq_lens, mass, budget,
                                     keep_first, keep_last)
        if r is not None:
            if type(r) is int:
                _check(r, "attn_sink_evict")
            return Evicted(*r)
    dev, i32 = k_cache.device, torch.int32
    b, pages, page, hkv, cols = _paged(k_cache, v_cache, block_table, seq_lens, dev)
    keys = _dims("mass", mass, 3)[2]
    _want("mass", mass, torch.float32, dev, (b, hkv, keys))
    _in_32_bits(mass=keys, budget=budget, keep_first=keep_first, keep_last=keep_last,
                block_table=b * cols)
    p = AttnSinkEvictParams(b, hkv, 64, page, pages, cols, keys, budget, keep_first, keep_last,
                            b * cols)
    with _on(dev, stream):
        mass_out = torch.empty_like(mass)
        lens = torch.empty(b, dtype=i32, device=dev)
        freed = torch.empty(b * cols, dtype=i32, device=dev)
        count = torch.empty(1, dtype=i32, device=dev)
        nbytes = attn_sink_evict_workspace_size(p)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check(attn_sink_evict(p, k_cache, v_cache, block_table, seq_lens, mass, mass_out, lens,
                               freed, count, ws, nbytes, _raw_stream(dev.index)),
               "attn_sink_evict")
    return Evicted(lens, mass_out, freed, count)
