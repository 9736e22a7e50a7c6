"""ctypes binding of the C ABI in ``include/spa.h`` (argument marshalling only).

Every function takes the same arguments as its C counterpart; device buffers
may be given as torch tensors (their ``data_ptr()``) or as raw integer
addresses, and ``stream`` as a ``torch.cuda.Stream``, a raw handle or ``None``
(the current torch stream).  All computation happens in ``lib/libspa.so``;
there is no fallback: importing this module fails loudly when the library has
not been built.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional

try:                        # device memory and streams; raw addresses need neither
    import torch as _torch
except ImportError:  # pragma: no cover
    _torch = None

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libspa.so")

SPA_OK, SPA_ERR_INVALID, SPA_ERR_UNSUPPORTED, SPA_ERR_WORKSPACE, SPA_ERR_CUDA, SPA_ERR_TIMEOUT = range(6)
SPA_MODE_ANCHOR, SPA_MODE_SALE, SPA_MODE_DENSE = 0, 1, 2
SPA_DEBUG_STALL_ATTN = 0x1
MODES = {"anchor": SPA_MODE_ANCHOR, "sale": SPA_MODE_SALE, "dense": SPA_MODE_DENSE}

EXPORTED = ("sparse_prefill_workspace_bytes", "sparse_prefill_plan", "sparse_prefill_attn",
            "sparse_prefill_stats", "sparse_prefill_status_string", "sparse_prefill_plan_static",
            "sparse_decode_scratch_bytes", "sparse_decode_prepare", "sparse_decode_attn",
            "sparse_fp8_scales_floats", "sparse_fp8_scratch_bytes", "sparse_fp8_quantize",
            "sparse_prefill_attn_fp8", "sparse_key_mass", "sparse_qk_norm_rope",
            "sparse_paged_append", "sparse_paged_workspace_bytes",
            "sparse_paged_attn_workspace_bytes", "sparse_paged_select", "sparse_paged_attn",
            "sparse_paged_status")


class SpaParams(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_kv", ctypes.c_int32),
        ("seq_len", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("causal", ctypes.c_int32),
        ("block_q", ctypes.c_int32), ("block_k", ctypes.c_int32), ("sink", ctypes.c_int32),
        ("local", ctypes.c_int32), ("step", ctypes.c_int32), ("mode", ctypes.c_int32),
        ("theta", ctypes.c_float), ("tau", ctypes.c_float), ("softmax_scale", ctypes.c_float),
        ("wait_limit_us", ctypes.c_uint32), ("debug_flags", ctypes.c_uint32),
        ("tau_per_head", ctypes.POINTER(ctypes.c_float)),
    ]


class SpaStats(ctypes.Structure):
    _fields_ = [
        ("error_bits", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
        ("query_blocks", ctypes.c_int64), ("candidates", ctypes.c_int64),
        ("kept_candidates", ctypes.c_int64), ("kept_pairs", ctypes.c_int64),
        ("dense_pairs", ctypes.c_int64),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_ if name != "reserved"}


class SpaRows(ctypes.Structure):
    """A view of bf16 rows of 128: address and element strides (``spa_rows``)."""

    _fields_ = [("data", ctypes.c_void_p), ("stride_batch", ctypes.c_int64),
                ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class SpaRopeParams(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("heads_q", ctypes.c_int32),
        ("heads_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("table_rows", ctypes.c_int32), ("eps", ctypes.c_float),
    ]


class SpaPagedParams(ctypes.Structure):
    _fields_ = [
        ("heads_q", ctypes.c_int32), ("heads_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("pages_per_seq", ctypes.c_int32), ("seqs", ctypes.c_int32), ("tokens", ctypes.c_int32),
        ("page_stride", ctypes.c_int64), ("softmax_scale", ctypes.c_float),
        ("sink_pages", ctypes.c_int32), ("local_pages", ctypes.c_int32),
        ("top_pages", ctypes.c_int32), ("wait_limit_us", ctypes.c_uint32),
        ("debug_flags", ctypes.c_uint32),
    ]


class SpaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {sparse_prefill_status_string(status)} (status {status})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m block_sparse_long_sm_b200.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(SpaParams)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.sparse_prefill_workspace_bytes.argtypes = [P]
    lib.sparse_prefill_workspace_bytes.restype = sz
    lib.sparse_prefill_plan.argtypes = [P, vp, vp, vp, sz, vp]
    lib.sparse_prefill_plan.restype = ctypes.c_int
    lib.sparse_prefill_attn.argtypes = [P, vp, vp, vp, vp, sz, vp, vp, vp]
    lib.sparse_prefill_attn.restype = ctypes.c_int
    lib.sparse_prefill_stats.argtypes = [P, vp, sz, ctypes.POINTER(SpaStats), vp]
    lib.sparse_prefill_stats.restype = ctypes.c_int
    lib.sparse_prefill_plan_static.argtypes = [P, vp, vp, vp, vp, sz, vp, vp]
    lib.sparse_prefill_plan_static.restype = ctypes.c_int
    i32 = ctypes.c_int32
    lib.sparse_decode_scratch_bytes.argtypes = [P, i32]
    lib.sparse_decode_scratch_bytes.restype = sz
    lib.sparse_decode_prepare.argtypes = [P, i32, vp, sz, vp, sz, vp]
    lib.sparse_decode_prepare.restype = ctypes.c_int
    lib.sparse_decode_attn.argtypes = [P, vp, vp, vp, i32, i32, vp, sz, vp, sz, vp, vp, vp]
    lib.sparse_decode_attn.restype = ctypes.c_int
    lib.sparse_fp8_scales_floats.argtypes = [P]
    lib.sparse_fp8_scales_floats.restype = sz
    lib.sparse_fp8_scratch_bytes.argtypes = [P]
    lib.sparse_fp8_scratch_bytes.restype = sz
    lib.sparse_fp8_quantize.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.sparse_fp8_quantize.restype = ctypes.c_int
    lib.sparse_prefill_attn_fp8.argtypes = [P, vp, vp, vp, vp, vp, sz, vp, vp, vp]
    lib.sparse_prefill_attn_fp8.restype = ctypes.c_int
    lib.sparse_key_mass.argtypes = [P, vp, vp, vp, i32, vp, sz, vp, vp]
    lib.sparse_key_mass.restype = ctypes.c_int
    R, G = ctypes.POINTER(SpaRopeParams), ctypes.POINTER(SpaPagedParams)
    rows = vp                        # a reference to an SpaRows, or the bytes of one
    lib.sparse_qk_norm_rope.argtypes = [R, rows, rows, vp, vp, vp, vp, rows, rows, vp, vp]
    lib.sparse_qk_norm_rope.restype = ctypes.c_int
    lib.sparse_paged_append.argtypes = [G, R, rows, rows, rows, vp, vp, vp, vp, vp, vp, rows, vp,
                                        vp, vp, vp, vp]
    lib.sparse_paged_append.restype = ctypes.c_int
    lib.sparse_paged_workspace_bytes.argtypes = [G]
    lib.sparse_paged_workspace_bytes.restype = sz
    lib.sparse_paged_attn_workspace_bytes.argtypes = [G]
    lib.sparse_paged_attn_workspace_bytes.restype = sz
    lib.sparse_paged_select.argtypes = [G, rows, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.sparse_paged_select.restype = ctypes.c_int
    lib.sparse_paged_attn.argtypes = [G, rows, vp, vp, vp, vp, vp, vp, vp, rows, vp, vp, sz, vp,
                                      vp]
    lib.sparse_paged_attn.restype = ctypes.c_int
    lib.sparse_paged_status.argtypes = [vp, vp]
    lib.sparse_paged_status.restype = ctypes.c_int
    lib.sparse_prefill_status_string.argtypes = [ctypes.c_int]
    lib.sparse_prefill_status_string.restype = ctypes.c_char_p
    return lib


_lib = _load()


def make_params(batch: int, heads_q: int, heads_kv: int, seq_len: int, *, mode="anchor",
                sink: int = 128, local: int = 256, theta: float = 5.0, tau: float = 1e-3,
                block_k: Optional[int] = None, softmax_scale: float = 0.0,
                wait_limit_us: int = 0, debug_flags: int = 0, head_dim: int = 128,
                causal: int = 1, block_q: int = 128, step: int = 1,
                tau_per_head=None) -> SpaParams:
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    if block_k is None:
        block_k = 32 if m == SPA_MODE_SALE else 1
    p = SpaParams(batch, heads_q, heads_kv, seq_len, head_dim, causal, block_q, block_k,
                  sink, local, step, m, float(theta), float(tau), float(softmax_scale),
                  int(wait_limit_us), int(debug_flags), None)
    if tau_per_head is not None:
        arr = (ctypes.c_float * len(tau_per_head))(*[float(t) for t in tau_per_head])
        p._tau_keepalive = arr          # the struct holds a raw pointer into this array
        p.tau_per_head = ctypes.cast(arr, ctypes.POINTER(ctypes.c_float))
    return p


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


# the current stream's handle of a device; the public torch.cuda.current_stream() builds a
# Stream object each time (3.2 us against 0.1 us a call)
_raw_stream = getattr(getattr(_torch, "_C", None), "_cuda_getCurrentRawStream", None)


def _stream(s) -> Optional[int]:
    if s.__class__ is int:
        return s
    if s is None:
        try:
            if _raw_stream is not None:
                return _raw_stream(_torch.cuda.current_device())
            return _torch.cuda.current_stream().cuda_stream
        except Exception:  # pragma: no cover - no torch / no device
            return None
    return s if isinstance(s, int) else s.cuda_stream


def _nbytes(x) -> int:
    if isinstance(x, int):
        raise TypeError("pass the workspace size explicitly when giving a raw pointer")
    return x.numel() * x.element_size()


def sparse_prefill_workspace_bytes(params: SpaParams) -> int:
    return int(_lib.sparse_prefill_workspace_bytes(ctypes.byref(params)))


def sparse_prefill_plan(params: SpaParams, q, k, workspace, workspace_bytes=None,
                        stream=None) -> int:
    wb = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    return int(_lib.sparse_prefill_plan(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(workspace),
                                        wb, _stream(stream)))


def sparse_prefill_attn(params: SpaParams, q, k, v, workspace, o, lse=None,
                        workspace_bytes=None, stream=None) -> int:
    wb = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    return int(_lib.sparse_prefill_attn(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v),
                                        _ptr(workspace), wb, _ptr(o), _ptr(lse), _stream(stream)))


def sparse_prefill_stats(params: SpaParams, workspace, workspace_bytes=None, stream=None):
    """Returns (status, SpaStats)."""
    wb = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    out = SpaStats()
    st = int(_lib.sparse_prefill_stats(ctypes.byref(params), _ptr(workspace), wb,
                                       ctypes.byref(out), _stream(stream)))
    return st, out


def sparse_prefill_plan_static(params: SpaParams, q, k, counts, lists, lists_elems=None,
                               error_word=None, stream=None) -> int:
    """Allocation-free ANCHOR plan: scratch in the library's fixed device array."""
    n = lists.numel() if lists_elems is None else int(lists_elems)
    return int(_lib.sparse_prefill_plan_static(ctypes.byref(params), _ptr(q), _ptr(k),
                                               _ptr(counts), _ptr(lists), n, _ptr(error_word),
                                               _stream(stream)))


def sparse_decode_scratch_bytes(params: SpaParams, kv_capacity: int) -> int:
    return int(_lib.sparse_decode_scratch_bytes(ctypes.byref(params), int(kv_capacity)))


def sparse_decode_prepare(params: SpaParams, kv_capacity: int, workspace, scratch,
                          workspace_bytes=None, scratch_bytes=None, stream=None) -> int:
    """Once per plan: the tagged union of each kv head's q-head selections."""
    wb = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    sb = _nbytes(scratch) if scratch_bytes is None else int(scratch_bytes)
    return int(_lib.sparse_decode_prepare(ctypes.byref(params), int(kv_capacity), _ptr(workspace),
                                          wb, _ptr(scratch), sb, _stream(stream)))


def sparse_decode_attn(params: SpaParams, q, k_cache, v_cache, kv_capacity: int, pos: int,
                       workspace, scratch, o, lse=None, workspace_bytes=None,
                       scratch_bytes=None, stream=None) -> int:
    """One decoding query per (b, q head) at position ``pos`` over sink + selection + window."""
    wb = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    sb = _nbytes(scratch) if scratch_bytes is None else int(scratch_bytes)
    return int(_lib.sparse_decode_attn(ctypes.byref(params), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                       int(kv_capacity), int(pos), _ptr(workspace), wb,
                                       _ptr(scratch), sb, _ptr(o), _ptr(lse), _stream(stream)))


def sparse_fp8_scales_floats(params: SpaParams) -> int:
    return int(_lib.sparse_fp8_scales_floats(ctypes.byref(params)))


def sparse_fp8_scratch_bytes(params: SpaParams) -> int:
    return int(_lib.sparse_fp8_scratch_bytes(ctypes.byref(params)))


def sparse_fp8_quantize(params: SpaParams, q, k, v, q8, k8, v8, scales, scratch,
                        scratch_bytes=None, stream=None) -> int:
    """E4M3 codes of q, k (mean-smoothed), v and their scales (layout in spa.h)."""
    sb = _nbytes(scratch) if scratch_bytes is None else int(scratch_bytes)
    return int(_lib.sparse_fp8_quantize(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(q8),
                                        _ptr(k8), _ptr(v8), _ptr(scales), _ptr(scratch), sb,
                                        _stream(stream)))


def sparse_prefill_attn_fp8(params: SpaParams, q8, k8, v8, scales, workspace, o, lse=None,
                            workspace_bytes=None, stream=None) -> int:
    """Attention over the plan's kept keys with E4M3 operands."""
    wb = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    return int(_lib.sparse_prefill_attn_fp8(ctypes.byref(params), _ptr(q8), _ptr(k8), _ptr(v8),
                                            _ptr(scales), _ptr(workspace), wb, _ptr(o), _ptr(lse),
                                            _stream(stream)))


def sparse_key_mass(params: SpaParams, q, k, lse, window: int, workspace, mass,
                    workspace_bytes=None, stream=None) -> int:
    """Attention mass per key from the prefill rows, from the prefill LSE."""
    wb = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    return int(_lib.sparse_key_mass(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(lse), int(window),
                                    _ptr(workspace), wb, _ptr(mass), _stream(stream)))


# ---------------------------------------------------------------------------
# the serving step around a paged cache
# ---------------------------------------------------------------------------
def make_rope_params(batch: int, tokens: int, heads_q: int, heads_kv: int, *, table_rows: int,
                     rotary_dim: int = 128, interleaved: int = 0, eps: float = 1e-6,
                     head_dim: int = 128) -> SpaRopeParams:
    return SpaRopeParams(batch, tokens, heads_q, heads_kv, head_dim, rotary_dim,
                         int(interleaved), int(table_rows), float(eps))


def make_paged_params(heads_q: int, heads_kv: int, *, page_size: int, num_pages: int, seqs: int,
                      tokens: int, pages_per_seq: int, page_stride: int = 0,
                      softmax_scale: float = 0.0, sink_pages: int = 0, local_pages: int = 1,
                      top_pages: int = 0, wait_limit_us: int = 0, debug_flags: int = 0,
                      head_dim: int = 128) -> SpaPagedParams:
    return SpaPagedParams(heads_q, heads_kv, head_dim, page_size, num_pages, pages_per_seq, seqs,
                          tokens, int(page_stride), float(softmax_scale), sink_pages, local_pages,
                          top_pages, int(wait_limit_us), int(debug_flags))


_pack_rows = struct.Struct("@Pqqq").pack
assert struct.calcsize("@Pqqq") == ctypes.sizeof(SpaRows)


def _rows(x, batch, tokens, heads, name):
    """A bf16 tensor [batch, tokens, heads, 128] or, for one batch element, [tokens, heads, 128]
    (any strides but the last dimension's), or an SpaRows, as a spa_rows to point at (its bytes:
    packing them takes a third of the time of making an SpaRows)."""
    if x is None:
        return None
    if x.__class__ is SpaRows:
        return ctypes.byref(x)
    st = x.stride()
    if len(st) == 3 and batch == 1:
        good, sb = x.shape == (tokens, heads, 128), 0
        s_t, s_h, s_d = st
    elif len(st) == 4:
        good = x.shape == (batch, tokens, heads, 128)
        sb, s_t, s_h, s_d = st
    else:
        good = False
    if not good:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, wanted {(batch, tokens, heads, 128)}")
    if x.dtype is not _BF16:
        raise TypeError(f"{name}: {x.dtype}, wanted torch.bfloat16")
    if s_d != 1 and x.numel():
        raise ValueError(f"{name}: the 128 elements of a row have to be contiguous")
    return _pack_rows(x.data_ptr(), sb, s_t, s_h)


def _flat(x, dtype, count, name):
    """Address of a contiguous tensor of at least ``count`` elements (raw addresses pass)."""
    if x is None or x.__class__ is int:
        return x
    if x.dtype is not dtype:
        raise TypeError(f"{name}: {x.dtype}, wanted {dtype}")
    if x.numel() < count:
        raise ValueError(f"{name}: {x.numel()} elements, wanted {count}")
    if not x.is_contiguous():
        raise ValueError(f"{name}: has to be contiguous")
    return x.data_ptr()


def _grid(x, dtype, shape, name):
    """Address of a contiguous tensor that the library reads as [shape]: of that shape, with more
    rows in front, or flat.  Rows of another length would be read with the wrong stride."""
    if x is None or x.__class__ is int:
        return x
    if x.shape == shape and x.dtype is dtype and x.is_contiguous():
        return x.data_ptr()
    given, count = tuple(x.shape), math.prod(shape)
    while len(given) > len(shape) and given[0] == 1:
        given = given[1:]
    if len(given) == len(shape):
        # a dimension's length is a stride unless there is only one row of it
        rows, good = 1, True
        for have, want in zip(given, shape):
            good = good and (have == want or (have > want and rows <= 1))
            rows *= want
    else:
        good = len(given) == 1 or x.numel() == count
    if not good:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, wanted {shape}")
    return _flat(x, dtype, count, name)


_I32, _BF16, _F32, _U32 = (getattr(_torch, t, None)
                           for t in ("int32", "bfloat16", "float32", "uint32"))
_WEIGHT = (128,)


def _angles(r, table):
    """Address of the rotation table; unused, and so unchecked, without a rotation."""
    if r is None or r.rotary_dim == 0:
        return _flat(table, _F32, 0, "table")
    return _grid(table, _F32, (r.table_rows, r.rotary_dim), "table")


def _word(x):
    """Address of the error word: one int32 or uint32."""
    if x is None or x.__class__ is int:
        return x
    return _flat(x, _U32 if x.dtype is _U32 else _I32, 1, "error")


def _device(*tensors):
    """The one CUDA device of the tensors given (None and raw addresses apart), or -1."""
    dev = None
    for x in tensors:
        if x is None or x.__class__ is int or x.__class__ is SpaRows:
            continue
        d = x.get_device()
        if d != dev:
            if d < 0:
                raise ValueError("a tensor in host memory: device memory is wanted")
            if dev is not None:
                raise ValueError(f"tensors on devices {dev} and {d}")
            dev = d
    return -1 if dev is None else dev


_current_device = getattr(getattr(_torch, "_C", None), "_cuda_getDevice", None) or (
    lambda: _torch.cuda.current_device())


def _call(fn, dev, stream, *args):
    """fn(*args, stream) with the tensors' device current, on the stream given or on that
    device's current one."""
    if dev < 0:
        return fn(*args, _stream(stream))
    if stream is None and _raw_stream is not None:
        stream = _raw_stream(dev)
    if dev == _current_device():
        return fn(*args, _stream(stream))
    with _torch.cuda.device(dev):
        return fn(*args, _stream(stream))


def _cache(p: SpaPagedParams, x, name):
    """Address of a K or V cache [num_pages, heads_kv, page_size, 128]."""
    if x is None or x.__class__ is int:
        return x
    page, heads = p.page_size, p.heads_kv
    if x.shape != (p.num_pages, heads, page, 128):
        raise ValueError(f"{name}: shape {tuple(x.shape)}, wanted "
                         f"{(p.num_pages, heads, page, 128)}")
    if x.dtype is not _BF16:
        raise TypeError(f"{name}: {x.dtype}, wanted torch.bfloat16")
    pitch = p.page_stride or heads * page * 128
    st = x.stride()
    if st != (pitch, page * 128, 128, 1) and (
            st[2:] != (128, 1) or (heads > 1 and st[1] != page * 128) or
            (p.num_pages > 1 and st[0] != pitch)):
        raise ValueError(f"{name}: strides {st} (pages {pitch} elements apart are wanted)")
    return x.data_ptr()


def sparse_qk_norm_rope(params: SpaRopeParams, q, k, q_weight, k_weight, positions, table, q_out,
                        k_out, error, stream=None) -> int:
    """Per-head RMS norm and position rotation of q and k; rows [batch, tokens, heads, 128]."""
    r = params
    b, t, hq, hk = r.batch, r.tokens, r.heads_q, r.heads_kv
    dev = _device(q, k, q_weight, k_weight, positions, table, q_out, k_out, error)
    return _call(
        _lib.sparse_qk_norm_rope, dev, stream, ctypes.byref(r), _rows(q, b, t, hq, "q"),
        _rows(k, b, t, hk, "k"), _grid(q_weight, _BF16, _WEIGHT, "q_weight"),
        _grid(k_weight, _BF16, _WEIGHT, "k_weight"), _grid(positions, _I32, (b, t), "positions"),
        _angles(r, table), _rows(q_out, b, t, hq, "q_out"),
        _rows(k_out, b, t, hk, "k_out"), _word(error))


def sparse_paged_append(params: SpaPagedParams, rope: Optional[SpaRopeParams], q, k, v, q_weight,
                        k_weight, table, cu_q, kv_lens, block_table, q_out, k_cache, v_cache,
                        summary, error, stream=None) -> int:
    """New tokens' k (normed, rotated) and v into the pages; q alike into q_out; summaries."""
    p = params
    t, hq, hk, seqs = p.tokens, p.heads_q, p.heads_kv, p.seqs
    dev = _device(q, k, v, q_weight, k_weight, table, cu_q, kv_lens, block_table, q_out, k_cache,
                  v_cache, summary, error)
    return _call(
        _lib.sparse_paged_append, dev, stream, ctypes.byref(p),
        None if rope is None else ctypes.byref(rope), _rows(q, 1, t, hq, "q"),
        _rows(k, 1, t, hk, "k"), _rows(v, 1, t, hk, "v"),
        _grid(q_weight, _BF16, _WEIGHT, "q_weight"), _grid(k_weight, _BF16, _WEIGHT, "k_weight"),
        _angles(rope, table), _flat(cu_q, _I32, seqs + 1, "cu_q"),
        _flat(kv_lens, _I32, seqs, "kv_lens"),
        _grid(block_table, _I32, (seqs, p.pages_per_seq), "block_table"),
        _rows(q_out, 1, t, hq, "q_out"),
        _cache(p, k_cache, "k_cache"), _cache(p, v_cache, "v_cache"),
        _grid(summary, _BF16, (p.num_pages, hk, 2, 128), "summary"), _word(error))


def sparse_paged_workspace_bytes(params: SpaPagedParams) -> int:
    """Workspace that serves the selection and the attention."""
    return int(_lib.sparse_paged_workspace_bytes(ctypes.byref(params)))


def sparse_paged_attn_workspace_bytes(params: SpaPagedParams) -> int:
    """Workspace of the attention alone, the same for every batch."""
    return int(_lib.sparse_paged_attn_workspace_bytes(ctypes.byref(params)))


def _list_width(p: SpaPagedParams) -> int:
    return p.sink_pages + p.local_pages + p.top_pages


def sparse_paged_select(params: SpaPagedParams, q, summary, cu_q, kv_lens, block_table, lists,
                        counts, workspace, error, workspace_bytes=None, stream=None) -> int:
    """Pages of every new token and kv head: sink, recent, and the best by upper bound."""
    p = params
    t, hk, seqs = p.tokens, p.heads_kv, p.seqs
    dev = _device(q, summary, cu_q, kv_lens, block_table, lists, counts, workspace, error)
    wb = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    return _call(
        _lib.sparse_paged_select, dev, stream, ctypes.byref(p), _rows(q, 1, t, p.heads_q, "q"),
        _grid(summary, _BF16, (p.num_pages, hk, 2, 128), "summary"),
        _flat(cu_q, _I32, seqs + 1, "cu_q"), _flat(kv_lens, _I32, seqs, "kv_lens"),
        _grid(block_table, _I32, (seqs, p.pages_per_seq), "block_table"),
        _grid(lists, _I32, (t, hk, _list_width(p)), "lists"),
        _grid(counts, _I32, (t, hk), "counts"), _ptr(workspace), wb, _word(error))


def sparse_paged_attn(params: SpaPagedParams, q, k_cache, v_cache, cu_q, kv_lens, block_table,
                      lists, counts, o, lse, workspace, error, workspace_bytes=None,
                      stream=None) -> int:
    """Causal attention of the new tokens over their pages (lists None), or the listed ones."""
    p = params
    t, hq, hk, seqs = p.tokens, p.heads_q, p.heads_kv, p.seqs
    dev = _device(q, k_cache, v_cache, cu_q, kv_lens, block_table, lists, counts, o, lse,
                  workspace, error)
    wb = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    return _call(
        _lib.sparse_paged_attn, dev, stream, ctypes.byref(p), _rows(q, 1, t, hq, "q"),
        _cache(p, k_cache, "k_cache"), _cache(p, v_cache, "v_cache"),
        _flat(cu_q, _I32, seqs + 1, "cu_q"), _flat(kv_lens, _I32, seqs, "kv_lens"),
        _grid(block_table, _I32, (seqs, p.pages_per_seq), "block_table"),
        _grid(lists, _I32, (t, hk, _list_width(p)), "lists"),
        _grid(counts, _I32, (t, hk), "counts"), _rows(o, 1, t, hq, "o"),
        _grid(lse, _F32, (t, hq), "lse"), _ptr(workspace), wb, _word(error))


def sparse_paged_status(error, stream=None) -> int:
    """Waits for the stream, reads and clears the error word."""
    return _call(_lib.sparse_paged_status, _device(error), stream, _word(error))


def sparse_prefill_status_string(status: int) -> str:
    return _lib.sparse_prefill_status_string(int(status)).decode()


def check(status: int, what: str = "spa") -> None:
    if status != SPA_OK:
        raise SpaError(status, what)


def kept_flops(stats: SpaStats, head_dim: int = 128) -> int:
    """Executed attention FLOPs on kept entries: 4 * d * sum_i |K_i|."""
    return 4 * head_dim * int(stats.kept_pairs)


def default_scale(head_dim: int = 128) -> float:
    return 1.0 / math.sqrt(head_dim)


# ---------------------------------------------------------------------------
# workspace views (the layout documented in include/spa.h)
# ---------------------------------------------------------------------------
def _align256(x: int) -> int:
    return (x + 255) // 256 * 256


def cap_prefix(n: int, local: int, sink: int, bq: int = 128) -> int:
    """P(n) = sum_{q < n} max(0, (q + 1) * bq - local - sink), in closed form."""
    return _cap_prefix_closed(n, local + sink, bq)


def _cap_prefix_closed(n: int, a: int, bq: int) -> int:
    q0 = a // bq
    if n <= q0:
        return 0
    return bq * ((n * (n + 1) - q0 * (q0 + 1)) // 2) - (n - q0) * a


class WorkspaceView:
    """Host-side indexing of the counts and lists inside a workspace tensor."""

    def __init__(self, params: SpaParams, workspace):
        import torch
        self.p = params
        self.nqb = (params.seq_len + 127) // 128
        self.nb = params.batch * params.heads_q * self.nqb
        self.unit = params.block_k if params.mode == SPA_MODE_SALE else 1
        self.per_head = _cap_prefix_closed(self.nqb, params.local + params.sink, 128) // self.unit
        ws8 = workspace.view(torch.uint8)
        self.counts = ws8[256:256 + 4 * self.nb].view(torch.int32)
        lo = _align256(256 + 4 * self.nb)
        n_list = params.batch * params.heads_q * self.per_head
        self.lists = ws8[lo:lo + 4 * n_list].view(torch.int32)

    def block_index(self, b: int, h: int, qb: int) -> int:
        return (b * self.p.heads_q + h) * self.nqb + qb

    def list_offset(self, b: int, h: int, qb: int) -> int:
        return ((b * self.p.heads_q + h) * self.per_head +
                _cap_prefix_closed(qb, self.p.local + self.p.sink, 128) // self.unit)
