"""ctypes marshalling of the attention half of a decoder block (C ABI:
include/ttt.h): rotary positions, the paged 4-bit key/value cache and
attention over it.

Only argument checking and marshalling live here, as in _binding.py. These
calls come once a token, so they keep to a few microseconds: descriptors are
built positionally and tensors are passed as plain addresses.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _binding as _b

ROPE_INTERLEAVED = 1 << 0
ATTN_ALL_KEYS = 1 << 0
ROPE_KINDS = {"linear": 1, "base": 2, "yarn": 3, "bands": 4}

_P, _I, _I64, _U = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32


class Rows(ctypes.Structure):
    _fields_ = [("data", _P), ("token_stride", _I64), ("head_stride", _I64), ("heads", _I),
                ("reserved", _I)]


class Rope(ctypes.Structure):
    _fields_ = [("table", _P), ("rot_dim", _I), ("max_pos", _I), ("flags", _U), ("reserved", _U)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", _I), ("reserved", _I), ("factor", ctypes.c_double),
                ("original", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("amplitude", ctypes.c_double)]


class Cache(ctypes.Structure):
    _fields_ = [("pages", _P), ("page_stride", _I64), ("page_table", _P), ("kv_lens", _P),
                ("q_starts", _P), ("batch", _I), ("max_pages", _I), ("n_pages", _I),
                ("page_size", _I), ("kv_heads", _I), ("head_dim", _I), ("reserved", _I)]


class Attn(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("window", _I), ("max_new", _I), ("max_kv", _I),
                ("flags", _U), ("reserved", _U)]


_lib = None


def _L():
    global _lib
    if _lib is not None:
        return _lib
    L = _b.lib()
    R, C, A, Z = (ctypes.POINTER(t) for t in (Rows, Cache, Attn, ctypes.c_size_t))
    T = ctypes.POINTER(Rope)
    L.ttt_rope_table.argtypes = [_P, _I, _I, ctypes.c_double, ctypes.POINTER(RopeScaling), _P]
    for fn in (L.ttt_rope_forward, L.ttt_rope_backward):
        fn.argtypes = [_I, _I, _I, _I, T, _P, R, R, R, R, _P]
    L.ttt_kv_page_bytes.argtypes = [_I, _I, _I, Z]
    L.ttt_kv_append.argtypes = [C, _I, _I, R, R, R, R, T, _P, _P]
    L.ttt_kv_read.argtypes = [C, _I, _I, R, R, _P]
    L.ttt_kv_attention_workspace_size.argtypes = [A, _I, _I, _I, _I, _I, _I, Z]
    L.ttt_kv_attention.argtypes = [C, A, _I, _I, R, R, _P, _P, ctypes.c_size_t, _P]
    for fn in ("rope_table", "rope_forward", "rope_backward", "kv_page_bytes", "kv_append",
               "kv_read", "kv_attention_workspace_size", "kv_attention"):
        getattr(L, "ttt_" + fn).restype = ctypes.c_int
    _lib = L
    return L


def _stream(stream):
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _rows(t, what, dtype=None, dim=None):
    """The view [rows, heads, dim] (or [B, T, heads, dim] whose sequences
    follow each other evenly) as the library takes it."""
    if not t.is_cuda:
        raise ValueError("all tensors must be on the GPU")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    shape, st = t.shape, t.stride()
    if len(shape) == 4:
        if shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
            raise ValueError(f"{what}: the sequences of a [B, T, heads, dim] tensor must follow "
                             "each other at T times the token stride")
        ts = st[1] if shape[1] > 1 else st[0]
        shape, st = (shape[0] * shape[1],) + tuple(shape[2:]), (ts,) + tuple(st[2:])
    if len(shape) != 3:
        raise ValueError(f"{what} must be [rows, heads, dim] or [B, T, heads, dim]")
    if shape[2] > 1 and st[2] != 1:
        raise ValueError(f"{what}: the values of a head must be contiguous")
    if dim is not None and shape[2] != dim:
        raise ValueError(f"{what}: head dim {shape[2]}, expected {dim}")
    # the stride of an axis of length 1 means nothing: any aligned one will do
    return Rows(t.data_ptr(), st[0] if shape[0] > 1 else shape[1] * shape[2],
                st[1] if shape[1] > 1 else shape[2], shape[1], 0), shape[0], shape[2]


def _ints(t, what, shape=None):
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor on the GPU")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{what} must have shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _rope(table, interleaved):
    if (table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32
            or not table.is_cuda or not table.is_contiguous()):
        raise ValueError("the rope table must be a contiguous float32 [max_pos, rot_dim / 2, 2] "
                         "tensor on the GPU")
    return Rope(table.data_ptr(), 2 * table.shape[1], table.shape[0],
                ROPE_INTERLEAVED if interleaved else 0, 0)


def rope_table(max_pos, rot_dim, base=10000.0, *, scaling=None, factor=1.0, original=None,
               low=1.0, high=None, amplitude=None, device="cuda", stream=None):
    """float32 [max_pos, rot_dim / 2, 2]: cos and sin of every position's
    angles (ttt_rope_table). scaling: None, "linear", "base", "yarn" or
    "bands", with its factor and, for the last two, the trained context
    `original` and the turns low and high (high: 32 for "yarn", 4 for
    "bands"). amplitude: None is 1, for "yarn" 0.1 log(factor) + 1."""
    if scaling is not None and scaling not in ROPE_KINDS:
        raise ValueError(f"scaling must be None or one of {sorted(ROPE_KINDS)}, got {scaling!r}")
    if scaling in ("yarn", "bands") and original is None:
        raise ValueError(f"{scaling!r} needs the trained context `original`")
    if amplitude is None:
        amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 0 else 1.0
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    table = torch.empty((max(int(max_pos), 0), max(int(rot_dim), 0) // 2, 2), dtype=torch.float32,
                        device=device)
    sc = RopeScaling(ROPE_KINDS.get(scaling, 0), 0, float(factor), float(original or 1.0),
                     float(low), float(high), float(amplitude))
    _b._check(_L().ttt_rope_table(table.data_ptr(), int(max_pos), int(rot_dim), float(base),
                                  ctypes.byref(sc), _stream(stream)))
    return table


def _rope_call(fn, q, k, table, positions, interleaved, q_out, k_out, stream):
    rq, n, dim = _rows(q, "q")
    act = _b._dtype_code(q, "q")
    seq = q.shape[1] if q.dim() == 4 else n
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    ro, no, _ = _rows(q_out, "q_out", q.dtype, dim)
    rk = rko = None
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        rk, nk, _ = _rows(k, "k", q.dtype, dim)
        rko, nko, _ = _rows(k_out, "k_out", q.dtype, dim)
        if nk != n or nko != n:
            raise ValueError("q, k and their outputs must have the same rows")
    if no != n:
        raise ValueError("q and q_out must have the same rows")
    rope = _rope(table, interleaved)
    pos = None
    if positions is not None:
        if positions.numel() != n:
            raise ValueError("positions must have one entry a row")
        pos = _ints(positions, "positions")
    ref = ctypes.byref
    st = fn(n, max(seq, 1), dim, act, ref(rope), pos, ref(rq), ref(rk) if rk is not None else None, ref(ro),
            ref(rko) if rko is not None else None, _stream(stream))
    if st:
        _b._check(st)
    return q_out, k_out


def rope_forward(q, k, table, *, positions=None, interleaved=False, q_out=None, k_out=None,
                 stream=None):
    """q and k (or None) with their first rot_dim values a head rotated
    (ttt_rope_forward): [rows, heads, dim] or [B, T, heads, dim] views of one
    dtype, table from rope_table. positions: int32, one a row; None counts
    from 0 in every sequence. q_out, k_out may be q and k themselves."""
    return _rope_call(_L().ttt_rope_forward, q, k, table, positions, interleaved, q_out, k_out,
                      stream)


def rope_backward(dq_out, dk_out, table, *, positions=None, interleaved=False, dq=None, dk=None,
                  stream=None):
    """The gradients of rope_forward's inputs from those of its outputs
    (ttt_rope_backward)."""
    return _rope_call(_L().ttt_rope_backward, dq_out, dk_out, table, positions, interleaved, dq,
                      dk, stream)


def kv_page_bytes(page_size, kv_heads, head_dim) -> int:
    n = ctypes.c_size_t(0)
    _b._check(_L().ttt_kv_page_bytes(page_size, kv_heads, head_dim, ctypes.byref(n)))
    return n.value


def kv_pages(n_pages, page_size, kv_heads, head_dim, device="cuda"):
    """An empty pool for the cache: uint8 [n_pages, kv_heads, bytes of a
    head's block]."""
    n = kv_page_bytes(page_size, kv_heads, head_dim)
    return torch.zeros((n_pages, kv_heads, n // kv_heads), dtype=torch.uint8, device=device)


def _cache(pages, page_table, kv_lens, q_starts, dim):
    if pages.dim() != 3 or pages.dtype != torch.uint8 or not pages.is_cuda:
        raise ValueError("pages must be a uint8 [n_pages, kv_heads, bytes] tensor on the GPU")
    n_pages, heads, block = pages.shape
    st = pages.stride()
    if st[2] != 1 or (heads > 1 and st[1] != block):
        raise ValueError("a page's heads must be contiguous")
    page, rest = divmod(block * 16, dim * 17)
    if rest or page < 1:
        raise ValueError(f"{block} bytes a head are no whole number of tokens of dim {dim}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    batch = page_table.shape[0]
    return Cache(pages.data_ptr(), st[0] if n_pages > 1 else heads * block,
                 _ints(page_table, "page_table"), _ints(kv_lens, "kv_lens", (batch,)),
                 _ints(q_starts, "q_starts", (batch + 1,)), batch, page_table.shape[1], n_pages,
                 page, heads, dim, 0)


def kv_append(pages, page_table, kv_lens, k, v, *, q=None, q_starts=None, rope_table=None,
              interleaved=False, positions=None, q_out=None, stream=None):
    """Appends k and v [rows, kv_heads, dim] to the cache (ttt_kv_append):
    pages from kv_pages, page_table int32 [batch, max_pages], kv_lens int32
    [batch] with the new tokens counted, q_starts int32 [batch + 1] (None:
    the same number of rows each). With rope_table, k is rotated first, and
    q, if given, beside it. Returns the rotated q (or None)."""
    rk, n, dim = _rows(k, "k")
    act = _b._dtype_code(k, "k")
    rv, nv, _ = _rows(v, "v", k.dtype, dim)
    if nv != n:
        raise ValueError("k and v must have the same rows")
    cache = _cache(pages, page_table, kv_lens, q_starts, dim)
    ref = ctypes.byref
    rq = ro = None
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        rq, nq, _ = _rows(q, "q", k.dtype, dim)
        ro, no, _ = _rows(q_out, "q_out", k.dtype, dim)
        if nq != n or no != n:
            raise ValueError("q, q_out and k must have the same rows")
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope = None if rope_table is None else _rope(rope_table, interleaved)
    pos = None
    if positions is not None:
        if positions.numel() != n:
            raise ValueError("positions must have one entry a row")
        pos = _ints(positions, "positions")
    st = _L().ttt_kv_append(ref(cache), n, act, ref(rk), ref(rv), None if rq is None else ref(rq),
                            None if ro is None else ref(ro), None if rope is None else ref(rope),
                            pos, _stream(stream))
    if st:
        _b._check(st)
    return q_out


def kv_read(pages, page_table, kv_lens, rows, head_dim, dtype=torch.bfloat16, *, q_starts=None,
            k_out=None, v_out=None, stream=None):
    """What the cache holds of each sequence's last tokens, `rows` in all, in
    the order kv_append takes them (ttt_kv_read): k, v [rows, kv_heads,
    head_dim]."""
    cache = _cache(pages, page_table, kv_lens, q_starts, head_dim)
    shape = (rows, pages.shape[1], head_dim)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=pages.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=pages.device)
    rk, nk, _ = _rows(k_out, "k_out", dtype, head_dim)
    rv, nv, _ = _rows(v_out, "v_out", dtype, head_dim)
    if nk != rows or nv != rows:
        raise ValueError("k_out and v_out must have `rows` rows")
    st = _L().ttt_kv_read(ctypes.byref(cache), rows, _b._dtype_code(k_out, "k_out"),
                          ctypes.byref(rk), ctypes.byref(rv), _stream(stream))
    if st:
        _b._check(st)
    return k_out, v_out


def _attn(scale, window, max_new, max_kv, causal, dim):
    return Attn(dim ** -0.5 if scale is None else scale, window, max_new, max_kv,
                0 if causal else ATTN_ALL_KEYS, 0)


def kv_attention_workspace_size(batch, rows, kv_heads, q_heads, head_dim, dtype=torch.bfloat16, *,
                                max_new, max_kv, window=0) -> int:
    n = ctypes.c_size_t(0)
    a = _attn(None, window, max_new, max_kv, True, head_dim)
    act = _b.TTT_F32 if dtype == torch.float32 else _b.TTT_BF16
    _b._check(_L().ttt_kv_attention_workspace_size(ctypes.byref(a), batch, rows, act, kv_heads,
                                                   q_heads, head_dim, ctypes.byref(n)))
    return n.value


def kv_attention(q, pages, page_table, kv_lens, *, q_starts=None, max_new=None, max_kv=None,
                 scale=None, window=0, causal=True, with_lse=False, out=None, lse=None,
                 workspace=None, stream=None):
    """Attention of q [rows, q_heads, dim] over the cache (ttt_kv_attention):
    each sequence's rows stand at the end of its kv_lens tokens. window: 0, or
    how many keys (its own included) a row sees. causal=False: every key of
    the sequence. scale: None is dim ** -0.5. max_new, max_kv: upper bounds of
    the sequences' rows and lengths, where the caller knows better ones than
    `rows` and what the page table can hold. Returns o, or (o, lse) with
    with_lse (lse float32 [rows, q_heads])."""
    rq, n, dim = _rows(q, "q")
    act = _b._dtype_code(q, "q")
    cache = _cache(pages, page_table, kv_lens, q_starts, dim)
    if max_new is None:
        max_new = max(1, n if q_starts is not None else n // cache.batch)
    if max_kv is None:
        max_kv = cache.max_pages * cache.page_size
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    ro, no, _ = _rows(out, "out", q.dtype, dim)
    if no != n:
        raise ValueError("q and out must have the same rows")
    if lse is None:
        if with_lse:
            lse = torch.empty((n, rq.heads), dtype=torch.float32, device=q.device)
    elif lse.dtype != torch.float32 or not lse.is_contiguous() or lse.numel() != n * rq.heads:
        raise ValueError("lse must be a contiguous float32 [rows, q_heads] tensor")
    a = _attn(scale, window, max_new, max_kv, causal, dim)
    L, ref = _L(), ctypes.byref
    if workspace is None:
        need = ctypes.c_size_t(0)
        st = L.ttt_kv_attention_workspace_size(ref(a), cache.batch, n, act, cache.kv_heads,
                                               rq.heads, dim, ref(need))
        if st:
            _b._check(st)
        if need.value:
            workspace = torch.empty(need.value, dtype=torch.uint8, device=q.device)
    st = L.ttt_kv_attention(ref(cache), ref(a), n, act, ref(rq), ref(ro),
                            None if lse is None else lse.data_ptr(),
                            None if workspace is None else workspace.data_ptr(),
                            0 if workspace is None else workspace.numel(), _stream(stream))
    if st:
        _b._check(st)
    return (out, lse) if with_lse or lse is not None else out
