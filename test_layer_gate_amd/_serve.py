"""ctypes marshalling of the attention half of a decoder block (C ABI:
include/ttt.h): rotary positions, the paged 4-bit key/value cache and
attention over it.

Only argument checking and marshalling live here, as in _binding.py. These
calls come once a token, so they keep to a few microseconds: descriptors are
packed as bytes in the layout of the header's structs (a third of the time that
filling a ctypes structure takes) and tensors are passed as plain addresses.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct

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


class AttnPlan(ctypes.Structure):
    _fields_ = [("many", _I), ("tile", _I), ("parts", _I), ("slices", _I), ("waves", _I),
                ("reserved", _I), ("workgroups", _I64)]


# The same layouts, packed; bytes are passed where the library takes a pointer.
_pack_rows = struct.Struct("PqqiI").pack
_pack_rope = struct.Struct("PiiII").pack
_pack_cache = struct.Struct("PqPPPiiiiiii4x").pack
_pack_attn = struct.Struct("fiiiII").pack

_lib = None
_ref = ctypes.byref


def _L():
    global _lib
    if _lib is not None:
        return _lib
    L = _b.lib()
    R = C = A = T = _P  # packed bytes, or a structure's address
    Z = ctypes.POINTER(ctypes.c_size_t)
    L.ttt_rope_table.argtypes = [_P, _I, _I, ctypes.c_double, ctypes.POINTER(RopeScaling), _P]
    for fn in (L.ttt_rope_forward, L.ttt_rope_backward):
        fn.argtypes = [_I, _I, _I, _I, T, _P, R, R, R, R, _P]
    L.ttt_kv_page_bytes.argtypes = [_I, _I, _I, Z]
    L.ttt_kv_append.argtypes = [C, _I, _I, R, R, R, R, T, _P, _P]
    L.ttt_kv_read.argtypes = [C, _I, _I, R, R, _P]
    L.ttt_kv_attention_workspace_size.argtypes = [A, _I, _I, _I, _I, _I, _I, Z]
    L.ttt_kv_attention_plan.argtypes = [A, _I, _I, _I, _I, _I, _I, ctypes.POINTER(AttnPlan)]
    L.ttt_kv_attention.argtypes = [C, A, _I, _I, R, R, _P, _P, ctypes.c_size_t, _P]
    for fn in ("rope_table", "rope_forward", "rope_backward", "kv_page_bytes", "kv_append",
               "kv_read", "kv_attention_workspace_size", "kv_attention_plan",
               "kv_attention"):
        getattr(L, "ttt_" + fn).restype = ctypes.c_int
    _lib = L
    return L


# The current stream's handle without building a torch.cuda.Stream (2.9 us of
# a call's 10) where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, t):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _on(stream, make, *args, **kw):
    """A tensor from the memory of the stream that the call runs on: torch may
    give it away, when it is dropped, only behind the kernels there."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _empty(t, stream):
    if stream is None:  # (torch.empty with a dtype and device takes twice as long)
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return _on(stream, torch.empty_like, t, memory_format=torch.contiguous_format)


def _rows_of(t, what):
    """(rows, heads, dim), (token stride, head stride) of the view [rows,
    heads, dim], or [B, T, heads, dim] whose sequences follow each other
    evenly."""
    if not t.is_cuda:
        raise ValueError("all tensors must be on the GPU")
    st = t.stride()
    if len(st) == 3:
        n, h, d = t.shape
        ts, hs, vs = st
    elif len(st) == 4:
        b, n, h, d = t.shape
        bs, ts, hs, vs = st
        if b > 1 and n > 1 and bs != n * ts:
            raise ValueError(f"{what}: the sequences of a [B, T, heads, dim] tensor must follow "
                             "each other at T times the token stride")
        ts = ts if n > 1 else bs
        n *= b
    else:
        raise ValueError(f"{what} must be [rows, heads, dim] or [B, T, heads, dim]")
    if vs != 1 and d > 1:
        raise ValueError(f"{what}: the values of a head must be contiguous")
    if n >> 31:  # ctypes would cut it to 32 bits
        raise ValueError(f"{what} has {n} rows; the library counts them in 32 bits")
    # the stride of an axis of length 1 means nothing: any aligned one will do
    return n, h, d, _pack_rows(t.data_ptr(), ts if n > 1 else h * d, hs if h > 1 else d, h, 0)


def _dense(t, h, d):
    """The same of a contiguous tensor made here."""
    return _pack_rows(t.data_ptr(), h * d, d, h, 0)


def _rows(t, what, n, dim, dtype):
    """The view as the library takes it, of `n` rows of heads of `dim`."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    m, _, d, r = _rows_of(t, what)
    if m != n or d != dim:
        raise ValueError(f"{what} must have {n} rows and heads of {dim}, got {m} and {d}")
    return r


def _ints(t, what, shape=None):
    if t is None:
        return None
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor on the GPU")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _positions(t, n):
    if t is None:
        return None
    if t.numel() != n:
        raise ValueError("positions must have one entry a row")
    return _ints(t, "positions")


def _act(t, what):
    d = t.dtype
    return 0 if d is torch.bfloat16 else 1 if d is torch.float32 else _b._dtype_code(t, what)


def _act_of(dtype):
    if dtype is torch.bfloat16 or dtype is torch.float32:
        return _b.TTT_F32 if dtype is torch.float32 else _b.TTT_BF16
    raise TypeError(f"rows must be bfloat16 or float32, got {dtype}")


def _rope(table, interleaved):
    shape = table.shape
    if (len(shape) != 3 or shape[2] != 2 or table.dtype is not torch.float32
            or not table.is_cuda or not table.is_contiguous()):
        raise ValueError("the rope table must be a contiguous float32 [max_pos, rot_dim / 2, 2] "
                         "tensor on the GPU")
    return _pack_rope(table.data_ptr(), 2 * shape[1], shape[0], ROPE_INTERLEAVED if interleaved else 0, 0)


def rope_table(max_pos, rot_dim, base=10000.0, *, scaling=None, factor=1.0, original=None,
               low=1.0, high=None, amplitude=None, device="cuda", stream=None):
    """float32 [max_pos, rot_dim / 2, 2]: cos and sin of every position's
    angles (ttt_rope_table). scaling: None, "linear", "base", "yarn" or
    "bands", with its factor and, for the last two, the trained context
    `original` and the turns low and high (high: 32 for "yarn", 4 for
    "bands"). amplitude: None is 1, for "yarn" 0.1 log(factor) + 1."""
    max_pos, rot_dim = int(max_pos), int(rot_dim)
    if scaling is not None and scaling not in ROPE_KINDS:
        raise ValueError(f"scaling must be None or one of {sorted(ROPE_KINDS)}, got {scaling!r}")
    if max(abs(max_pos), abs(rot_dim)) >> 31:  # ctypes would cut them to 32 bits
        raise ValueError("max_pos and rot_dim must lie below 2^31")
    if scaling in ("yarn", "bands") and original is None:
        raise ValueError(f"{scaling!r} needs the trained context `original`")
    if amplitude is None:
        amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 0 else 1.0
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    table = _on(stream, torch.empty, (max(max_pos, 0), max(rot_dim, 0) // 2, 2),
                dtype=torch.float32, device=device)
    if not table.is_cuda:
        raise ValueError("the rope table is made on the GPU")
    sc = RopeScaling(ROPE_KINDS.get(scaling, 0), 0, float(factor), float(original or 1.0),
                     float(low), float(high), float(amplitude))
    _b._check(_L().ttt_rope_table(table.data_ptr(), max_pos, rot_dim, float(base),
                                  ctypes.byref(sc), _stream(stream, table)))
    return table


def _rope_call(fn, q, k, table, positions, interleaved, q_out, k_out, stream):
    n, h, dim, rq = _rows_of(q, "q")
    act, dtype = _act(q, "q"), q.dtype
    if q_out is None:
        q_out = _empty(q, stream)
        ro = _dense(q_out, h, dim)
    else:
        ro = _rows(q_out, "q_out", n, dim, dtype)
    rk = rko = None
    if k is not None:
        rk = _rows(k, "k", n, dim, dtype)
        if k_out is None:
            k_out = _empty(k, stream)
            rko = _dense(k_out, k.shape[-2], dim)
        else:
            rko = _rows(k_out, "k_out", n, dim, dtype)
    st = fn(n, max(q.shape[1], 1) if q.dim() == 4 else max(n, 1), dim, act,
            _rope(table, interleaved), _positions(positions, n), rq, rk, ro, rko,
            _stream(stream, q))
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
    shape, st = pages.shape, pages.stride()
    if len(shape) != 3 or pages.dtype is not torch.uint8 or not pages.is_cuda:
        raise ValueError("pages must be a uint8 [n_pages, kv_heads, bytes] tensor on the GPU")
    n_pages, heads, block = shape
    if st[2] != 1 or (heads > 1 and st[1] != block):
        raise ValueError("a page's heads must be contiguous")
    page, rest = divmod(block * 16, dim * 17)
    if rest or page < 1:
        raise ValueError(f"{block} bytes a head are no whole number of tokens of dim {dim}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    batch, max_pages = page_table.shape
    return _pack_cache(pages.data_ptr(), st[0] if n_pages > 1 else heads * block,
                       _ints(page_table, "page_table"), _ints(kv_lens, "kv_lens", (batch,)) or 0,
                       _ints(q_starts, "q_starts", (batch + 1,)) or 0, batch, max_pages, n_pages, page,
                       heads, dim, 0)


def kv_append(pages, page_table, kv_lens, k, v, *, q=None, q_starts=None, rope_table=None,
              interleaved=False, positions=None, q_out=None, stream=None):
    """Appends k and v [rows, kv_heads, dim] to the cache (ttt_kv_append):
    pages from kv_pages, page_table int32 [batch, max_pages], kv_lens int32
    [batch] with the new tokens counted, q_starts int32 [batch + 1] (None:
    the same number of rows each). With rope_table, k is rotated first, and
    q, if given, beside it. Returns the rotated q (or None)."""
    n, _, dim, rk = _rows_of(k, "k")
    act, dtype = _act(k, "k"), k.dtype
    rv = _rows(v, "v", n, dim, dtype)
    cache = _cache(pages, page_table, kv_lens, q_starts, dim)
    rq = ro = None
    if q is not None:
        rq = _rows(q, "q", n, dim, dtype)
        if q_out is None:
            q_out = _empty(q, stream)
            ro = _dense(q_out, q.shape[-2], dim)
        else:
            ro = _rows(q_out, "q_out", n, dim, dtype)
    elif q_out is not None:
        raise ValueError("q_out without q")
    st = _L().ttt_kv_append(cache, n, act, rk, rv, rq, ro,
                            None if rope_table is None else _rope(rope_table, interleaved),
                            _positions(positions, n), _stream(stream, k))
    if st:
        _b._check(st)
    return q_out


def kv_read(pages, page_table, kv_lens, rows, head_dim, dtype=torch.bfloat16, *, q_starts=None,
            k_out=None, v_out=None, stream=None):
    """What the cache holds of each sequence's last tokens, `rows` in all, in
    the order kv_append takes them (ttt_kv_read): k, v [rows, kv_heads,
    head_dim]."""
    cache = _cache(pages, page_table, kv_lens, q_starts, head_dim)
    heads = pages.shape[1]
    shape = (rows, heads, head_dim)
    if k_out is None:
        k_out = _on(stream, torch.empty, shape, dtype=dtype, device=pages.device)
        rk = _dense(k_out, heads, head_dim)
    else:
        rk = _rows(k_out, "k_out", rows, head_dim, dtype)
    if v_out is None:
        v_out = _empty(k_out, stream)
        rv = _dense(v_out, heads, head_dim)
    else:
        rv = _rows(v_out, "v_out", rows, head_dim, dtype)
    st = _L().ttt_kv_read(cache, rows, _act(k_out, "k_out"), rk, rv,
                          _stream(stream, pages))
    if st:
        _b._check(st)
    return k_out, v_out


@functools.lru_cache(maxsize=1024)  # of sizes alone
def _workspace(batch, rows, act, kv_heads, q_heads, dim, max_new, max_kv, window):
    n = ctypes.c_size_t(0)
    a = _pack_attn(1.0, window, max_new, max_kv, 0, 0)
    _b._check(_L().ttt_kv_attention_workspace_size(a, batch, rows, act, kv_heads, q_heads, dim,
                                                   _ref(n)))
    return n.value


def kv_attention_workspace_size(batch, rows, kv_heads, q_heads, head_dim, dtype=torch.bfloat16, *,
                                max_new, max_kv, window=0) -> int:
    return _workspace(batch, rows, _act_of(dtype), kv_heads, q_heads, head_dim, max_new, max_kv, window)


def kv_attention_plan(batch, rows, kv_heads, q_heads, head_dim, dtype=torch.bfloat16, *,
                      max_new, max_kv, window=0) -> dict:
    """How kv_attention takes such a call (ttt_kv_attention_plan): its kernel
    (many: True or False), rows of a tile, parts of a sequence's keys or slices
    of all, workgroups and their waves."""
    p = AttnPlan()
    _b._check(_L().ttt_kv_attention_plan(
        _pack_attn(1.0, window, max_new, max_kv, 0, 0), batch, rows, _act_of(dtype),
        kv_heads, q_heads, head_dim, _ref(p)))
    return dict(many=bool(p.many), tile=p.tile, parts=p.parts, slices=p.slices, waves=p.waves,
                workgroups=p.workgroups)


def kv_attention(q, pages, page_table, kv_lens, *, q_starts=None, max_new=None, max_kv=None,
                 scale=None, window=0, causal=True, with_lse=False, out=None, lse=None,
                 workspace=None, stream=None):
    """Attention of q [rows, q_heads, dim] over the cache (ttt_kv_attention):
    each sequence's rows stand at the end of its kv_lens tokens. window: 0, or
    how many keys (its own included) a row sees. causal=False: every key of
    the sequence. scale: None is dim ** -0.5. max_new, max_kv: upper bounds of
    the sequences' rows and lengths, where the caller knows better ones than
    `rows` and what the page table can hold; up to 16 rows a key head, which
    max_new tells, keep 16 bits of bf16 rows' weights, more rows 8. Returns o, or (o, lse) with
    with_lse (lse float32 [rows, q_heads])."""
    n, heads, dim, rq = _rows_of(q, "q")
    act = _act(q, "q")
    cache = _cache(pages, page_table, kv_lens, q_starts, dim)
    batch, kv_heads = page_table.shape[0], pages.shape[1]
    if max_new is None:
        max_new = max(1, n if q_starts is not None else n // max(batch, 1))
    if max_kv is None:
        max_kv = min(max(1, page_table.shape[1] * (pages.shape[2] * 16 // (dim * 17))), 1 << 30)
    if out is None:
        out = _empty(q, stream)
        ro = _dense(out, heads, dim)
    else:
        ro = _rows(out, "out", n, dim, q.dtype)
    if lse is None:
        if with_lse:
            lse = _on(stream, torch.empty, (n, heads), dtype=torch.float32, device=q.device)
    elif (lse.dtype is not torch.float32 or not lse.is_cuda or not lse.is_contiguous()
          or lse.numel() != n * heads):
        raise ValueError("lse must be a contiguous float32 [rows, q_heads] tensor on the GPU")
    a = _pack_attn(dim ** -0.5 if scale is None else scale, window, max_new, max_kv,
                   0 if causal else ATTN_ALL_KEYS, 0)
    if workspace is None:
        need = _workspace(batch, n, act, kv_heads, heads, dim, max_new, max_kv, window)
        if need:
            workspace = _on(stream, torch.empty, need, dtype=torch.uint8, device=q.device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the GPU")
    st = _L().ttt_kv_attention(cache, a, n, act, rq, ro,
                               None if lse is None else lse.data_ptr(),
                               None if workspace is None else workspace.data_ptr(),
                               0 if workspace is None else workspace.nbytes, _stream(stream, q))
    if st:
        _b._check(st)
    return (out, lse) if with_lse or lse is not None else out
