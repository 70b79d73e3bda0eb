"""ctypes marshalling of the operators around and beside a decoder block (C
ABI: include/ttt.h): the norms of its residual stream, linear attention, and
the AdamW step.

Only argument checking and marshalling live here, as in _serve.py, whose
helpers it shares.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import struct

import torch

from . import _binding as _b
from . import _serve as _s

NORM_POST, NORM_PRE = 1 << 0, 1 << 1

_P, _I, _I64, _U, _F = _s._P, _s._I, _s._I64, _s._U, ctypes.c_float
_D, _S = ctypes.c_double, ctypes.c_size_t


class Norm(ctypes.Structure):
    _fields_ = [("rows", _I), ("d", _I), ("gates", _I), ("act_dtype", _I), ("res_dtype", _I), ("weight_dtype", _I),
                ("scale", _F), ("eps", _F), ("flags", _U), ("reserved", _U)]


class Linear(ctypes.Structure):
    _fields_ = [("log_decay", _P), ("q_starts", _P), ("batch", _I), ("tokens", _I), ("max_new", _I), ("act_dtype", _I),
                ("kv_heads", _I), ("q_heads", _I), ("dim_k", _I), ("dim_v", _I), ("scale", _F), ("reserved", _U)]


class Param(ctypes.Structure):
    _fields_ = [("p", _P), ("master", _P), ("g", _P), ("n", _I64)]


class AdamW(ctypes.Structure):
    _fields_ = [("param_dtype", _I), ("grad_dtype", _I), ("bits", _I), ("step", _I), ("lr", _D), ("beta1", _D),
                ("beta2", _D), ("eps", _D), ("weight_decay", _D), ("max_norm", _D), ("norm", _P), ("lr_device", _P),
                ("step_device", _P)]


# The same layouts, packed; bytes are passed where the library takes a pointer.
_pack_norm = struct.Struct("iiiiiiffII").pack
_pack_linear = struct.Struct("PPiiiiiiiifI").pack
_pack_adamw = struct.Struct("iiii6dPPP").pack

_lib = None
_ref = ctypes.byref


def _L():
    global _lib
    if _lib is not None:
        return _lib
    L = _b.lib()
    R = N = A = _P  # packed bytes, or a structure's address
    Z = ctypes.POINTER(_S)
    L.ttt_block_norm.argtypes = [N, R, R, _P, _P, R, R, R, _P]
    L.ttt_block_norm_backward_workspace_size.argtypes = [N, Z]
    L.ttt_block_norm_backward.argtypes = [N, R, R, R, R, _P, _P, R, R, R, R, _P, _P, _P, _S, _P]
    L.ttt_linear_attention_workspace_size.argtypes = [N, Z]
    L.ttt_linear_attention_backward_workspace_size.argtypes = [N, Z]
    L.ttt_linear_attention.argtypes = [N, R, R, R, R, _P, _P, _S, _P]
    L.ttt_linear_attention_backward.argtypes = [N, R, R, R, R, _P, _P, R, R, R, _P, _P, _S, _P]
    L.ttt_adamw_state_size.argtypes = [_P, _I, _I, Z]
    L.ttt_adamw_step.argtypes = [A, _P, _I, _P, _S, _P]
    L.ttt_adamw_read.argtypes = [_P, _I64, _I, _P, _P, _P]
    L.ttt_grad_norm_workspace_size.argtypes = [_I, Z]
    L.ttt_grad_norm.argtypes = [_P, _P, _I, _I, _P, _P, _S, _P]
    for fn in ("block_norm", "block_norm_backward_workspace_size", "block_norm_backward",
               "linear_attention_workspace_size", "linear_attention_backward_workspace_size", "linear_attention",
               "linear_attention_backward", "adamw_state_size", "adamw_step", "adamw_read",
               "grad_norm_workspace_size", "grad_norm"):
        getattr(L, "ttt_" + fn).restype = ctypes.c_int
    _lib = L
    return L


def _alone(t, *others):
    """Every tensor is on t's GPU, and that is the current one: kernels are
    launched there."""
    if not t.is_cuda:
        raise ValueError("all tensors must be on the GPU")
    d = t.get_device()
    for o in others:
        if o is not None and o.get_device() != d:
            raise ValueError("all tensors must be on one GPU")
    if d != torch.cuda.current_device():
        raise ValueError("the tensors must be on the current GPU (torch.cuda.device selects it)")


def _new(shape, dtype, like, stream):
    if dtype is like.dtype:
        if shape == like.shape:
            return _s._empty(like, stream)
        return _s._on(stream, like.new_empty, shape)
    return _s._on(stream, like.new_empty, shape, dtype=dtype)


def _workspace(need, like, workspace, stream):
    """(tensor, address, bytes) of the caller's workspace, or of a new one."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _new((need,), torch.uint8, like, stream)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the GPU")
    return workspace, workspace.data_ptr(), workspace.nbytes


# ------------------------------------------------------------------ norms


def _row_view(t, what):
    """(rows, d, row stride) of [..., d], its rows evenly apart."""
    shape, st = t.shape, t.stride()
    if not shape:
        raise ValueError(f"{what} must be [..., d]")
    d = shape[-1]
    if t.is_contiguous():
        return (t.numel() // d if d else 0), d, d
    if d > 1 and st[-1] != 1:
        raise ValueError(f"{what}: the values of a row must be contiguous")
    rows, row = 1, 0
    for n, s in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if n == 1:
            continue
        if rows == 1:
            row = s
        elif s != rows * row:
            raise ValueError(f"{what}: the rows must be evenly apart")
        rows *= n
    return rows, d, row if rows > 1 else d


def _pack_view(t, what, rows, d, dtype):
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.is_contiguous() and t.shape[-1:] == (d,) and t.numel() == rows * d:
        return _s._pack_rows(t.data_ptr(), d, d, 1, 0)
    n, m, stride = _row_view(t, what)
    if n != rows or m != d:
        raise ValueError(f"{what} must have {rows} rows of {d}, got {n} of {m}")
    return _s._pack_rows(t.data_ptr(), stride, d, 1, 0)


def _out(t, what, like, rows, d, dtype, stream):
    """(tensor, packed view) of an output that the caller gives, or a new one."""
    if t is None:
        t = _new(like.shape, dtype, like, stream)
        return t, _s._pack_rows(t.data_ptr(), d, d, 1, 0)
    return t, _pack_view(t, what, rows, d, dtype)


def _weight(w, what, d, kind):
    """(flag, address, dtype) of a norm: None, True (no weight) or its weight [d]."""
    if w is None or w is False:
        return False, None, kind
    if w is True:
        return True, None, kind
    if w.shape != (d,) or not w.is_cuda or not w.is_contiguous():
        raise ValueError(f"{what} must be a contiguous [{d}] tensor on the GPU")
    if kind is not None and w.dtype is not kind:
        raise TypeError("post and pre must have one dtype")
    return True, w.data_ptr(), w.dtype


def _gate_view(gate, rows, d, dtype):
    """(gates, packed view)."""
    if gate is None:
        return 0, None
    gates = _row_view(gate, "gate")[0]
    if gates < 1 or rows % gates:
        raise ValueError(f"{rows} rows are no multiple of {gates} gates")
    return gates, _pack_view(gate, "gate", gates, d, dtype)


def _norm_desc(rows, d, gates, act, res, w, post, pre, scale, eps):
    if rows >> 31 or d >> 31:
        raise ValueError("rows and d must lie below 2^31")
    flags = (NORM_POST if post else 0) | (NORM_PRE if pre else 0)
    return _pack_norm(rows, d, gates, _s._act_of(act), _s._act_of(res), 0 if w is None else _s._act_of(w), scale, eps,
                      flags, 0)


def block_norm(x, f=None, *, post=None, pre=None, gate=None, scale=1.0, eps=1e-6, r=None, h=None, stream=None):
    """The norms before and after a block, its gate and residual scale
    (ttt_block_norm): (r, h) with r = x + scale * gate * n, n = f or its RMS
    norm, and h the RMS norm of r. x: the residual stream [..., d]; f: what the
    block added to it, likewise (None: h of x alone, r is None). post, pre: the
    norms' weights [d], True for a norm without one, None for no norm (pre:
    None: h is None). gate: [..., d] of one row, of all rows, or of rows / n, each
    for n rows that follow each other (a gate a sequence; it does not broadcast
    over sequences). r and h may be given; r may be x."""
    rows, d, stride = _row_view(x, "x")
    act = x.dtype if f is None else f.dtype
    if f is None and h is not None:
        act = h.dtype
    _alone(x, f, gate, r, h, *(w for w in (post, pre) if isinstance(w, torch.Tensor)))
    has_post, wpost, kind = _weight(post, "post", d, None)
    has_pre, wpre, kind = _weight(pre, "pre", d, kind)
    gates, rgate = _gate_view(gate, rows, d, act)
    desc = _norm_desc(rows, d, gates, act, x.dtype, kind, has_post, has_pre, scale, eps)
    rf = rr = rh = None
    if f is not None:
        rf = _pack_view(f, "f", rows, d, act)
        r, rr = _out(r, "r", x, rows, d, x.dtype, stream)
    elif r is not None:
        raise ValueError("r without f")
    if has_pre:
        h, rh = _out(h, "h", x, rows, d, act, stream)
    elif h is not None:
        raise ValueError("h without pre")
    st = _L().ttt_block_norm(desc, _s._pack_rows(x.data_ptr(), stride, d, 1, 0), rf, wpost, wpre, rgate, rr, rh,
                             _s._stream(stream, x))
    if st:
        _b._check(st)
    return r, h


@functools.lru_cache(maxsize=1024)  # of sizes alone
def _norm_workspace(desc):
    n = _S(0)
    _b._check(_L().ttt_block_norm_backward_workspace_size(desc, _ref(n)))
    return n.value


def block_norm_backward(dr, dh, r, f=None, *, post=None, pre=None, gate=None, scale=1.0, eps=1e-6, dx=None, df=None,
                        workspace=None, stream=None):
    """The gradients of block_norm's inputs from those of r and h
    (ttt_block_norm_backward): a dict of dx, df, dgate, dpost and dpre, None
    for what was not given. dr: None is zero; dh and r (the forward's; x where
    there was no f): needed with pre. Sums over rows (dpost, dpre, dgate of
    gates that rows share) are float32; dx may be dr."""
    like = next((t for t in (r, dr, f) if t is not None), None)
    if like is None:
        raise ValueError("one of dr, r and f is needed")
    rows, d, _ = _row_view(like, "r")
    act = f.dtype if f is not None else dh.dtype if dh is not None else like.dtype
    res = r.dtype if r is not None else dr.dtype if dr is not None else dx.dtype if dx is not None else act
    _alone(like, dr, dh, r, f, gate, dx, df, *(w for w in (post, pre) if isinstance(w, torch.Tensor)))
    has_post, wpost, kind = _weight(post, "post", d, None)
    has_pre, wpre, kind = _weight(pre, "pre", d, kind)
    if has_pre and (dh is None or r is None):
        raise ValueError("pre needs dh and r")
    if dh is not None and not has_pre:
        raise ValueError("dh without pre")
    gates, rgate = _gate_view(gate, rows, d, act)
    desc = _norm_desc(rows, d, gates, act, res, kind, has_post, has_pre, scale, eps)
    rdr = None if dr is None else _pack_view(dr, "dr", rows, d, res)
    rdh = _pack_view(dh, "dh", rows, d, act) if has_pre else None
    rr = _pack_view(r, "r", rows, d, res) if has_pre else None
    dx, rdx = _out(dx, "dx", like, rows, d, res, stream)
    rf = rdf = rdg = dgate = None
    if f is not None:
        rf = _pack_view(f, "f", rows, d, act)
        df, rdf = _out(df, "df", f, rows, d, act, stream)
    elif df is not None:
        raise ValueError("df without f")
    if gate is not None:
        dgate = _new(gate.shape, act if gates == rows else torch.float32, gate, stream)
        rdg = _s._pack_rows(dgate.data_ptr(), d, d, 1, 0)
    dpost = None if wpost is None else _new((d,), torch.float32, like, stream)
    dpre = None if wpre is None else _new((d,), torch.float32, like, stream)
    workspace, ws, size = _workspace(_norm_workspace(desc), like, workspace, stream)
    st = _L().ttt_block_norm_backward(desc, rdr, rdh, rr, rf, wpost, wpre, rgate, rdx, rdf, rdg,
                                      None if dpost is None else dpost.data_ptr(),
                                      None if dpre is None else dpre.data_ptr(), ws, size, _s._stream(stream, like))
    if st:
        _b._check(st)
    return dict(dx=dx, df=df, dgate=dgate, dpost=dpost, dpre=dpre)


# -------------------------------------------------------- linear attention


def _linear_desc(q, k, v, log_decay, q_starts, max_new, scale, state):
    """(packed descriptor, its sizes without addresses, packed q, k, v, ...)"""
    n, hq, dk, rq = _s._rows_of(q, "q")
    act, dtype = _s._act(q, "q"), q.dtype
    _, hk, dv, _ = _s._rows_of(v, "v")
    rk, rv = _s._rows(k, "k", n, dk, dtype), _s._rows(v, "v", n, dv, dtype)
    if k.shape[-2] != hk:
        raise ValueError("k and v must have the same heads")
    if log_decay.dtype is not torch.float32 or log_decay.shape != (hk,) or not log_decay.is_cuda \
            or not log_decay.is_contiguous():
        raise ValueError(f"log_decay must be a contiguous float32 [{hk}] tensor on the GPU")
    if q_starts is not None:
        batch = q_starts.numel() - 1
        starts = _s._ints(q_starts, "q_starts", (batch + 1,))
    else:
        batch = q.shape[0] if q.dim() == 4 else state.shape[0] if state is not None and state.dim() == 4 else 1
        starts = None
    if batch < 1 or (q_starts is None and n % batch):
        raise ValueError(f"{n} rows are no whole number for each of {batch} sequences")
    if max_new is None:
        max_new = max(1, n if q_starts is not None else n // batch)
    if max_new >> 31 or max_new < 0:
        raise ValueError("max_new must lie below 2^31")
    if scale is None:
        scale = dk ** -0.5
    sizes = (batch, n, max_new, act, hk, hq, dk, dv)
    desc = _pack_linear(log_decay.data_ptr(), starts or 0, *sizes, scale, 0)
    return desc, sizes, rq, rk, rv


def _state_of(state, what, sizes):
    if state is None:
        return None
    shape = (sizes[0], sizes[4], sizes[6], sizes[7])
    if state.dtype is not torch.float32 or state.shape != shape or not state.is_cuda or not state.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 {list(shape)} tensor on the GPU")
    return state.data_ptr()


@functools.lru_cache(maxsize=1024)  # of sizes alone
def _linear_workspace(sizes, back):
    n = _S(0)
    fn = _L().ttt_linear_attention_backward_workspace_size if back else _L().ttt_linear_attention_workspace_size
    desc = _pack_linear(0, 0, sizes[0], 0, *sizes[2:], 1.0, 0)
    _b._check(fn(desc, _ref(n)))
    return n.value


def linear_attention(q, k, v, log_decay, *, state=None, q_starts=None, max_new=None, scale=None, out=None,
                     workspace=None, stream=None):
    """Linear attention with a decay for each head (ttt_linear_attention):
    S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t. q [rows,
    q_heads, dim_k], k [rows, kv_heads, dim_k], v [rows, kv_heads, dim_v], or
    [B, T, heads, dim] views; log_decay: float32 [kv_heads]. state: float32
    [batch, kv_heads, dim_k, dim_v], S before the first token, updated in place
    (None: zero, and not returned). q_starts: int32 [batch + 1], the sequences'
    first rows (None: the same number each); max_new: an upper bound of their
    rows where the caller knows a better one than all. scale: None is dim_k **
    -0.5. Returns o [rows, q_heads, dim_v] (rows that no sequence claims are
    left as they are)."""
    desc, sizes, rq, rk, rv = _linear_desc(q, k, v, log_decay, q_starts, max_new, scale, state)
    _alone(q, k, v, log_decay, q_starts, state, out)
    _, n, _, _, _, hq, _, dv = sizes
    if out is None:
        out = _new(q.shape[:-1] + (dv,), q.dtype, q, stream)
        ro = _s._dense(out, hq, dv)
    else:
        ro = _s._rows(out, "out", n, dv, q.dtype)
        if out.shape[-2] != hq:
            raise ValueError(f"out must have {hq} heads")
    ps = _state_of(state, "state", sizes)
    workspace, ws, size = _workspace(_linear_workspace(sizes, False), q, workspace, stream)
    st = _L().ttt_linear_attention(desc, rq, rk, rv, ro, ps, ws, size, _s._stream(stream, q))
    if st:
        _b._check(st)
    return out


def linear_attention_backward(do, q, k, v, log_decay, *, state=None, d_state=None, d_state0=None, q_starts=None,
                              max_new=None, scale=None, workspace=None, stream=None):
    """The gradients of linear_attention (ttt_linear_attention_backward): (dq,
    dk, dv, d_state0). do: the gradient of o; state: S before the first token
    (the forward's, before it was updated; None: zero); d_state: the gradient of
    S after the last (None: zero). d_state0, the gradient of the first state, is
    returned where state, d_state or d_state0 is given; it may be d_state. Rows that
    no sequence claims have gradients of zero."""
    desc, sizes, rq, rk, rv = _linear_desc(q, k, v, log_decay, q_starts, max_new, scale,
                                           next((s for s in (state, d_state, d_state0) if s is not None), None))
    _alone(q, do, k, v, log_decay, q_starts, state, d_state, d_state0)
    batch, n, _, _, hk, hq, dk, dv = sizes
    rdo = _s._rows(do, "do", n, dv, q.dtype)
    if do.shape[-2] != hq:
        raise ValueError(f"do must have {hq} heads")
    p0, p1 = _state_of(state, "state", sizes), _state_of(d_state, "d_state", sizes)
    if d_state0 is None and (p0 or p1):
        d_state0 = _new((batch, hk, dk, dv), torch.float32, q, stream)
    p2 = _state_of(d_state0, "d_state0", sizes)
    dq, g_k, g_v = (_s._empty(t, stream) for t in (q, k, v))
    workspace, ws, size = _workspace(_linear_workspace(sizes, True), q, workspace, stream)
    st = _L().ttt_linear_attention_backward(desc, rdo, rq, rk, rv, p0, p1, _s._dense(dq, hq, dk),
                                            _s._dense(g_k, hk, dk), _s._dense(g_v, hk, dv), p2, ws, size,
                                            _s._stream(stream, q))
    if st:
        _b._check(st)
    return dq, g_k, g_v, d_state0


# ------------------------------------------------------------------- AdamW


_T = torch.Tensor
_dtype_of = operator.attrgetter("dtype")


def _list(ts, what, dtype=None, sizes=None):
    """(addresses, sizes, dtype) of dense tensors of one dtype, the current
    GPU's. (Maps of methods: with some hundred tensors a comprehension's steps
    would take longer than the kernel.)"""
    ts = list(ts)
    if not ts:
        return [], [], dtype
    dtypes = set(map(_dtype_of, ts))
    if dtype is None:
        dtype = ts[0].dtype
    if (dtypes != {dtype} or set(map(_T.get_device, ts)) != {torch.cuda.current_device()}
            or not all(map(_T.is_contiguous, ts))):
        raise ValueError(f"{what} must be contiguous {dtype} tensors on the current GPU")
    n = list(map(_T.numel, ts))
    if sizes is not None and n != sizes:
        raise ValueError(f"{what} must have the parameters' sizes")
    return list(map(_T.data_ptr, ts)), n, dtype


def _scalar(x, what, dtype):
    """(value, address) of a number, or of one on the GPU."""
    if not isinstance(x, torch.Tensor):
        return x, 0
    if x.dtype is not dtype or x.numel() != 1 or x.get_device() != torch.cuda.current_device():
        raise ValueError(f"{what} on the device must be one {dtype} value on the current GPU")
    return 0, x.data_ptr()


def adamw_state_size(sizes, bits=32) -> int:
    """Bytes of the states of tensors of `sizes` values (ttt_adamw_state_size)."""
    sizes = list(sizes)
    n = _S(0)
    _b._check(_L().ttt_adamw_state_size((ctypes.c_int64 * len(sizes))(*sizes), len(sizes), bits, _ref(n)))
    return n.value


@functools.lru_cache(maxsize=256)  # of sizes alone
def _state_bytes(sizes, bits):
    """adamw_state_size, without a call for every step (0 for bits that the library refuses)."""
    return sum([-(-n // 256) for n in sizes]) * {32: 256 * 8, 8: 256 * 2 + 8}.get(bits, 0)


def adamw_state(params, bits=32):
    """Fresh states of adamw_step for `params`: a uint8 buffer of zeros."""
    params = list(params)
    return torch.zeros(adamw_state_size([p.numel() for p in params], bits), dtype=torch.uint8,
                       device=params[0].device if params else "cuda")


def adamw_step(params, grads, state, *, lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, bits=32,
               masters=None, norm=None, max_norm=0.0, stream=None):
    """One AdamW step on `params` (bfloat16 or float32, updated in place) from
    `grads` (bfloat16 or float32, the params' sizes), with the states of
    adamw_state(params, bits) (ttt_adamw_step). step counts from 1; lr and step
    may be a float32 and an int32 value on the GPU, which a captured call reads
    again at every replay (a step below 1 there changes nothing). masters: float32 values of bfloat16 params, which
    take the step in their place. norm: grad_norm(grads), to limit the
    gradients to max_norm; where it is infinite or NaN, nothing changes."""
    pp, sizes, pt = _list(params, "params")
    pg, _, gt = _list(grads, "grads", None, sizes)
    n = len(pp)
    if not n:
        return
    pm = [0] * n if masters is None else _list(masters, "masters", torch.float32, sizes)[0]
    if state.dtype is not torch.uint8 or state.get_device() != torch.cuda.current_device() or not state.is_contiguous():
        raise ValueError("state must be a contiguous uint8 tensor on the current GPU")
    need = _state_bytes(tuple(sizes), bits)
    if state.nbytes != need and need:  # (a larger one would be other tensors', or of other bits)
        raise ValueError(f"state must be adamw_state(params, {bits}), of {need} bytes")
    lr, plr = _scalar(lr, "lr", torch.float32)
    step, pstep = _scalar(step, "step", torch.int32)
    step = operator.index(step)  # (a TypeError for what is no whole number)
    pnorm = 0 if norm is None else _scalar(norm, "norm", torch.float32)[1]
    if norm is not None and not pnorm:
        raise ValueError("norm must be on the GPU")
    if not -(1 << 31) <= step < 1 << 31:
        raise ValueError("step must fit 32 bits")
    flat = [0] * (4 * n)
    flat[0::4], flat[1::4], flat[2::4], flat[3::4] = pp, pm, pg, sizes
    st = _L().ttt_adamw_step(
        _pack_adamw(_s._act_of(pt), _s._act_of(gt), bits, step, lr, betas[0], betas[1], eps, weight_decay, max_norm,
                    pnorm, plr, pstep),
        struct.pack("%dQ" % (4 * n), *flat), n, state.data_ptr(), state.nbytes, _s._stream(stream, state))
    if st:
        _b._check(st)


def adamw_read(state, bits=32, *, dtype=torch.float32, stream=None):
    """(m, v) that a state buffer holds: values of all tensors one after the
    other, each tensor padded to a multiple of 256. 32 bits: views of the
    buffer; 8 bits: what the codes stand for, rounded to dtype
    (ttt_adamw_read)."""
    if state.dtype is not torch.uint8 or not state.is_cuda or not state.is_contiguous():
        raise ValueError("state must be a contiguous uint8 tensor on the GPU")
    per = {32: 256 * 8, 8: 256 * 2 + 8}.get(bits)
    if per is None or state.numel() % per:
        raise ValueError(f"{state.numel()} bytes are no states of {bits} bits")
    n = state.numel() // per * 256
    if bits == 32:
        if dtype is not torch.float32:
            raise TypeError("states of 32 bits are read as float32")
        m, v = state.view(torch.float32).view(2, n)
        return m, v
    _alone(state)
    m, v = (_new((n,), dtype, state, stream) for _ in range(2))
    st = _L().ttt_adamw_read(state.data_ptr(), n, _s._act_of(dtype), m.data_ptr(), v.data_ptr(),
                             _s._stream(stream, state))
    if st:
        _b._check(st)
    return m, v


@functools.lru_cache(maxsize=1024)  # of sizes alone
def _grad_norm_workspace(n):
    size = _S(0)
    _b._check(_L().ttt_grad_norm_workspace_size(n, _ref(size)))
    return size.value


def grad_norm(grads, *, out=None, workspace=None, stream=None):
    """The 2-norm of all values of `grads` (bfloat16 or float32) together
    (ttt_grad_norm): a float32 value on the GPU."""
    grads = list(grads)
    pg, sizes, gt = _list(grads, "grads")
    if not pg:
        raise ValueError("no gradients")
    if out is None:
        out = _new((), torch.float32, grads[0], stream)
    elif out.dtype is not torch.float32 or out.numel() != 1 or out.get_device() != grads[0].get_device():
        raise ValueError("out must be one float32 value on the GPU")
    workspace, ws, size = _workspace(_grad_norm_workspace(len(pg)), grads[0], workspace, stream)
    n = len(pg)
    st = _L().ttt_grad_norm(struct.pack("%dQ" % n, *pg), struct.pack("%dq" % n, *sizes), n, _s._act_of(gt),
                            out.data_ptr(), ws, size, _s._stream(stream, grads[0]))
    if st:
        _b._check(st)
    return out
