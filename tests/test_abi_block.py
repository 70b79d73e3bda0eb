"""CPU-only: the entry points of norms, linear attention and AdamW reject bad
arguments before any launch. No call here reaches a kernel; pointers are fake
aligned addresses that are never dereferenced."""
import ctypes
import struct

import pytest

from test_layer_gate_amd import _binding as bnd
from test_layer_gate_amd import _block as bl
from test_layer_gate_amd import _serve as sv

OK, INVALID, UNSUPPORTED, WORKSPACE, ALIAS = 0, -1, -2, -3, -4
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    return bl._L()


def ref(x):
    return None if x is None else ctypes.byref(x)


def change(s, kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def row(at, d=256, ts=None, heads=1):
    return sv.Rows(at * MB, d if ts is None else ts, d, heads, 0)


# ------------------------------------------------------------------ norms


def norm(**kw):
    return change(bl.Norm(16, 256, 1, 0, 0, 0, 1.0, 1e-6, 3, 0), kw)


def norm_call(L, none=(), at=None, **kw):
    p = dict(x=row(1), f=row(2), post=3 * MB, pre=4 * MB, gate=row(5), r=row(6), h=row(7))
    p.update(at or {})
    p.update({n: None for n in none})
    return L.ttt_block_norm(ref(norm(**kw)), ref(p["x"]), ref(p["f"]), p["post"], p["pre"], ref(p["gate"]), ref(p["r"]),
                            ref(p["h"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(rows=(1 << 24) + 1), UNSUPPORTED), (dict(d=0), INVALID), (dict(d=12), UNSUPPORTED),
    (dict(d=16392), UNSUPPORTED), (dict(act_dtype=2), INVALID), (dict(res_dtype=3), INVALID),
    (dict(weight_dtype=-1), INVALID), (dict(act_dtype=1), UNSUPPORTED), (dict(gates=-1), INVALID), (dict(gates=3), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(flags=4), INVALID), (dict(reserved=1), INVALID), (dict(gates=0), INVALID),
    (dict(none=("gate",)), INVALID), (dict(none=("x",)), INVALID), (dict(none=("f",)), INVALID), (dict(none=("r",)), INVALID),
    (dict(none=("h",)), INVALID), (dict(flags=1), INVALID), (dict(flags=2), INVALID),
    (dict(none=("f", "r", "post", "gate"), gates=0, flags=0), INVALID),
    (dict(at=dict(x=row(1, heads=2))), INVALID), (dict(at=dict(post=3 * MB + 8)), INVALID),
    (dict(at=dict(f=row(2, ts=255))), INVALID), (dict(at=dict(r=row(6, ts=128))), ALIAS),
    (dict(at=dict(r=row(2))), ALIAS), (dict(at=dict(h=row(1))), ALIAS), (dict(at=dict(h=row(6))), ALIAS),
    (dict(at=dict(h=row(5))), ALIAS), (dict(at=dict(r=sv.Rows(3 * MB - 64, 256, 256, 1, 0))), ALIAS),
    (dict(at=dict(r=row(1, ts=512))), ALIAS),
])
def test_norm_refuses(L, kw, code):
    assert norm_call(L, **kw) == code, L.ttt_last_error()


def test_norm_without_rows_is_a_call(L):
    assert norm_call(L, rows=0, gates=1) == OK


def back_call(L, none=(), at=None, size=None, **kw):
    n = norm(**kw)
    p = dict(dr=row(1), dh=row(2), r=row(3), f=row(4), post=5 * MB, pre=6 * MB, gate=row(7), dx=row(8), df=row(9), dgate=row(10),
             dpost=11 * MB, dpre=12 * MB, ws=13 * MB)
    p.update(at or {})
    p.update({k: None for k in none})
    return L.ttt_block_norm_backward(ref(n), *(ref(p[k]) for k in ("dr", "dh", "r", "f")), p["post"], p["pre"],
                                     ref(p["gate"]), ref(p["dx"]), ref(p["df"]), ref(p["dgate"]), p["dpost"], p["dpre"],
                                     p["ws"], 8 * MB if size is None else size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(none=("dh",)), INVALID), (dict(none=("r",)), INVALID), (dict(none=("dx",)), INVALID), (dict(none=("df",)), INVALID),
    (dict(none=("dgate",)), INVALID), (dict(none=("dpost",)), INVALID), (dict(none=("dpre",)), INVALID),
    (dict(none=("post",)), INVALID), (dict(none=("ws",)), INVALID), (dict(size=16), WORKSPACE),
    (dict(at=dict(ws=13 * MB + 16)), INVALID), (dict(at=dict(dx=row(3))), ALIAS), (dict(at=dict(df=row(1))), ALIAS),
    (dict(at=dict(dx=row(1, ts=512))), ALIAS), (dict(at=dict(dgate=row(7))), ALIAS), (dict(at=dict(dpost=12 * MB)), ALIAS),
    (dict(at=dict(ws=4 * MB)), ALIAS), (dict(at=dict(dpre=6 * MB)), ALIAS), (dict(d=20), UNSUPPORTED),
])
def test_norm_backward_refuses(L, kw, code):
    assert back_call(L, **kw) == code, L.ttt_last_error()


# -------------------------------------------------------- linear attention


def linear(**kw):
    return change(bl.Linear(1 * MB, 2 * MB, 4, 400, 128, 0, 2, 4, 64, 128, 0.125, 0), kw)


def heads(at, h, d, ts=None, hs=None):
    return sv.Rows(at * MB, h * d if ts is None else ts, d if hs is None else hs, h, 0)


def linear_call(L, none=(), at=None, size=64 * MB, **kw):
    p = dict(q=heads(10, 4, 64), k=heads(20, 2, 64), v=heads(30, 2, 128), o=heads(40, 4, 128), state=50 * MB, ws=100 * MB)
    p.update(at or {})
    p.update({n: None for n in none})
    return L.ttt_linear_attention(ref(linear(**kw)), ref(p["q"]), ref(p["k"]), ref(p["v"]), ref(p["o"]), p["state"], p["ws"],
                                  size, None)


BAD_LINEAR = [
    (dict(batch=0), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(tokens=-1), INVALID), (dict(tokens=(1 << 24) + 1), UNSUPPORTED),
    (dict(max_new=0), INVALID), (dict(max_new=1 << 25), UNSUPPORTED), (dict(act_dtype=2), INVALID), (dict(kv_heads=0), INVALID),
    (dict(kv_heads=3), INVALID), (dict(q_heads=2048), UNSUPPORTED), (dict(dim_k=96), UNSUPPORTED), (dict(dim_v=0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(reserved=1), INVALID), (dict(q_starts=None, batch=3), INVALID),
    (dict(log_decay=None), INVALID), (dict(log_decay=MB + 2), INVALID), (dict(q_starts=MB + 1), INVALID),
    (dict(batch=65535, kv_heads=1024, q_heads=1024), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_LINEAR + [
    (dict(none=("q",)), INVALID), (dict(none=("o",)), INVALID), (dict(at=dict(k=heads(20, 4, 64))), INVALID),
    (dict(at=dict(o=heads(40, 2, 128))), INVALID), (dict(at=dict(q=heads(10, 4, 64, ts=255))), INVALID),
    (dict(at=dict(state=50 * MB + 4)), INVALID), (dict(at=dict(o=heads(10, 4, 128))), ALIAS),
    (dict(at=dict(state=30 * MB)), ALIAS), (dict(at=dict(state=40 * MB)), ALIAS), (dict(at=dict(o=heads(40, 4, 128, ts=128))), ALIAS),
    (dict(max_new=4096, none=("ws",)), INVALID), (dict(max_new=4096, size=1), WORKSPACE),
    (dict(max_new=4096, at=dict(ws=30 * MB)), ALIAS), (dict(max_new=4096, at=dict(ws=100 * MB + 8)), INVALID),
    (dict(at=dict(o=sv.Rows(1 * MB - 128, 512, 128, 4, 0))), ALIAS),
])
def test_linear_refuses(L, kw, code):
    assert linear_call(L, **kw) == code, L.ttt_last_error()


def linear_back(L, none=(), at=None, size=256 * MB, **kw):
    p = dict(do=heads(10, 4, 128), q=heads(20, 4, 64), k=heads(30, 2, 64), v=heads(40, 2, 128), s=50 * MB, ds=60 * MB,
             dq=heads(70, 4, 64), dk=heads(80, 2, 64), dv=heads(90, 2, 128), ds0=100 * MB, ws=128 * MB)
    p.update(at or {})
    p.update({n: None for n in none})
    return L.ttt_linear_attention_backward(ref(linear(**kw)), *(ref(p[n]) for n in ("do", "q", "k", "v")), p["s"], p["ds"],
                                           *(ref(p[n]) for n in ("dq", "dk", "dv")), p["ds0"], p["ws"], size, None)


@pytest.mark.parametrize("kw,code", BAD_LINEAR + [
    (dict(none=("do",)), INVALID), (dict(none=("dv",)), INVALID), (dict(at=dict(dk=heads(70, 2, 64))), ALIAS),
    (dict(at=dict(dq=heads(20, 4, 64))), ALIAS), (dict(at=dict(ds0=50 * MB)), ALIAS), (dict(at=dict(do=heads(10, 2, 128))), INVALID),
    (dict(max_new=4096, none=("ws",)), INVALID), (dict(max_new=4096, size=1), WORKSPACE),
])
def test_linear_backward_refuses(L, kw, code):
    assert linear_back(L, **kw) == code, L.ttt_last_error()


def test_linear_workspace(L):
    n = ctypes.c_size_t(7)
    assert L.ttt_linear_attention_workspace_size(ref(linear(max_new=8)), ctypes.byref(n)) == OK and n.value == 0
    assert L.ttt_linear_attention_workspace_size(ref(linear(max_new=1 << 20, dim_k=256, dim_v=256, batch=1)),
                                                 ctypes.byref(n)) == OK
    assert 0 < n.value <= 1024 * 256 * 256 * 4          # bounded, however long the prompt
    one = n.value
    assert L.ttt_linear_attention_backward_workspace_size(ref(linear(max_new=1 << 20, dim_k=256, dim_v=256, batch=1)),
                                                          ctypes.byref(n)) == OK and 0 < n.value <= 2 * one  # (two sets, fewer parts)
    assert L.ttt_linear_attention_workspace_size(ref(linear()), None) == INVALID
    assert L.ttt_linear_attention_workspace_size(None, ctypes.byref(n)) == INVALID


# ------------------------------------------------------------------- AdamW


def params(*ps):
    return b"".join(struct.pack("4Q", *p) for p in ps)


def adamw(**kw):
    a = bl.AdamW(0, 1, 8, 1, 1e-3, 0.9, 0.999, 1e-8, 0.1, 1.0, None, None, None)
    return change(a, kw)


def step(L, ps=None, n=None, state=64 * MB, size=32 * MB, **kw):
    ps = [(1 * MB, 0, 10 * MB, 1000)] if ps is None else ps
    return L.ttt_adamw_step(ref(adamw(**kw)), params(*ps), len(ps) if n is None else n, state, size, None)


GOOD = (1 * MB, 0, 10 * MB, 1000)


@pytest.mark.parametrize("kw,code", [
    (dict(param_dtype=2), INVALID), (dict(grad_dtype=2), INVALID), (dict(bits=16), INVALID), (dict(step=0), INVALID),
    (dict(lr=-1.0), INVALID), (dict(lr=float("nan")), INVALID), (dict(beta1=1.0), INVALID), (dict(beta2=-0.1), INVALID),
    (dict(beta2=float("nan")), INVALID), (dict(eps=-1.0), INVALID), (dict(weight_decay=float("inf")), INVALID),
    (dict(norm=2 * MB, max_norm=0.0), INVALID), (dict(norm=2 * MB + 2), INVALID), (dict(n=-1), INVALID),
    (dict(lr_device=3), INVALID), (dict(step_device=5), INVALID),
    (dict(ps=[(1 * MB + 8, 0, 10 * MB, 8)]), INVALID), (dict(ps=[(1 * MB, 0, 10 * MB + 4, 8)]), INVALID),
    (dict(ps=[(0, 0, 10 * MB, 8)]), INVALID), (dict(ps=[(1 * MB, 0, 0, 8)]), INVALID),
    (dict(ps=[(1 * MB, 5 * MB + 8, 10 * MB, 8)]), INVALID), (dict(ps=[(1 * MB, 5 * MB, 10 * MB, 8)], param_dtype=1), INVALID),
    (dict(ps=[GOOD, (2 * MB, 5 * MB, 11 * MB, 8)]), INVALID), (dict(ps=[(1 * MB, 0, 10 * MB, (1 << 40) + 1)]), UNSUPPORTED),
    (dict(state=None), INVALID), (dict(state=64 * MB + 16), INVALID), (dict(size=100), WORKSPACE),
    (dict(ps=[GOOD, GOOD]), ALIAS),                                             # the same tensor twice
    (dict(ps=[GOOD, (1 * MB + 1984, 0, 11 * MB, 1000)]), ALIAS),
    (dict(ps=[(1 * MB, 0, 1 * MB, 1000)]), ALIAS), (dict(state=10 * MB), ALIAS), (dict(norm=1 * MB), ALIAS),
    (dict(norm=64 * MB), ALIAS), (dict(ps=[(1 * MB, 10 * MB, 10 * MB, 1000)]), ALIAS),
])
def test_adamw_refuses(L, kw, code):
    assert step(L, **kw) == code, L.ttt_last_error()


def test_adamw_of_nothing_is_a_call(L):
    assert step(L, ps=[], state=None, size=0) == OK
    assert step(L, ps=[(0, 0, 0, 0)], state=None, size=0) == OK


def test_adamw_state_size(L):
    n = ctypes.c_size_t(0)
    sizes = (ctypes.c_int64 * 3)(1, 256, 257)
    assert L.ttt_adamw_state_size(sizes, 3, 32, ctypes.byref(n)) == OK and n.value == 1024 * 8
    assert L.ttt_adamw_state_size(sizes, 3, 8, ctypes.byref(n)) == OK and n.value == 1024 * 2 + 4 * 8
    assert L.ttt_adamw_state_size(sizes, 3, 4, ctypes.byref(n)) == INVALID
    assert L.ttt_adamw_state_size((ctypes.c_int64 * 1)(-1), 1, 8, ctypes.byref(n)) == INVALID
    assert L.ttt_adamw_state_size((ctypes.c_int64 * 2)(1 << 40, 1), 2, 8, ctypes.byref(n)) == UNSUPPORTED
    assert L.ttt_adamw_state_size(None, 1, 8, ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("args,code", [
    ((64 * MB, 100, 0, MB, 2 * MB), INVALID), ((64 * MB, 256, 2, MB, 2 * MB), INVALID), ((None, 256, 0, MB, 2 * MB), INVALID),
    ((64 * MB, 256, 0, None, 2 * MB), INVALID), ((64 * MB, 256, 0, MB, MB), ALIAS), ((64 * MB, 256, 1, 64 * MB, MB), ALIAS),
    ((64 * MB, -256, 0, MB, 2 * MB), INVALID), ((64 * MB, 0, 0, None, None), OK)])
def test_adamw_read_refuses(L, args, code):
    assert L.ttt_adamw_read(*args, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(grads=[MB + 8]), INVALID), (dict(grads=[0]), INVALID), (dict(dtype=2), INVALID), (dict(norm=None), INVALID),
    (dict(norm=MB), ALIAS), (dict(ws=MB), ALIAS), (dict(ws=None), INVALID), (dict(size=8), WORKSPACE), (dict(sizes=[-1]), INVALID),
    (dict(sizes=[(1 << 40) + 1]), UNSUPPORTED), (dict(norm=4 * MB), ALIAS)])
def test_grad_norm_refuses(L, kw, code):
    a = dict(grads=[MB], sizes=[100], dtype=0, norm=8 * MB, ws=4 * MB, size=MB)
    a.update(kw)
    n = len(a["grads"])
    assert L.ttt_grad_norm(struct.pack("%dQ" % n, *a["grads"]), struct.pack("%dq" % n, *a["sizes"]), n, a["dtype"], a["norm"],
                           a["ws"], a["size"], None) == code


def test_packed_descriptors_have_the_structures_layout():
    assert len(bl._pack_norm(*[0] * 10)) == ctypes.sizeof(bl.Norm)
    assert len(bl._pack_linear(*[0] * 12)) == ctypes.sizeof(bl.Linear)
    assert len(bl._pack_adamw(*[0] * 13)) == ctypes.sizeof(bl.AdamW)
    assert ctypes.sizeof(bl.Param) == 32
    n = bl.Norm.from_buffer_copy(bl._pack_norm(1, 2, 3, 4, 5, 6, 0.5, 0.25, 7, 0))
    assert (n.rows, n.d, n.gates, n.scale, n.eps, n.flags) == (1, 2, 3, 0.5, 0.25, 7)
    a = bl.AdamW.from_buffer_copy(bl._pack_adamw(1, 2, 3, 4, *[float(x) for x in range(6)], 7, 8, 9))
    assert (a.bits, a.step, a.lr, a.max_norm, a.norm, a.step_device) == (3, 4, 0.0, 5.0, 7, 9)
    assert bnd.lib() is not None
