"""CPU-only: the entry points of the attention half of a block reject bad
arguments before any launch. No call here reaches a kernel; pointers are fake
aligned addresses that are never dereferenced."""
import ctypes

import pytest

from test_layer_gate_amd import _binding as bnd
from test_layer_gate_amd import _serve as sv

OK, INVALID, UNSUPPORTED, WORKSPACE, ALIAS = 0, -1, -2, -3, -4
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    return sv._L()


def ref(x):
    return None if x is None else ctypes.byref(x)


def rows(at, heads=8, dim=128, ts=None, hs=None):
    return sv.Rows(at, heads * dim if ts is None else ts, dim if hs is None else hs, heads, 0)


def rope(**kw):
    r = sv.Rope(1000 * MB, 128, 4096, 0, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def cache(**kw):
    c = sv.Cache(2000 * MB, 8 * 64 * 136, 3000 * MB, 3001 * MB, 3002 * MB, 4, 16, 64, 64, 8, 128, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def attn(**kw):
    a = sv.Attn(0.1, 0, 16, 1024, 0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def rope_call(L, tokens=16, seq=16, dim=128, act=0, r=None, pos=4000 * MB, q=None, k=None, qo=None,
              ko=None, none=()):
    a = dict(q=q or rows(1 * MB, 32), k=k or rows(5 * MB), qo=qo or rows(9 * MB, 32), ko=ko or rows(13 * MB),
             r=r or rope())
    a.update({n: None for n in none})
    return L.ttt_rope_forward(tokens, seq, dim, act, ref(a["r"]), pos, ref(a["q"]), ref(a["k"]),
                              ref(a["qo"]), ref(a["ko"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVALID), (dict(tokens=(1 << 24) + 1), UNSUPPORTED), (dict(act=2), INVALID),
    (dict(dim=8), INVALID), (dict(dim=120), UNSUPPORTED), (dict(dim=2048), UNSUPPORTED),
    (dict(pos=None, seq=0), INVALID), (dict(pos=4000 * MB + 2), INVALID),
    (dict(r=rope(table=None)), INVALID), (dict(r=rope(table=1000 * MB + 8)), INVALID),
    (dict(r=rope(rot_dim=0)), INVALID), (dict(r=rope(rot_dim=144)), INVALID),
    (dict(r=rope(rot_dim=40)), UNSUPPORTED), (dict(r=rope(max_pos=0)), INVALID),
    (dict(r=rope(flags=2)), INVALID), (dict(r=rope(reserved=1)), INVALID),
    (dict(none=("q",)), INVALID), (dict(none=("qo",)), INVALID), (dict(none=("k",)), INVALID),
    (dict(none=("ko",)), INVALID), (dict(none=("r",)), INVALID),
    (dict(q=rows(1 * MB + 8, 32)), INVALID), (dict(q=rows(None, 32)), INVALID),
    (dict(q=rows(1 * MB, 32, ts=4100)), INVALID), (dict(q=rows(1 * MB, 32, hs=-128)), INVALID),
    (dict(q=rows(1 * MB, 0)), INVALID), (dict(q=rows(1 * MB, 2000)), UNSUPPORTED),
    (dict(q=rows(1 * MB, 31)), INVALID), (dict(ko=rows(13 * MB, 4)), INVALID),
    (dict(qo=rows(9 * MB, 32, ts=0)), ALIAS), (dict(qo=rows(9 * MB, 32, hs=64)), ALIAS),
    (dict(qo=rows(1 * MB + 4096, 32)), ALIAS), (dict(qo=rows(5 * MB, 32)), ALIAS),
    (dict(ko=rows(9 * MB)), ALIAS), (dict(qo=rows(1000 * MB, 32)), ALIAS),
    (dict(ko=rows(4000 * MB)), ALIAS),
])
def test_rope_refusals(L, kw, code):
    assert rope_call(L, **kw) == code, L.ttt_last_error()
    assert L.ttt_last_error().decode()


def test_rope_empty_and_aliases_that_are_fine(L):
    assert rope_call(L, tokens=0) == OK
    fused = 48 * 128
    q, k = rows(1 * MB, 32, ts=fused), rows(1 * MB + 32 * 128 * 2, 8, ts=fused)
    # in place in a fused projection: refused only for what follows the checks
    # (a table inside the output), which shows that the views passed
    assert rope_call(L, q=q, k=k, qo=q, ko=k, r=rope(table=1 * MB)) == ALIAS
    assert b"rope table" in L.ttt_last_error()
    v = rows(1 * MB + 31 * 128 * 2, 8, ts=fused)       # overlaps q's last head
    assert rope_call(L, q=q, k=v, qo=q, ko=v) == ALIAS
    assert b"rope table" not in L.ttt_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), INVALID), (dict(max_pos=0), INVALID), (dict(rot=0), INVALID),
    (dict(rot=20), UNSUPPORTED), (dict(max_pos=(1 << 26) + 1), UNSUPPORTED), (dict(base=1.0), INVALID), (dict(base=float("inf")), INVALID),
    (dict(kind=5), INVALID), (dict(kind=-1), INVALID), (dict(factor=0.5), INVALID),
    (dict(kind=3, original=0.0), INVALID), (dict(kind=3, low=0.0), INVALID),
    (dict(kind=4, low=4.0, high=4.0), INVALID), (dict(amplitude=0.0), INVALID),
    (dict(factor=float("nan")), INVALID), (dict(reserved=1), INVALID),
])
def test_rope_table_refusals(L, kw, code):
    a = dict(table=16 * MB, max_pos=64, rot=64, base=1e4, kind=1, factor=2.0, original=64.0, low=1.0,
             high=4.0, amplitude=1.0, reserved=0)
    a.update(kw)
    sc = sv.RopeScaling(a["kind"], a["reserved"], a["factor"], a["original"], a["low"], a["high"],
                        a["amplitude"])
    assert L.ttt_rope_table(a["table"], a["max_pos"], a["rot"], a["base"], ref(sc), None) == code


@pytest.mark.parametrize("page,heads,dim,code", [
    (64, 8, 128, OK), (16, 1, 64, OK), (48, 3, 256, OK), (4096, 1, 128, OK), (0, 8, 128, INVALID),
    (64, 0, 128, INVALID), (64, 8, 0, INVALID), (40, 8, 128, UNSUPPORTED), (8192, 8, 128, UNSUPPORTED),
    (64, 8, 96, UNSUPPORTED), (64, 2000, 128, UNSUPPORTED)])
def test_page_bytes(L, page, heads, dim, code):
    n = ctypes.c_size_t(0)
    assert L.ttt_kv_page_bytes(page, heads, dim, ref(n)) == code
    if code == OK:
        assert n.value == heads * page * (dim // 2 + dim // 32) * 2
    assert L.ttt_kv_page_bytes(64, 8, 128, None) == INVALID


BAD_CACHES = [
    (dict(reserved=1), INVALID), (dict(batch=0), INVALID), (dict(batch=70000), UNSUPPORTED),
    (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(page_size=40), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(kv_heads=0), INVALID), (dict(page_stride=1024), INVALID),
    (dict(page_stride=8 * 64 * 136 + 8), INVALID), (dict(pages=None), INVALID),
    (dict(pages=2000 * MB + 8), INVALID), (dict(page_table=None), INVALID), (dict(kv_lens=None), INVALID),
    (dict(kv_lens=3001 * MB + 1), INVALID), (dict(q_starts=3002 * MB + 2), INVALID),
    (dict(q_starts=None, batch=3), INVALID), (dict(max_pages=1 << 26), UNSUPPORTED),
    (dict(max_pages=(1 << 24) + 1), UNSUPPORTED)]


def append_call(L, c=None, tokens=16, act=0, k=None, v=None, q=None, qo=None, r=None, pos=None, none=()):
    a = dict(c=c or cache(), k=k or rows(5 * MB), v=v or rows(9 * MB), q=q or rows(13 * MB, 32),
             qo=qo or rows(17 * MB, 32), r=r or rope())
    a.update({n: None for n in none})
    return L.ttt_kv_append(ref(a["c"]), tokens, act, ref(a["k"]), ref(a["v"]), ref(a["q"]), ref(a["qo"]),
                           ref(a["r"]), pos, None)


@pytest.mark.parametrize("kw,code", [(dict(c=cache(**k)), code) for k, code in BAD_CACHES] + [
    (dict(none=("c",)), INVALID), (dict(none=("k",)), INVALID), (dict(none=("v",)), INVALID),
    (dict(none=("q",)), INVALID), (dict(none=("r",)), INVALID), (dict(tokens=-4), INVALID),
    (dict(act=9), INVALID), (dict(k=rows(5 * MB, 4)), INVALID), (dict(v=rows(9 * MB, 4)), INVALID),
    (dict(qo=rows(17 * MB, 16)), INVALID), (dict(k=rows(2000 * MB)), ALIAS), (dict(qo=rows(5 * MB, 32)), ALIAS),
    (dict(qo=rows(2000 * MB, 32)), ALIAS), (dict(qo=rows(3001 * MB, 32)), ALIAS),
    (dict(pos=4000 * MB + 1), INVALID), (dict(pos=2000 * MB), ALIAS), (dict(r=rope(table=2000 * MB)), ALIAS),
    (dict(c=cache(kv_lens=2000 * MB)), ALIAS)])
def test_append_refusals(L, kw, code):
    assert append_call(L, **kw) == code, L.ttt_last_error()
    assert append_call(L, tokens=0) == OK


@pytest.mark.parametrize("kw,code", [(dict(c=cache(**k)), code) for k, code in BAD_CACHES] + [
    (dict(k=rows(5 * MB, 4)), INVALID), (dict(k=rows(5 * MB, 8, ts=0)), ALIAS), (dict(act=5), INVALID),
    (dict(k=rows(9 * MB)), ALIAS), (dict(v=rows(2000 * MB)), ALIAS), (dict(v=rows(3000 * MB)), ALIAS)])
def test_read_refusals(L, kw, code):
    a = dict(c=cache(), tokens=16, act=0, k=rows(5 * MB), v=rows(9 * MB))
    a.update(kw)
    assert L.ttt_kv_read(ref(a["c"]), a["tokens"], a["act"], ref(a["k"]), ref(a["v"]), None) == code
    assert L.ttt_kv_read(ref(cache()), 0, 0, ref(rows(5 * MB)), ref(rows(9 * MB)), None) == OK


BAD_ATTN = [
    (dict(reserved=1), INVALID), (dict(flags=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(window=-1), INVALID), (dict(window=4, flags=1), INVALID), (dict(max_new=0), INVALID),
    (dict(max_kv=0), INVALID)]


@pytest.mark.parametrize("kw,code", [(dict(c=cache(**k)), code) for k, code in BAD_CACHES] +
                         [(dict(a=attn(**k)), code) for k, code in BAD_ATTN] + [
    (dict(tokens=-4), INVALID), (dict(act=7), INVALID),
    (dict(tokens=1 << 24, q=rows(5 * MB, 128), o=rows(9 * MB, 128)), UNSUPPORTED), (dict(q=rows(5 * MB, 12), o=rows(9 * MB, 12)), INVALID),
    (dict(o=rows(9 * MB, 16)), INVALID), (dict(o=rows(5 * MB, 32)), ALIAS), (dict(o=rows(2000 * MB, 32)), ALIAS),
    (dict(lse=5 * MB), ALIAS), (dict(lse=13 * MB + 2), INVALID), (dict(lse=9 * MB), ALIAS),
    (dict(ws=None), INVALID), (dict(ws=100 * MB + 16), INVALID), (dict(ws=5 * MB), ALIAS),
    (dict(ws=2000 * MB), ALIAS), (dict(ws_bytes=64), WORKSPACE)])
def test_attention_refusals(L, kw, code):
    a = dict(c=cache(), a=attn(max_new=4, max_kv=65536), tokens=16, act=0, q=rows(5 * MB, 32),
             o=rows(9 * MB, 32), lse=13 * MB, ws=100 * MB, ws_bytes=500 * MB)
    a.update(kw)
    st = L.ttt_kv_attention(ref(a["c"]), ref(a["a"]), a["tokens"], a["act"], ref(a["q"]), ref(a["o"]),
                            a["lse"], a["ws"], a["ws_bytes"], None)
    assert st == code, L.ttt_last_error()


def test_attention_workspace(L):
    def size(tokens, batch=1, hk=8, hq=32, dim=128, **kw):
        n = ctypes.c_size_t(0)
        st = L.ttt_kv_attention_workspace_size(ref(attn(**kw)), batch, tokens, 0, hk, hq, dim, ref(n))
        return st, n.value
    st, n = size(1, max_new=1, max_kv=131072)
    assert st == OK and n >= 32 * 128 * 4 * 2
    assert size(8192, max_new=8192, max_kv=8192) == (OK, 0)       # rows enough without splitting
    assert size(1, max_new=1, max_kv=16) == (OK, 0)
    for kw, code in BAD_ATTN:
        assert size(1, **kw)[0] == code
    assert size(-1)[0] == INVALID and size(1, hq=9)[0] == INVALID and size(1, dim=80)[0] == UNSUPPORTED
    assert L.ttt_kv_attention_workspace_size(ref(attn()), 1, 1, 0, 8, 32, 128, None) == INVALID


def test_struct_layouts_match_the_header():
    """The sizes a C compiler gives the header's structs on x86-64."""
    for t, n in ((sv.Rows, 32), (sv.Rope, 24), (sv.RopeScaling, 48), (sv.Cache, 72), (sv.Attn, 24)):
        assert ctypes.sizeof(t) == n
    assert bnd.TTT_BF16 == 0
