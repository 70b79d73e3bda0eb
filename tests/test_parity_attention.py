"""GPU parity of attention over the paged 4-bit cache against the float64
oracle on the same cache bytes.

Tolerances (per output value, w = sum_j p_j |v_j| from the oracle). A weight
p_j carries the relative error of its exponent: a score is a sum of D exact
products (bf16 times bf16) accumulated in fp32, so at most D 2^-24 sum |q k|
scale, typically its square root; then the exponential's own 2^-22. Rounding
p to bf16 (8 significant bits) is at most 2^-8 of it, the output's own rounding
2^-8 of the value. fp32
rows take neither; their three-term queries and weights leave 2^-24 each.
Accumulating n weighted values in fp32 adds at most 2^-24 n w, typically its
square root (held to 4 sqrt(n) below)."""
import numpy as np
import pytest
import torch

import oracle.serve_oracle as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def pool_of(rng, lens, page, hk, dim, garbage=True):
    """Pages holding Gaussian keys and values; whatever no token fills is
    random bytes, NaN scales among them."""
    need = [-(-int(x) // page) for x in lens]
    n_pages = sum(need) + 2
    ids = rng.permutation(n_pages)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int64)
    at = 0
    pages = rng.integers(0, 256, (n_pages, hk, page * dim * 17 // 16)).astype(np.uint8)
    for b, m in enumerate(need):
        table[b, :m] = ids[at:at + m]
        at += m
    k = [rng.standard_normal((int(x), hk, dim)) * (1 + 2 * (rng.random((1, hk, dim)) > 0.95))
         for x in lens]
    v = [rng.standard_normal((int(x), hk, dim)) for x in lens]
    where = [(b, j) for b, x in enumerate(lens) for j in range(int(x))]
    if where:
        pages = so.put(pages, table, where, np.concatenate(k), np.concatenate(v))
    return pages, table


# The bounds size the launch, and with it choose the kernel: under large ones
# bf16 rows with heads of 64 and 128 go to the many-row kernel whatever there
# is of them, the first in few parts, the second in many (some of them empty),
# the third under a window too.
MANY = [dict(max_new=4096, max_kv=1 << 16), dict(max_new=200, max_kv=1 << 22),
        dict(max_new=1 << 20, max_kv=1 << 16)]


def check(ttt, dtype, page, hk, hq, dim, news, lens, *, q=None, seed=0, **kw):
    rng = np.random.default_rng(seed)
    if kw.get("pages") is None:
        kw["pages"], kw["table"] = pool_of(rng, lens, page, hk, dim)
    if q is None:
        q = torch.from_numpy(kw.pop("sharp", 1.5) * rng.standard_normal((sum(news), hq, dim))).to(dtype).cuda()
    refs = {}
    o = check_one(ttt, dtype, page, hk, hq, dim, news, lens, q, refs, **kw)
    if dtype == BF and dim <= 128 and "max_new" not in kw:
        for bounds in MANY:
            check_one(ttt, dtype, page, hk, hq, dim, news, lens, q, refs, **kw, **bounds)
    return o


def check_one(ttt, dtype, page, hk, hq, dim, news, lens, q, refs, *, window=0, causal=True,
              pages=None, table=None, no_starts=False, **kw):
    starts = np.concatenate([[0], np.cumsum(news)])
    scale = dim ** -0.5
    o, lse = ttt.kv_attention(q, torch.from_numpy(pages).cuda(), ints(table), ints(lens),
                              q_starts=None if no_starts else ints(starts), window=window,
                              causal=causal, with_lse=True, **kw)
    torch.cuda.synchronize()
    assert o.dtype == dtype and o.shape == q.shape
    o, lse, qh = host(o), host(lse), host(q)
    for b, (m, length) in enumerate(zip(news, lens)):
        r = slice(starts[b], starts[b + 1])
        if b not in refs:
            k, v, have = so.gather(pages, table, b, int(length), dim)
            refs[b] = (k, *so.attend(qh[r], k, v, have, int(length), scale, window, causal))
        k, ref, lref, w = refs[b]
        ks = np.abs(np.nan_to_num(k)).repeat(hq // hk, 1)
        terms = scale * np.einsum("thd,jhd->thj", np.abs(qh[r]), ks).max(-1) if length else 0.0
        rel = (4 * np.sqrt(dim) * 2 ** -24 * terms + 2 ** -21 + 4 * np.sqrt(max(length, 1)) * 2 ** -24)
        rel = np.broadcast_to(rel, lref.shape)
        tol = (rel[..., None] + (2 ** -8 if dtype == BF else 2 ** -23)) * w
        tol = tol + (2 ** -8 * 1.01 if dtype == BF else 2 ** -23) * np.abs(ref) + 1e-30
        assert np.array_equal(np.isnan(o[r]), np.isnan(ref)), b
        err = np.abs(o[r] - ref)
        assert not (err > tol).any(), (b, float(np.nanmax(err / tol)), np.argwhere(err > tol)[:3])
        empty = np.isneginf(lref)
        assert np.array_equal(np.isneginf(lse[r]), empty)
        assert not o[r][empty].any()
        d = np.abs(lse[r] - lref)[~empty & ~np.isnan(lref)]
        room = (rel + 2 ** -22 * (1 + np.abs(lref)))[~empty & ~np.isnan(lref)]
        assert (d <= room).all(), (b, float((d / room).max()))
    return o


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 300]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_single_tokens_of_every_length(ttt, dtype, dim):
    check(ttt, dtype, 32, 2, 8, dim, [1] * len(LENGTHS), LENGTHS, no_starts=True)


@pytest.mark.parametrize("page", [16, 48, 64, 112, 256])
@pytest.mark.parametrize("hk,hq", [(1, 1), (2, 2), (1, 5), (2, 32), (1, 17), (4, 8)])
def test_head_layouts_and_pages(ttt, page, hk, hq):
    check(ttt, BF, page, hk, hq, 128, [1, 3, 1], [200, 77, 513], seed=page + hq)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim,hk,hq", [(64, 2, 4), (128, 1, 4), (128, 2, 10), (256, 1, 3)])
@pytest.mark.parametrize("news,lens", [
    ([5], [5]), ([64], [64]), ([65, 1, 130], [65, 100, 260]), ([100, 33], [333, 33]),
    ([257], [700])])
def test_segments(ttt, dtype, dim, hk, hq, news, lens):
    check(ttt, dtype, 48, hk, hq, dim, news, lens, seed=dim + sum(news))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 5000])
def test_windows(ttt, dtype, window):
    check(ttt, dtype, 32, 2, 8, 128, [70, 1, 1, 9], [300, 300, 40, 9], window=window, seed=window)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_all_keys(ttt, dtype):
    check(ttt, dtype, 32, 2, 4, 64, [70, 1, 9], [300, 40, 9], causal=False)
    check(ttt, dtype, 32, 2, 4, 128, [130, 3], [130, 300], causal=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_see_nothing(ttt, dtype, dim):
    """No keys, fewer keys than rows, no rows, and rows whose pages are gone."""
    check(ttt, dtype, 16, 2, 4, dim, [3, 20, 0, 1, 40], [0, 7, 50, 1, 3], seed=3)
    rng = np.random.default_rng(4)
    pages, table = pool_of(rng, [100, 200], 32, 2, dim)
    table[0, :] = -1                   # the whole sequence
    table[1, :5] = [-1, 99, -1, -1, -7]   # everything but the last 40 tokens
    check(ttt, dtype, 32, 2, 4, dim, [50, 70], [100, 200], pages=pages, table=table)
    check(ttt, dtype, 32, 2, 4, dim, [1, 1], [100, 200], pages=pages, table=table, window=64)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news,where", [([1], [70]), ([40], [170, 185]), ([200], [3, 100, 199])])
def test_nan_reaches_only_the_rows_that_see_it(ttt, dtype, dim, news, where):
    length = 200
    for part in ("k", "v"):
        rng = np.random.default_rng(5)
        pages, table = pool_of(rng, [length], 16, 1, dim)
        k, v = (rng.standard_normal((length, 1, dim)) for _ in range(2))
        for j in where:
            (k if part == "k" else v)[j, 0, dim // 2] = np.nan
        pages = so.put(pages, table, [(0, j) for j in range(length)], k, v)
        o = check(ttt, dtype, 16, 1, 4, dim, news, [length], pages=pages, table=table)
        first = min(where)
        seen = np.arange(length - news[0], length) >= first
        assert np.isnan(o[seen]).all() and np.isfinite(o[~seen]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_caches_and_sharp_rows(ttt, dtype):
    """Long enough to be split over many workgroups; rows that all but pick
    one key, and rows over scores of hundreds."""
    check(ttt, dtype, 64, 1, 4, 128, [1], [9001], seed=1)
    check(ttt, dtype, 64, 1, 4, 128, [3], [2500], seed=2, sharp=30.0)
    check(ttt, dtype, 64, 2, 4, 64, [1, 1], [4097, 5], seed=3, sharp=300.0)


def test_bounds_are_hints(ttt):
    """max_new and max_kv size the launch; wrong ones change no result."""
    rng = np.random.default_rng(6)
    pages, table = pool_of(rng, [3000, 40], 64, 2, 128)
    for dtype in (BF, F32):
        for kw in (dict(max_new=1, max_kv=1), dict(max_new=64, max_kv=64), dict(max_new=9999, max_kv=10 ** 8),
                   dict(max_new=1, max_kv=10 ** 8)):
            check(ttt, dtype, 64, 2, 8, 128, [37, 5], [3000, 40], pages=pages, table=table, **kw)
    # one small workgroup of rows for all of them
    check(ttt, BF, 64, 2, 8, 128, [300], [3000], max_new=33, max_kv=1 << 22)


def test_strided_rows_other_streams_and_outputs(ttt):
    rng = np.random.default_rng(7)
    pages, table = pool_of(rng, [500, 61], 64, 2, 128)
    x = torch.from_numpy(rng.standard_normal((50, 12, 128))).to(BF).cuda()
    q = x[:, :8]
    ref = check(ttt, BF, 64, 2, 8, 128, [45, 5], [500, 61], pages=pages, table=table, q=q)
    p, t, n, st = torch.from_numpy(pages).cuda(), ints(table), ints([500, 61]), ints([0, 45, 50])
    out = torch.full((8, 50, 128), 7.0, dtype=BF, device="cuda")     # head-major
    ws = torch.empty(ttt.kv_attention_workspace_size(2, 50, 2, 8, 128, max_new=50, max_kv=t.shape[1] * 64),
                     dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ttt.kv_attention(q, p, t, n, q_starts=st, out=out.transpose(0, 1), workspace=ws, stream=s)
    s.synchronize()
    assert np.array_equal(host(got), ref)
    e = ttt.kv_attention(q[:0], p, t, n, q_starts=ints([0, 0, 0]))
    assert e.shape == (0, 8, 128)


def test_captured_step_follows_the_lengths(ttt):
    """Append and attention of one token in a graph: each replay reads the
    lengths, pages and rows as they are then."""
    hk, hq, dim, page = 2, 8, 128, 16
    rng = np.random.default_rng(8)
    pages = ttt.kv_pages(9, page, hk, dim)
    table = ints([[4, 2, 7, 0], [1, 8, 3, 5]])
    rope = ttt.rope_table(64, dim, 1e4)
    xs = torch.from_numpy(rng.standard_normal((40, 2, hq + 2 * hk, dim))).to(BF).cuda()
    x, lens = xs[0].clone(), ints([1, 3])
    ws = torch.empty(max(1, ttt.kv_attention_workspace_size(2, 2, hk, hq, dim, max_new=1, max_kv=64)),
                     dtype=torch.uint8, device="cuda")
    q, o = torch.empty((2, 2, hq, dim), dtype=BF, device="cuda")

    def step(pool):
        ttt.kv_append(pool, table, lens, x[:, hq:hq + hk], x[:, hq + hk:], q=x[:, :hq],
                      rope_table=rope, q_out=q)
        ttt.kv_attention(q, pool, table, lens, max_kv=64, out=o, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(pages)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(pages)
    pages.zero_()
    eager = ttt.kv_pages(9, page, hk, dim)
    for t in range(40):
        x.copy_(xs[t])
        lens.copy_(ints([t + 1, t + 3]))
        g.replay()
        torch.cuda.synchronize()
        got = o.clone()
        o.zero_()
        step(eager)
        torch.cuda.synchronize()
        assert torch.equal(got, o), t
        assert torch.equal(pages, eager), t


@pytest.mark.parametrize("dim", [64, 128])
def test_many_rows_over_long_caches(ttt, dim):
    """Rows and keys enough for the many-row kernel by themselves, whole and in
    parts: page tables longer than the 64 tiles it looks up at once."""
    check(ttt, BF, 16, 1, 2, dim, [66, 70], [4700, 9000], window=0, max_new=70, max_kv=1 << 22)
    check(ttt, BF, 256, 1, 2, dim, [66], [9000], window=5000, max_new=4096, max_kv=1 << 13)


def test_negative_and_zero_scales(ttt):
    """A scale of either sign, and none: the maximum is followed unscaled."""
    rng = np.random.default_rng(9)
    pages, table = pool_of(rng, [300], 32, 2, 128)
    q = torch.from_numpy(rng.standard_normal((20, 4, 128)))
    k, v, have = so.gather(pages, table, 0, 300, 128)
    for dtype in (BF, F32):
        x = q.to(dtype).cuda()
        for scale in (-0.1, 0.0, 1e-30):
            ref, lref, w = so.attend(host(x), k, v, have, 300, scale)
            for kw in ({}, *MANY):
                o, lse = ttt.kv_attention(x, torch.from_numpy(pages).cuda(), ints(table), ints([300]),
                                          scale=scale, with_lse=True, **kw)
                u = 2 ** -7 if dtype == BF else 2 ** -17
                assert (np.abs(host(o) - ref) <= u * (w + np.abs(ref))).all()
                assert (np.abs(host(lse) - lref) <= 2 ** -17 * (1 + np.abs(lref))).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 100])
def test_slices_over_ragged_sequences(ttt, dtype, dim, window):
    """Up to 16 rows a sequence and a long bound: even slices of all keys.
    Slices of many sequences, some of them without rows or keys; slices of one
    long one between short ones; and more rows than the bound said."""
    rng = np.random.default_rng(14)
    news, lens = rng.integers(0, 9, 120), rng.integers(0, 300, 120)
    lens[::7], news[3:9], news[-2:] = 0, 0, 0
    check(ttt, dtype, 16, 8, 16, dim, list(news), list(lens), window=window, max_new=8, max_kv=1 << 16, seed=1)
    lens = [3, 0, 2500, 1, 129, 700, 0]
    check(ttt, dtype, 64, 2, 6, dim, [1] * 7, lens, window=window, max_new=1, max_kv=8192, no_starts=True, seed=2)
    check(ttt, dtype, 64, 2, 6, dim, [1, 0, 40, 1, 0, 7, 3], lens, window=window, max_new=1, max_kv=8192, seed=3)


@pytest.mark.parametrize("batch", [64, 65, 256, 257])
def test_slices_by_batch(ttt, batch):
    lens = 1 + np.arange(batch) * 37 % 301
    check(ttt, BF, 32, 1, 4, 128, [1] * batch, list(lens), max_new=1, max_kv=4096, no_starts=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_before_the_first_token_under_the_widest_window(ttt, dtype):
    """More rows than tokens: the first stand before the sequence and see
    nothing, whatever the window; the others see all before them."""
    for window in (2 ** 31 - 1, 2 ** 31 - 3):
        check(ttt, dtype, 32, 2, 8, 128, [8, 300], [5, 200], window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_longest_sequence(ttt, dtype):
    """2^30 tokens: its last ones give what they give at the end of 8192."""
    page, dim = 4096, 64
    rng = np.random.default_rng(12)
    longest = (1 << 30) // page
    pool = ttt.kv_pages(3, page, 1, dim)
    table = torch.full((2, longest), -1, dtype=torch.int32, device="cuda")
    table[0, :2] = table[1, -2:] = ints([2, 1])
    short, far = (ints([x]) for x in (8192, 1 << 30))
    x = torch.from_numpy(rng.standard_normal((300, 3, dim))).to(dtype).cuda()
    read = []
    for t, lens in ((table[:1], short), (table[1:], far)):
        pool.zero_()
        ttt.kv_append(pool, t, lens, x[:, 1:2], x[:, 2:])
        read.append((pool.clone(), *ttt.kv_read(pool, t, lens, 300, dim, dtype)))
    assert all(torch.equal(a, b) for a, b in zip(*read)) and read[0][1].any()
    for rows in (1, 300):
        for kw in ({}, MANY[0], dict(max_new=1 << 20)):
            got = [ttt.kv_attention(x[:rows, :1].expand(rows, 4, dim).contiguous(), pool, t, lens, window=100,
                                    with_lse=True, **kw) for t, lens in ((table[:1], short), (table[1:], far))]
            assert all(torch.equal(a, b) for a, b in zip(*got)), (rows, kw)
            assert torch.isfinite(got[0][1]).all()


def test_more_workgroups_than_a_dimension_holds(ttt):
    """65535 sequences of 256 key heads, the last four of them with a row."""
    rng = np.random.default_rng(13)
    batch, heads, dim = 65535, 256, 64
    pool = torch.from_numpy(pool_of(rng, [16], 16, heads, dim, garbage=False)[0]).cuda()
    table = torch.full((batch, 1), -1, dtype=torch.int32, device="cuda")
    table[-4:] = ints([[0], [2], [1], [0]])
    lens, starts = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    lens[-4:], starts[-4:] = ints([3, 9, 16, 1]), ints([1, 2, 3, 4])
    q = torch.from_numpy(rng.standard_normal((4, heads, dim))).to(BF).cuda()
    last = (table[-4:].contiguous(), lens[-4:].contiguous(), starts[-5:].contiguous())
    for max_new in (1, 1 << 24):     # either kernel
        few = ttt.kv_attention(q, pool, *last[:2], q_starts=last[2], max_new=max_new, max_kv=16)
        got = ttt.kv_attention(q, pool, table, lens, q_starts=starts, max_new=max_new, max_kv=16)
        torch.cuda.synchronize()
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(few)) and got.any()


def test_outputs_live_on_the_stream_of_the_call(ttt):
    """Memory taken for a call on another stream is that stream's, so that
    nothing else is given it while the kernels there are under way."""
    def owner(t):
        return [s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
    s = torch.cuda.Stream()
    table, lens = ints([[0], [1]]), ints([9, 9])
    pool, rope = ttt.kv_pages(2, 64, 2, 64), ttt.rope_table(64, 64)
    x = torch.ones((18, 2, 64), dtype=BF, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    q = ttt.kv_append(pool, table, lens, x, x, q=x, rope_table=rope, stream=s)
    o, lse = ttt.kv_attention(q, pool, table, lens, max_kv=1 << 16, with_lse=True, stream=s)
    made = [q, o, lse, *ttt.kv_read(pool, table, lens, 18, 64, stream=s),
            *ttt.rope_forward(x, x, rope, stream=s), ttt.rope_table(64, 64, stream=s)]
    s.synchronize()
    assert all(owner(t) == [s.cuda_stream] for t in made)
    assert torch.equal(o[::9], x[::9])     # every row's values are ones, which the cache holds exactly


@pytest.mark.parametrize("dtype,hk,hq,dim", [(BF, 1, 3, 256), (F32, 2, 4, 64), (F32, 1, 2, 128), (F32, 1, 2, 256)])
def test_tiles_enough_for_every_wave(ttt, dtype, hk, hq, dim):
    """So many sequences that each wave has rows of its own (short keys, so
    that they are not split): prompts, a window, rows without keys."""
    rng = np.random.default_rng(15)
    batch, new = 70, 40
    news = rng.integers(0, new + 1, batch)
    lens = news + rng.integers(-2, 30, batch).clip(-news, None)
    lens[5] = 0
    # max_new is a bound: tiles of rows that are not there make up the number
    for window in (0, 7):
        check(ttt, dtype, 16, hk, hq, dim, list(news), list(lens), window=window, max_new=1 << 12, max_kv=128, seed=4)
