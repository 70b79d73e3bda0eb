"""GPU parity of the paged 4-bit cache: every byte that ttt_kv_append writes
(and every one it must leave alone) against the oracle's, and ttt_kv_read
against what the bytes stand for. All comparisons are exact: the rotation is
defined to the bit in float32, and the codes are defined from it."""
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
    return t.detach().float().cpu().numpy()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def bf16_np(x):
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(BF).float().numpy()


def case(ttt, dtype, page, hk, hq, dim, rot, inter, news, before, seed, positions=False, wide=False,
         no_starts=False):
    rng = np.random.default_rng(seed)
    n, batch = sum(news), len(news)
    lens = np.array(before) + news
    need = [-(-int(x) // page) for x in lens]
    n_pages = sum(need) + 2
    ids = rng.permutation(n_pages)
    table = np.full((batch, max(need) + 1), -1, np.int64)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = ids[at:at + m]
        at += m
    starts = np.concatenate([[0], np.cumsum(news)])
    x = rng.standard_normal((n, hq + 2 * hk, dim)).astype(np.float32)
    if wide:  # values over the whole range of the type, zeros, and non-finite ones
        x *= 2.0 ** rng.integers(-140, 127, (n, hq + 2 * hk, dim // 32, 1)).repeat(32, -1).reshape(x.shape)
        x[rng.random(x.shape[:2]) < 0.1] = 0.0
        x[rng.random(x.shape[:2]) < 0.05, 3] = np.nan
        x[rng.random(x.shape[:2]) < 0.05, dim - 1] = -np.inf
    x = torch.from_numpy(x).to(dtype).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    old = rng.integers(0, 256, (n_pages, hk, page * dim * 17 // 16)).astype(np.uint8)
    pages = torch.from_numpy(old).cuda()
    where = so.owners(n, batch, lens, starts)
    rope = ttt.rope_table(int(lens.max()) + 3, rot, 1e4) if rot else None
    pos = rng.integers(0, int(lens.max()) + 3, n) if positions else np.array([i for _, i in where])
    kw = dict(q_starts=None if no_starts else ints(starts))
    y = ttt.kv_append(pages, ints(table), ints(lens), k, v, q=q if rot else None, rope_table=rope,
                      interleaved=inter, positions=ints(pos) if positions else None, **kw)
    torch.cuda.synchronize()
    kr = host(k)
    if rot:
        cs = host(rope)[pos]
        with np.errstate(invalid="ignore", over="ignore"):
            kr = so.rotate32(kr, cs, inter)
            qr = so.rotate32(host(q), cs, inter)
        want = bf16_np(qr) if dtype == BF else qr
        assert np.array_equal(host(y), want, equal_nan=True)
    want = so.put(old, table, where, kr, host(v))
    got = pages.cpu().numpy()
    bad = np.argwhere(got != want)
    assert not len(bad), (len(bad), bad[:4], got[tuple(bad[0])], want[tuple(bad[0])])
    for rt in (BF, F32):
        ko, vo = ttt.kv_read(pages, ints(table), ints(lens), n, dim, rt, **kw)
        for m, (b, idx) in enumerate(where):
            kv = so.get(want, table, b, idx, dim)
            assert np.array_equal(host(ko[m]), kv[0], equal_nan=True)
            assert np.array_equal(host(vo[m]), kv[1], equal_nan=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page,hk,hq,dim,rot,inter,news,before", [
    (16, 1, 1, 64, 64, False, [1], [0]),
    (16, 2, 4, 64, 32, True, [5, 1, 18], [0, 15, 16]),
    (64, 8, 8, 128, 128, False, [1, 1, 1, 1], [63, 64, 0, 200]),
    (48, 1, 5, 128, 64, True, [33, 0, 50], [40, 7, 0]),
    (32, 2, 2, 256, 256, False, [7, 29], [30, 1]),
    (256, 3, 3, 256, 48, True, [13], [250]),
    (112, 2, 2, 128, 0, False, [9, 4], [110, 0]),
])
def test_append_and_read(ttt, dtype, page, hk, hq, dim, rot, inter, news, before):
    case(ttt, dtype, page, hk, hq, dim, rot, inter, news, before, 7)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_whole_range_of_values(ttt, dtype, dim):
    """Subnormals to the type's largest, zero blocks, NaN and infinities."""
    case(ttt, dtype, 32, 2, 2, dim, 0, False, [61, 8], [3, 0], 8, wide=True)


def test_every_rounding_boundary(ttt):
    """The hardware's conversion at, just below and just above every tie and
    saturation point, for both signs and several scales."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0], np.float32)
    near = np.concatenate([ties, np.nextafter(ties, np.float32(9)), np.nextafter(ties, np.float32(-9))])
    near = near[near <= 7]
    rows = []
    for e in (-125, -120, -7, 0, 5, 125):
        for s in (1, -1):
            b = np.zeros(32, np.float32)
            b[:len(near)] = s * near
            b[31] = 7.0 if e < 125 else 6.0
            rows.append((b.astype(np.float64) * 2.0 ** e).astype(np.float32))
    x = np.stack(rows).reshape(len(rows) // 2, 1, 64)
    n = x.shape[0]
    pages = ttt.kv_pages(1, 16, 1, 64)
    t = torch.from_numpy(x).cuda()
    ttt.kv_append(pages, ints([[0]]), ints([n]), t, t)
    k, v = ttt.kv_read(pages, ints([[0]]), ints([n]), n, 64, F32)
    want = so.decode(*so.encode(x))
    assert np.array_equal(host(k), want.astype(np.float32)) and torch.equal(k, v)


def test_positions_and_even_batches(ttt):
    case(ttt, BF, 32, 2, 4, 128, 128, False, [3, 3], [10, 40], 9, positions=True)
    case(ttt, BF, 32, 2, 4, 128, 128, False, [1, 1, 1], [10, 40, 31], 10, no_starts=True)


def test_tokens_without_a_page_are_not_written(ttt):
    """Pages of -1 and past the pool, indices past the table or below zero,
    rows of no sequence: nothing is written, and reading gives zero."""
    x = torch.randn(6, 1, 64, device="cuda")
    for table, lens, starts, none in (
            ([[0, -1]], [18], [0, 6], [4, 5]),       # tokens 12 .. 17, the second page is none
            ([[0, 9]], [18], [0, 6], [4, 5]),        # a page past the pool
            ([[0]], [18], [0, 6], [4, 5]),           # past the table
            ([[0]], [4], [0, 6], [0, 1]),            # indices -2 and -1
            ([[0]], [3], [1, 4], [0, 4, 5])):        # rows 0, 4 and 5 of no sequence
        pages = ttt.kv_pages(2, 16, 1, 64)
        pages.fill_(85)
        ttt.kv_append(pages, ints(table), ints(lens), x, x, q_starts=ints(starts))
        k, _ = ttt.kv_read(pages, ints(table), ints(lens), 6, 64, F32, q_starts=ints(starts))
        want = so.put(np.full((2, 1, 16 * 68), 85, np.uint8), np.array(table),
                      so.owners(6, 1, lens, starts), host(x), host(x))
        assert np.array_equal(pages.cpu().numpy(), want)
        held = so.decode(*so.encode(host(x))).astype(np.float32)
        held[none] = 0
        assert np.array_equal(host(k), held)


def test_large_pools_and_strides(ttt):
    """A pool of several layers side by side, over 2^32 bytes: page offsets
    pass 32 bits."""
    page, hk, dim, n_pages = 256, 8, 128, 2200
    layers = torch.zeros((n_pages, 8, hk, page * 136), dtype=torch.uint8, device="cuda")
    assert layers.numel() > 2 ** 32
    x = torch.randn(300, 3 * hk, dim, device="cuda").to(BF)
    tables = ints([[n_pages - 1, 0]])
    for layer in (0, 7):
        pages = layers[:, layer]
        ttt.kv_append(pages, tables, ints([300]), x[:, :hk], x[:, hk:2 * hk])
        k, v = ttt.kv_read(pages, tables, ints([300]), 300, dim, BF)
        assert np.array_equal(host(k), so.decode(*so.encode(host(x[:, :hk]))))
        assert np.array_equal(host(v), so.decode(*so.encode(host(x[:, hk:2 * hk]))))
    assert not layers[:, 1:7].any() and not layers[1:-1].any()
    out = ttt.kv_attention(x[-1:, 2 * hk:], layers[:, 7], tables, ints([300]))
    k, v = (so.decode(*so.encode(host(x[:, a:a + hk]))) for a in (0, hk))
    ref, _, w = so.attend(host(x[-1:, 2 * hk:]).astype(np.float64), k, v, np.ones(300, bool), 300,
                          dim ** -0.5)
    assert (np.abs(host(out) - ref) <= 2 ** -8 * w + 2 ** -8 * np.abs(ref)).all()
