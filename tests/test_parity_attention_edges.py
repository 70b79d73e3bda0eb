"""GPU parity of attention over the paged 4-bit cache where sequences, pages
and launches end: the checks and tolerances of test_parity_attention."""
import numpy as np
import pytest
import torch

import oracle.serve_oracle as so
from test_parity_attention import check, host, ints, pool_of, ttt  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SLICES = dict(max_new=1, max_kv=1 << 16)     # several sequences: cut into slices of all their keys


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(), dict(window=20), dict(causal=False)], ids=["causal", "window", "all"])
def test_sequences_longer_than_their_page_table(ttt, dtype, dim, kw):
    """Rows stand where kv_lens says, as they do for append; what the table
    has no entry for is seen by none of them."""
    rng = np.random.default_rng(21)
    lens = [200, 70, 45, 51]
    pages, table = pool_of(rng, lens, 16, 2, dim)
    table = table[:, :3]      # 48 tokens each
    for news in ([170, 30, 5, 6], [1, 1, 1, 1], [3, 23, 1, 4]):
        check(ttt, dtype, 16, 2, 4, dim, news, lens, pages=pages, table=table, **kw)
        check(ttt, dtype, 16, 2, 4, dim, news, lens, pages=pages, table=table, **kw, **SLICES)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths_at_the_ends_of_32_bits(ttt, dtype):
    rng = np.random.default_rng(22)
    pages, table = pool_of(rng, [48], 16, 2, 128)
    p, t = torch.from_numpy(pages).cuda(), ints(table)
    q = torch.from_numpy(rng.standard_normal((20, 4, 128))).to(dtype).cuda()
    for kw in (dict(), dict(max_new=4096, max_kv=1 << 16), dict(max_new=200, max_kv=1 << 22)):
        ref = ttt.kv_attention(q, p, t, ints([48]), causal=False, with_lse=True, **kw)
        got = ttt.kv_attention(q, p, t, ints([2 ** 31 - 1]), with_lse=True, **kw)
        assert all(torch.equal(a, b) for a, b in zip(ref, got)) and torch.isfinite(got[1]).all()
        for length, opt in ((2 ** 31 - 1, dict(window=9)), (-1, dict()), (-2 ** 31, dict()), (-2 ** 31, dict(window=9)),
                            (-2 ** 31, dict(causal=False))):
            o, lse = ttt.kv_attention(q, p, t, ints([length]), with_lse=True, **opt, **kw)
            assert not o.any() and torch.isneginf(lse).all(), (length, opt, kw)


def spoil(pages, table, page, dim, part, where):
    """NaN scales at (token, key head, block): only there."""
    pages = pages.copy()
    for n, (j, h, c) in enumerate(where):
        at = so.page_offsets(page, dim, j % page)[2 if part == "k" else 3][c]
        pages[table[0, j // page], h, at] = 253 + n % 3
    return pages


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news", [1, 30, 200])
def test_nan_scales_of_single_blocks(ttt, dtype, dim, news):
    """A scale above 252 is its block's: of K the rows that see it are NaN, of
    V those values of theirs, whichever kernel takes them."""
    length, page = 200, 16
    pages, table = pool_of(np.random.default_rng(23), [length], page, 2, dim)
    first = max(length - news, 0)
    q = torch.from_numpy(1.5 * np.random.default_rng(24).standard_normal((news, 8, dim))).to(dtype).cuda()
    for part in ("k", "v"):
        for c in range(dim // 32):
            where = [(first + news // 2, 0, c), (3, 1, c), (length - 1, 1, (c + 1) % (dim // 32))]
            bad = spoil(pages, table, page, dim, part, where)
            o = check(ttt, dtype, page, 2, 8, dim, [news], [length], q=q, pages=bad, table=table)
            _, lse = ttt.kv_attention(q, torch.from_numpy(bad).cuda(), ints(table), ints([length]), with_lse=True)
            nan = np.isnan(o)
            if part == "k":      # whole rows
                assert (nan.any(-1) == nan.all(-1)).all() and np.array_equal(np.isnan(host(lse)), nan.any(-1))
            else:                # the block of every row from there on, of the head's four
                want = np.zeros_like(nan)
                for j, h, b in where:
                    want[max(0, j - first):, 4 * h:4 * h + 4, 32 * b:32 * b + 32] = True
                assert np.array_equal(nan, want) and torch.isfinite(lse).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hk,hq,new", [(1, 1, 1), (2, 8, 1), (1, 4, 2), (1, 9, 1), (2, 10, 3), (1, 16, 1)])
@pytest.mark.parametrize("lens", [[777], [1024], [1025], [60, 300, 1500]])
def test_up_to_16_rows_keep_16_bits_of_the_weights(ttt, dim, hk, hq, new, lens):
    """Under any max_kv. Two bf16 terms leave 2^-16 of a weight; the rest is the
    tolerance of test_parity_attention, without one term's 2^-8."""
    rng = np.random.default_rng(25)
    page, scale = 64, dim ** -0.5
    pages, table = pool_of(rng, lens, page, hk, dim)
    q = torch.from_numpy(1.5 * rng.standard_normal((new * len(lens), hq, dim))).to(BF).cuda()
    refs = []
    for b, n in enumerate(lens):
        k, v, have = so.gather(pages, table, b, n, dim)
        qh = host(q[b * new:(b + 1) * new])
        ref, _, w = so.attend(qh, k, v, have, n, scale)
        terms = scale * np.einsum("thd,jhd->thj", np.abs(qh), np.abs(k).repeat(hq // hk, 1)).max(-1)
        rel = 4 * np.sqrt(dim) * 2 ** -24 * terms + 2 ** -21 + 4 * np.sqrt(n) * 2 ** -24 + 2 ** -16
        refs.append((ref, rel[..., None] * w + 2 ** -8 * np.abs(ref)))
    ref, tol = (np.concatenate(x) for x in zip(*refs))
    for max_kv in (max(lens), 1024, 1025, 1 << 17):
        o = ttt.kv_attention(q, torch.from_numpy(pages).cuda(), ints(table), ints(lens), max_kv=max_kv)
        err = np.abs(host(o) - ref)
        assert (err <= tol).all(), (max_kv, float((err / tol).max()), int((err > tol).sum()))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,new,length,kw", [
    (16, 200, 9000, dict()), (48, 131, 9001, dict(window=5000)), (16, 70, 13000, dict(window=8500)),
    (112, 130, 8500, dict(causal=False)), (64, 300, 700, dict(window=65))])
def test_many_rows_in_parts(ttt, dim, page, new, length, kw):
    """The many-row kernel with each sequence's keys in two parts: of more than
    the 64 tiles whose pages it looks up at once, of fewer, and of windows that
    begin within a tile; rows for more than one wave."""
    kw = dict(kw, max_new=1 << 14, max_kv=1 << 16)
    plan = ttt.kv_attention_plan(1, new, 1, 2, dim, max_new=1 << 14, max_kv=1 << 16, window=kw.get("window", 0))
    assert plan["many"] and (plan["parts"] == 2 or kw.get("window") == 65), plan
    check(ttt, BF, page, 1, 2, dim, [new], [length], seed=length, **kw)


@pytest.mark.parametrize("dim", [64, 128])
def test_many_rows_whole_and_ragged(ttt, dim):
    """The same kernel over one part, several sequences and key heads."""
    plan = ttt.kv_attention_plan(3, 340, 2, 8, dim, max_new=1 << 14, max_kv=1 << 16)
    assert plan["many"] and plan["parts"] == 1, plan
    for kw in (dict(), dict(window=100), dict(causal=False)):
        check(ttt, BF, 48, 2, 8, dim, [150, 1, 189], [4700, 300, 189], seed=31, max_new=1 << 14, max_kv=1 << 16, **kw)
