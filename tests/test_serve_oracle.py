"""CPU-only: the oracle of the attention half of a block pinned to closed
forms, and shown to notice planted mistakes."""
import numpy as np
import pytest

import oracle.serve_oracle as so


def test_rotation_is_relative():
    """<R(p) q, R(j) k> depends on p - j alone; norms stay."""
    rng = np.random.default_rng(0)
    cs = so.table(64, 32)
    q, k = rng.standard_normal((2, 1, 1, 48))
    for inter in (False, True):
        def dot(p, j):
            return float((so.rotate(q, cs[[p]], inter) * so.rotate(k, cs[[j]], inter)).sum())
        assert abs(dot(7, 3) - dot(47, 43)) < 1e-12
        assert abs(dot(7, 3) - dot(7, 4)) > 1e-6
        y = so.rotate(q, cs[[9]], inter)
        assert abs((y ** 2).sum() - (q ** 2).sum()) < 1e-12
        back = so.rotate(y, cs[[9]], inter, transposed=True)
        assert np.abs(back - q).max() < 1e-14


def test_layouts_pair_different_values():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((1, 1, 32))
    cs = so.table(8, 32)
    half, inter = so.rotate(q, cs[[5]], False), so.rotate(q, cs[[5]], True)
    assert np.abs(half - inter).max() > 1e-2
    # one is the other under the layouts' permutation
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    assert np.allclose(so.rotate(q[..., perm], cs[[5]], False), inter[..., perm], atol=1e-15)


@pytest.mark.parametrize("kind,kw", [("linear", {}), ("base", {}),
                                     ("yarn", dict(original=4096, low=1, high=32)),
                                     ("bands", dict(original=8192, low=1, high=4))])
def test_scalings_keep_the_fast_end_and_stretch_the_slow(kind, kw):
    w = so.angle_steps(128, 5e5)
    s = so.angle_steps(128, 5e5, kind, factor=8.0, **kw)
    assert abs(s[-1] / (w[-1] / 8) - 1) < 1e-12
    assert abs(s[0] / (w[0] / 8 if kind == "linear" else w[0]) - 1) < 1e-12
    assert (np.diff(s) < 0).all()


def test_codes_hold_the_grid_and_round_to_nearest_even():
    x = np.zeros(32)
    x[:8], x[8:16] = so.GRID, -so.GRID
    for e in (-125, -3, 0, 9, 125):
        c, s = so.encode(x * 2.0 ** e)
        assert s[0] == e + 127 and np.array_equal(so.decode(c, s), x * 2.0 ** e)
    ties = {0.25: 0, 0.75: 1, 1.25: 1, 1.75: 2, 2.5: 2, 3.5: 4, 5.0: 4, 6.9: 6}
    for v, want in ties.items():
        x = np.full(32, v)
        x[0] = 6.0
        c, s = so.encode(x)
        assert so.decode(c, s)[1] == want, v
    assert so.encode(np.full(32, 7.01))[1] == 128      # 7 is the limit
    assert so.encode(np.full(32, 7.0))[1] == 127


def test_non_finite_values_take_the_head():
    x = np.ones((2, 64))
    x[1, 40] = np.inf
    v = so.decode(*so.encode(x))
    assert np.isfinite(v[0]).all() and np.isnan(v[1]).all()


def test_page_bytes_are_disjoint_and_complete():
    for page, dim in ((16, 64), (48, 128), (32, 256)):
        seen = np.concatenate([np.concatenate(so.page_offsets(page, dim, t)) for t in range(page)])
        assert np.array_equal(np.sort(seen), np.arange(page * (dim + dim // 16)))


def test_put_get_round_trip():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 21, 2, 64))
    table = np.array([[3, 1], [0, -1]])
    starts, lens = np.array([0, 19, 21]), np.array([20, 18])
    where = so.owners(21, 2, lens, starts)
    pages = so.put(np.zeros((4, 2, 16 * 68), np.uint8), table, where, k, v)
    for n, (b, idx) in enumerate(where):
        kv = so.get(pages, table, b, idx, 64)
        if b == 1:          # tokens 16, 17 of a sequence whose second page is none
            assert idx >= 16 and kv is None
            continue
        assert np.array_equal(kv[0], so.decode(*so.encode(k[n])))
        assert np.array_equal(kv[1], so.decode(*so.encode(v[n])))


def test_attention_against_one_key_and_uniform_keys():
    rng = np.random.default_rng(3)
    q = rng.standard_normal((3, 2, 64))
    v = rng.standard_normal((3, 1, 64))
    have = np.ones(3, bool)
    o, lse, _ = so.attend(q, np.zeros((3, 1, 64)), v, have, 3, 0.125)
    for t in range(3):                           # equal scores: the mean of what is seen
        assert np.allclose(o[t], v[:t + 1, 0].mean(0))
        assert np.allclose(lse[t], np.log(t + 1))
    o, lse, _ = so.attend(q, np.zeros((3, 1, 64)), v, have, 3, 0.125, window=1)
    assert np.allclose(o, v)
    o, lse, _ = so.attend(q, np.zeros((0, 1, 64)), np.zeros((0, 1, 64)), have[:0], 0, 0.125)
    assert not o.any() and np.isneginf(lse).all()


def test_planted_mistakes_are_far_outside_the_tolerances():
    """A key too many or too few, a neighbour's head and an unrounded block
    each move the output by far more than the GPU tests allow (2^-7)."""
    rng = np.random.default_rng(4)
    q = rng.standard_normal((2, 4, 64)) * 2
    k, v = rng.standard_normal((2, 40, 2, 64))
    have = np.ones(40, bool)
    o, _, w = so.attend(q, k, v, have, 40, 0.125)

    def off(other):
        return float((np.abs(other - o) / w).max())
    assert off(so.attend(q, k, v, have, 40, 0.125, causal=False)[0]) > 2 ** -5
    late = have.copy()
    late[0] = False
    assert off(so.attend(q, k, v, late, 40, 0.125)[0]) > 2 ** -5
    assert off(so.attend(q, k[:, ::-1], v[:, ::-1], have, 40, 0.125)[0]) > 2 ** -5
    held = so.decode(*so.encode(v))
    assert off(so.attend(q, k, held, have, 40, 0.125)[0]) > 2 ** -5
