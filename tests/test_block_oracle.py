"""CPU-only: the oracle of norms, linear attention and AdamW against
differences, closed forms and torch's float8, and planted mistakes against the
GPU tests' tolerances."""
import numpy as np
import pytest
import torch

import oracle.block_oracle as bo


def slope(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("norm_post", [False, True])
@pytest.mark.parametrize("norm_pre", [False, True])
def test_norm_gradients_against_differences(norm_post, norm_pre):
    rng = np.random.default_rng(0)
    n, d, scale, eps = 3, 16, 0.7, 1e-3
    v = {k: rng.standard_normal(s) for k, s in dict(x=(n, d), f=(n, d), gate=(n, d), post=(d,), pre=(d,)).items()}
    dr, dh = rng.standard_normal((2, n, d))

    def loss(w):
        r, _ = bo.residual(w["x"], w["f"], w["post"], w["gate"], scale, eps, norm_post)
        return (dr * r).sum() + ((dh * bo.pre_norm(r, w["pre"], eps)).sum() if norm_pre else 0.0)
    r, _ = bo.residual(v["x"], v["f"], v["post"], v["gate"], scale, eps, norm_post)
    g = bo.norm_backward(dr, dh, r, v["f"], v["post"], v["pre"], v["gate"], scale, eps, norm_post, norm_pre)
    got = dict(x=g["dx"], f=g["df"], gate=g["dgate"])
    if norm_post:
        got["post"] = g["dpost"].sum(0)
    if norm_pre:
        got["pre"] = g["dpre"].sum(0)
    for k, dk in got.items():
        u = rng.standard_normal(v[k].shape)
        assert abs(slope(lambda z: loss({**v, k: z}), v[k], u) - (dk * u).sum()) < 1e-6, k


def case(rng, n=9, hq=4, hk=2, a=5, b=3):
    q, k, v = rng.standard_normal((n, hq, a)), rng.standard_normal((n, hk, a)), rng.standard_normal((n, hk, b))
    return q, k, v, np.array([0.9, 0.3])[:hk], 0.6, rng.standard_normal((hk, a, b))


def test_linear_against_pairs():
    """o_t = scale (sum_j g^(t - j) (q_t k_j) v_j + g^(t + 1) S0^T q_t)."""
    q, k, v, g, scale, s0 = case(np.random.default_rng(1))
    o, s = bo.linear(q, k, v, g, scale, s0)
    n = len(q)
    for h in range(4):
        kh = h // 2
        d = np.tril(g[kh] ** np.subtract.outer(np.arange(n), np.arange(n)).clip(0))
        want = scale * (((q[:, h] @ k[:, kh].T) * d) @ v[:, kh] + g[kh] ** (np.arange(n) + 1)[:, None] * (q[:, h] @ s0[kh]))
        assert np.allclose(o[:, h], want)
    left = g[:, None] ** np.arange(n - 1, -1, -1)
    assert np.allclose(s, g[:, None, None] ** n * s0 + np.einsum("hn,nha,nhb->hab", left, k, v))


def test_linear_gradients_against_differences():
    rng = np.random.default_rng(2)
    q, k, v, g, scale, s0 = case(rng)
    do, ds = rng.standard_normal((9, 4, 3)), rng.standard_normal(s0.shape)

    def loss(q, k, v, s0):
        o, s = bo.linear(q, k, v, g, scale, s0)
        return (do * o).sum() + (ds * s).sum()
    got = bo.linear_backward(do, q, k, v, g, scale, s0, ds)
    args = [q, k, v, s0]
    for i, grad in enumerate(got):
        u = rng.standard_normal(grad.shape)

        def at(x):
            return loss(*args[:i], x, *args[i + 1:])
        assert abs(slope(at, args[i], u) - (grad * u).sum()) < 1e-6, i


def test_codes():
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(bo.e4m3(c), want, equal_nan=True)
    x = bo.e4m4(c)
    assert x[0] == 0 and x[255] == 496 and (np.diff(x) > 0).all()
    assert np.allclose(np.diff(x)[16:] / x[16:-1], 2.0 ** -4, rtol=0.51)


def test_planted_mistakes_are_far_outside_the_tolerances():
    """A token too many, a decay too many and a neighbour's head move linear
    attention's outputs by far more than the 2^-8 that bf16's tests allow of
    all of them together."""
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((100, 4, 64)), rng.standard_normal((100, 2, 64)), rng.standard_normal((100, 2, 64))
    g = np.array([0.95, 0.99])
    o, _ = bo.linear(q, k, v, g, 0.125)

    def off(x):
        return np.linalg.norm(x - o) / np.linalg.norm(o)
    late = k.copy()
    late[0] = 0
    assert off(bo.linear(q, late, v, g, 0.125)[0]) > 2 ** -5
    assert off(bo.linear(q, k, v, g * g, 0.125)[0]) > 2 ** -5
    assert off(bo.linear(q, k[:, ::-1], v, g, 0.125)[0]) > 2 ** -5
    assert off(bo.linear(q, np.roll(k, 1, 0), np.roll(v, 1, 0), g, 0.125)[0]) > 2 ** -5
