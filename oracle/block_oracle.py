"""CPU oracle of the operators around and beside a block, in NumPy float64
(test infrastructure only; the library never calls it): the norms with gate and
residual scale, linear attention token by token, AdamW and its 8-bit states.

Where a test bounds an error by the size of what was summed, the functions
return those sums of magnitudes too.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ norms


def rms(x, eps):
    return 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def residual(x, f, post=None, gate=None, scale=1.0, eps=1e-6, norm=False):
    """r = x + scale * gate * n (gate: rows, or broadcast), and |x| + |its other part|."""
    n = f
    if norm:
        n = f * rms(f, eps) * (1.0 if post is None else post)
    y = scale * n * (1.0 if gate is None else gate)
    return x + y, np.abs(x) + np.abs(y)


def pre_norm(r, pre=None, eps=1e-6):
    return r * rms(r, eps) * (1.0 if pre is None else pre)


def norm_backward(dr, dh, r, f, post, pre, gate, scale, eps, norm_post, norm_pre):
    """Gradients by row (dgate, dpost and dpre not summed yet), and for dx and
    df the sums of magnitudes of which they are differences."""
    out, D, size = {}, dr, np.abs(dr)
    d = D.shape[-1]
    if norm_pre:
        rho = rms(r, eps)
        t = dh * (1.0 if pre is None else pre)
        D = D + rho * (t - r * rho ** 2 * (r * t).mean(-1, keepdims=True))
        size = size + rho * (np.abs(t) + np.abs(r) * rho ** 2 * (np.abs(r * t)).sum(-1, keepdims=True) / d)
        out["dpre"] = dh * r * rho
    out["dx"], out["dx_size"] = D, size
    if f is not None:
        w = 1.0 if post is None or not norm_post else post
        phi = rms(f, eps) if norm_post else 1.0
        n = f * phi * w
        g = 1.0 if gate is None else gate
        dn = scale * g * D
        out["dgate"], out["dgate_size"] = scale * n * D, np.abs(scale * n) * size
        out["df"], out["df_size"] = dn, np.abs(scale * g) * size
        if norm_post:
            u, us = dn * w, np.abs(scale * g * w) * size
            out["dpost"], out["dpost_size"] = dn * f * phi, np.abs(scale * g * f * phi) * size
            out["df"] = phi * (u - f * phi ** 2 * (f * u).mean(-1, keepdims=True))
            out["df_size"] = phi * (us + np.abs(f) * phi ** 2 * (np.abs(f) * us).mean(-1, keepdims=True))
    return out


# -------------------------------------------------------- linear attention


def linear(q, k, v, decay, scale, state=None):
    """One sequence, token by token: q [n, hq, a], k [n, hk, a], v [n, hk, b],
    decay [hk] (the factor), state [hk, a, b]. Returns o, the last state."""
    n, hq, a = q.shape
    hk, b = v.shape[1:]
    s = np.zeros((hk, a, b)) if state is None else state.copy()
    o = np.zeros((n, hq, b))
    kept = np.asarray(decay)[:, None, None]
    for t in range(n):
        s = np.where(kept == 0, 0.0, kept * s) + k[t][:, :, None] * v[t][:, None]
        o[t] = scale * np.einsum("ha,hab->hb", q[t], np.repeat(s, hq // hk, 0))
    return o, s


def linear_backward(do, q, k, v, decay, scale, state=None, d_state=None):
    """Gradients of linear's q, k, v and first state, from do and d_state: the
    states forwards, their gradients backwards, token by token."""
    n, hq, a = q.shape
    hk, b = v.shape[1:]
    g = hq // hk
    s = np.zeros((hk, a, b)) if state is None else state.copy()
    kept = np.asarray(decay)[:, None, None]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for t in range(n):
        s = kept * s + k[t][:, :, None] * v[t][:, None]
        dq[t] = scale * np.einsum("hab,hb->ha", np.repeat(s, g, 0), do[t])
    d = np.zeros((hk, a, b)) if d_state is None else d_state.copy()
    for t in range(n - 1, -1, -1):
        d = d + scale * (q[t][:, :, None] * do[t][:, None]).reshape(hk, g, a, b).sum(1)
        dk[t] = np.einsum("hab,hb->ha", d, v[t])
        dv[t] = np.einsum("hab,ha->hb", d, k[t])
        d = kept * d
    return dq, dk, dv, d


# ------------------------------------------------------------------- AdamW


def adamw(p, g, m, v, lr, step, b1, b2, eps, wd):
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    u = lr * (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * wd) - u, m, v, u


def e4m3(c):
    """What an E4M3 code stands for."""
    c = np.asarray(c, np.int64)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    x = np.where((c & 127) == 127, np.nan, x)
    return np.where(c & 128, -x, x)


def e4m4(c):
    """What a code of 4 exponent and 4 fraction bits stands for."""
    c = np.asarray(c, np.int64)
    return np.where(c < 16, c * 2.0 ** -10, (16 + c % 16) * 2.0 ** (c // 16 - 11.0))


def read_states(state, total):
    """(m, r) of a buffer of 8-bit states (uint8)."""
    n = total
    scales = state[2 * n:].view(np.float32).astype(np.float64)
    sm, sr = (np.repeat(x, 256) for x in np.split(scales, 2))
    return e4m3(state[:n]) * sm, e4m4(state[n:2 * n]) * sr


def held(x, most, step_bits, least):
    """Half the distance between neighbours of the 8-bit grid at x (float64
    [n], n a multiple of 256): how far what is held may be from it. most: the
    largest code's value; step_bits: fraction bits; least: the least code above 0."""
    b = np.abs(x.reshape(-1, 256))
    s = np.maximum(b.max(1, keepdims=True) / most, 2.0 ** -126)
    y = b / s
    return (s * np.maximum(y * 2.0 ** -(step_bits + 1), least / 2)).reshape(-1)
