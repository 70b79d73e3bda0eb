"""CPU oracle of the attention half of a decoder block, in NumPy float64
(test infrastructure only; the library never calls it): rotary positions, the
4-bit blocks and their page layout, and attention of rows over keys.

The one place that works in float32 is `rotate32`, which forms the two
products and their sum each rounded to float32, as the cache's definition
asks: what is quantised afterwards is then the same to the bit.
"""
from __future__ import annotations

import math

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
NAN_SCALE = 255


def angle_steps(rot, base, kind=None, factor=1.0, original=1.0, low=1.0, high=4.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if kind == "base":
        base = base * factor ** (rot / (rot - 2))
    w = base ** (-2.0 * i / rot)
    if kind == "linear":
        return w / factor
    if kind == "yarn":
        def index(turns):  # the pair that turns this often over the original context
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        a, b = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
        ramp = np.clip((i - a) / (b - a if b != a else 0.001), 0, 1)
        return w * (1 - ramp) + w / factor * ramp
    if kind == "bands":
        turns = original * w / (2 * math.pi)
        keep = np.clip((turns - low) / (high - low), 0, 1)
        return keep * w + (1 - keep) * w / factor
    return w


def table(max_pos, rot, base=10000.0, amplitude=1.0, **kw):
    a = np.arange(max_pos, dtype=np.float64)[:, None] * angle_steps(rot, base, **kw)
    return np.stack([np.cos(a), np.sin(a)], -1) * amplitude


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, cs, interleaved, transposed=False):
    """x [n, h, dim] in any precision, cs [n, rot / 2, 2] of the same."""
    rot = 2 * cs.shape[1]
    one, two = pairs(rot, interleaved)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    if transposed:
        s = -s
    y = x.copy()
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def rotate32(x, cs, interleaved):
    return rotate(x.astype(np.float32), cs.astype(np.float32), interleaved)


def encode(x, limit=7.0):
    """Codes [..., dim] and scale bytes [..., dim / 32] of x [..., dim]."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(x).all(-1)
    b = np.where(bad[..., None, None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.full(top.shape, -125)
    for k in range(-125, 125):  # the least e that holds the block's largest value
        e = np.where(top > limit * 2.0 ** k, k + 1, e)
    y = np.abs(b) / 2.0 ** e[..., None]
    d = np.abs(y[..., None] - GRID)
    code = np.zeros(y.shape, np.int64)
    best = d[..., 0]
    for k in range(1, 8):
        # nearer, or as near and even
        take = (d[..., k] < best) | ((d[..., k] == best) & (k % 2 == 0))
        code, best = np.where(take, k, code), np.where(take, d[..., k], best)
    code = code + 8 * np.signbit(b)
    code = np.where(bad[..., None, None], 0, code).reshape(x.shape)
    scale = np.where(bad[..., None], NAN_SCALE, e + 127)
    return code.astype(np.uint8), scale.astype(np.uint8)


def decode(code, scale):
    v = GRID[code & 7] * np.where(code >> 3, -1.0, 1.0)
    s = np.where(scale > 252, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    b = v.reshape(v.shape[:-1] + (-1, 32)) * s[..., None]
    return b.reshape(v.shape)


def page_offsets(page, dim, off):
    """Byte offsets, in a head's block, of token `off`: its K bytes [dim / 2],
    V bytes [dim / 2], K scales and V scales [dim / 32]."""
    j, s = np.arange(dim // 2), np.arange(dim // 32)
    k = off * (dim // 2) + j
    v = page * (dim // 2) + (off // 4) * 2 * dim + (j // 4) * 16 + (off % 4) * 4 + j % 4
    ks = page * dim + off * (dim // 32) + s
    vs = page * dim + page * (dim // 32) + s * page + off
    return k, v, ks, vs


def token_page(page_table, n_pages, page, b, idx):
    """The page of token idx of sequence b, or None."""
    if idx < 0 or idx // page >= page_table.shape[1]:
        return None
    p = int(page_table[b, idx // page])
    return p if 0 <= p < n_pages else None


def owners(n, batch, kv_lens, q_starts):
    """(sequence, index) of every row; (None, None) for rows of none."""
    if q_starts is None:
        q_starts = np.arange(batch + 1) * (n // batch)
    out = [(None, None)] * n
    for b in range(batch):
        for r in range(q_starts[b], q_starts[b + 1]):
            out[r] = (b, int(kv_lens[b] - (q_starts[b + 1] - r)))
    return out


def put(pages, page_table, where, k, v):
    """Writes k and v [n, heads, dim] (already rotated) into a copy of pages
    [n_pages, heads, block]."""
    pages = pages.copy()
    dim = k.shape[2]
    page = pages.shape[2] * 16 // (dim * 17)
    kc, ks = encode(k)
    vc, vs = encode(v)
    for n, (b, idx) in enumerate(where):
        p = None if b is None else token_page(page_table, pages.shape[0], page, b, idx)
        if p is None:
            continue
        ok, ov, oks, ovs = page_offsets(page, dim, idx % page)
        for h in range(k.shape[1]):
            pages[p, h, ok] = kc[n, h, 0::2] | kc[n, h, 1::2] << 4
            pages[p, h, ov] = vc[n, h, 0::2] | vc[n, h, 1::2] << 4
            pages[p, h, oks], pages[p, h, ovs] = ks[n, h], vs[n, h]
    return pages


def get(pages, page_table, b, idx, dim):
    """k and v [heads, dim] of token idx of sequence b; None without a page."""
    page = pages.shape[2] * 16 // (dim * 17)
    p = token_page(page_table, pages.shape[0], page, b, idx)
    if p is None:
        return None
    ok, ov, oks, ovs = page_offsets(page, dim, idx % page)

    def one(c, s):
        raw = pages[p][:, c]
        return decode(np.stack([raw & 15, raw >> 4], -1).reshape(raw.shape[0], dim), pages[p][:, s])
    return one(ok, oks), one(ov, ovs)


def gather(pages, page_table, b, length, dim):
    """k, v [length, heads, dim] and which tokens have a page."""
    heads = pages.shape[1]
    k, v = np.zeros((length, heads, dim)), np.zeros((length, heads, dim))
    have = np.zeros(length, bool)
    for j in range(length):
        kv = get(pages, page_table, b, j, dim)
        if kv is not None:
            k[j], v[j], have[j] = kv[0], kv[1], True
    return k, v, have


def attend(q, k, v, have, length, scale, window=0, causal=True):
    """q [new, q_heads, dim] at the end of `length` keys. Returns o, lse and
    sum_j p_j |v_j| (what a relative error of the weights is multiplied by)."""
    new, hq, dim = q.shape
    hk = k.shape[1]
    o = np.zeros((new, hq, dim))
    weight = np.zeros((new, hq, dim))
    lse = np.full((new, hq), -np.inf)
    for t in range(new):
        p = length - new + t
        hi = min(p + 1, length) if causal else length
        lo = max(0, p - window + 1) if window else 0
        j = np.arange(lo, max(hi, lo))
        j = j[have[j]]
        if not len(j):
            continue
        for h in range(hq):
            g = h // (hq // hk)
            s = k[j, g] @ q[t, h] * scale
            m = s.max()
            e = np.exp(s - m)
            o[t, h] = (e / e.sum()) @ v[j, g]
            weight[t, h] = (e / e.sum()) @ np.abs(v[j, g])
            lse[t, h] = m + np.log(e.sum())
    return o, lse, weight
