"""The cases on which the attention half of a decoder block is measured:
rotary positions (rope), appending to a paged 4-bit key/value cache (append)
and attention over that cache (attention).

The cache is a pool of pages, a uint8 tensor [pages, kv heads, bytes]. A page
holds `page` tokens; for one of its heads, with D values a head:
    K codes   [page][D / 2]             byte j: value 2j low, 2j + 1 high
    V codes   [page / 4][D / 8][4][4]   of four tokens: 8 values (4 bytes) of each
    K scales  [page][D / 32]
    V scales  [D / 32][page]
A value is (+-){0, .5, 1, 1.5, 2, 3, 4, 6} * 2^(scale - 127), 32 neighbouring
values of a token sharing the scale byte; scale 255 stands for NaN. The scale
is the least power of two 2^e with max|x| <= 7 * 2^e, -125 <= e <= 125.
Page p of sequence b is page_table[b, p]; kv_lens counts a sequence's tokens,
the new ones included, and q_starts bounds its new tokens in the rows.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases


def _rope(name, tokens, hq, hk, dim, rot, dtype, interleaved, backward, max_pos):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hk": hk, "dim": dim, "rot": rot, "dtype": dtype,
            "interleaved": interleaved, "backward": backward, "max_pos": max_pos}


def _append(name, batch, tokens, cached, hq, hk, dim, rot, dtype, interleaved, page, lens):
    """`tokens` new ones over `batch` sequences, each with up to `cached` tokens before them."""
    return {"name": name, "op": "append", "batch": batch, "tokens": tokens, "cached": cached, "hq": hq, "hk": hk, "dim": dim,
            "rot": rot, "dtype": dtype, "interleaved": interleaved, "page": page, "lens": lens}


def _attention(name, batch, new, kv, hq, hk, dim, dtype, page, window, lens):
    """Up to `new` query tokens a sequence over up to `kv` cached ones; lens 0: every sequence has just those."""
    return {"name": name, "op": "attention", "batch": batch, "new": new, "kv": kv, "hq": hq, "hk": hk, "dim": dim,
            "dtype": dtype, "page": page, "window": window, "lens": lens}


def listed():
    return [
        # one token each of four sequences being decoded together
        _rope("rope_step", 4, 32, 8, 128, 128, "bf16", False, False, 131072),
        # a training sequence of 64k tokens, queries and keys of one fused projection
        _rope("rope_train_64k", 65536, 32, 8, 128, 128, "bf16", False, False, 65536),
        # the gradient in fp32, a part of the head rotated, neighbouring pairs, an odd token count
        _rope("rope_backward_f32", 30001, 16, 16, 96, 32, "f32", True, True, 32768),
        # the smallest serving call: one token of one sequence enters its cache
        _append("append_step", 1, 1, 4095, 32, 8, 128, 128, "bf16", False, 64, 0),
        # a step of continuous batching: ragged prompts and single tokens together, fp32, small heads
        _append("append_ragged_f32", 37, 3001, 5000, 16, 4, 64, 32, "f32", True, 16, 11),
        # a whole 64k prompt written at once
        _append("append_prompt_64k", 1, 65536, 0, 32, 8, 128, 128, "bf16", False, 128, 0),
        # one token over a short chat, where latency counts
        _attention("attend_step_short", 1, 1, 777, 32, 8, 128, "bf16", 64, 0, 0),
        # one token over a 128k context, five query heads a key head
        _attention("attend_step_128k", 1, 1, 131072, 40, 8, 128, "bf16", 128, 0, 0),
        # one token each of 32 sequences of ragged lengths up to 32k
        _attention("attend_step_batch32", 32, 1, 32768, 32, 8, 128, "bf16", 64, 0, 5),
        # the next chunk of 1024 tokens of a 64k document
        _attention("attend_segment_64k", 1, 1024, 65536, 32, 8, 128, "bf16", 128, 0, 0),
        # a prompt of 8k tokens
        _attention("attend_prompt_8k", 1, 8192, 8192, 32, 8, 128, "bf16", 64, 0, 0),
        # ragged segments in fp32, wide heads, a sliding window, pages that end inside a tile
        _attention("attend_window_f32", 5, 611, 3500, 12, 4, 256, "f32", 48, 1000, 7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    inter = rng.random() < 0.4
    group = rng.choice([1, 2, 4, 5, 8, 16])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * group
    dim = rng.choice([64, 128, 128, 256])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= dim] + [dim])
        most = 65536 * 40 * 128 * 2 // ((hq + hk) * dim * SIZE[dtype])
        c = _rope("", _log(rng, 1, min(65536, most)), hq, hk, dim, rot, dtype, inter, rng.random() < 0.5, rng.choice([65536, 131072]))
    elif op == "append":
        rot = rng.choice([r for r in (32, 64, 128) if r <= dim] + [dim])
        batch = _log(rng, 1, 64)
        most = 65536 * 48 * 128 * 2 // ((hq + 2 * hk) * dim * SIZE[dtype])
        c = _append("", batch, max(batch, _log(rng, 1, min(65536, most))), _log(rng, 1, 8192), hq, hk, dim, rot, dtype, inter,
                    rng.choice([16, 32, 48, 64, 128, 256]), rng.randrange(1, 1000))
    elif rng.random() < 0.5:  # single tokens
        batch = _log(rng, 1, 64)
        kv = _log(rng, 1, min(131072, 32 * 32768 * 8 * 128 // (batch * hk * dim)))
        c = _attention("", batch, rng.choice([1, 1, 1, 2, 4]), kv, hq, hk, dim, dtype, rng.choice([16, 32, 48, 64, 128, 256]),
                       rng.choice([0, 0, _log(rng, 1, 4096)]), rng.choice([0, rng.randrange(1, 1000)]))
    else:  # segments
        batch = _log(rng, 1, 8)
        new = _log(rng, 16, 4096)
        kv = max(new, _log(rng, 16, max(16, min(65536, 1024 * 65536 * 32 * 128 // (batch * new * hq * dim)))))
        new = min(new, max(1, 1024 * 65536 * 32 * 128 // (batch * kv * hq * dim)))
        c = _attention("", batch, new, kv, hq, hk, dim, dtype, rng.choice([16, 32, 48, 64, 128, 256]),
                       rng.choice([0, 0, _log(rng, 1, 4096)]), rng.choice([0, rng.randrange(1, 1000)]))
    del c["name"]
    return c


def _lens(case):
    """(new tokens, cached and new tokens) of every sequence: the case's own, so that its work is known."""
    r = random.Random(case["lens"])
    if case["op"] == "append":
        n, left = [1] * case["batch"], case["tokens"] - case["batch"]
        for b in range(case["batch"]):  # a few sequences take most of the new tokens
            take = left if b == case["batch"] - 1 else min(left, int(left * r.random() ** 2))
            n[b] += take
            left -= take
        r.shuffle(n)
        return n, [x + (r.randint(0, case["cached"]) if case["lens"] else case["cached"]) for x in n]
    if not case["lens"]:
        return [case["new"]] * case["batch"], [case["kv"]] * case["batch"]
    n = [r.randint(1, case["new"]) for _ in range(case["batch"])]
    return n, [max(x, r.randint(case["kv"] // 8, case["kv"])) for x in n]


def _pairs(q, kv, window):
    """(Query, key) pairs that a sequence's rows see, and the keys that any of them sees."""
    first = kv - q  # the position of the first row
    if not window:
        return q * first + q * (q + 1) // 2, kv
    return sum(min(window, first + t + 1) for t in range(q)), kv - max(0, first - window + 1)


def work(case):
    size, dim = SIZE[case["dtype"]], case["dim"]
    if case["op"] == "rope":
        rows = case["tokens"] * (case["hq"] + case["hk"])
        return {"bytes": rows * dim * size * 2 + case["tokens"] * (case["rot"] * 4 + 4), "flops": rows * case["rot"] * 3}
    if case["op"] == "append":
        t, hq, hk = case["tokens"], case["hq"], case["hk"]
        stored = 2 * t * hk * (dim // 2 + dim // 32)  # written, and read back
        return {"bytes": t * (2 * hq + 4 * hk) * dim * size + 2 * stored + t * case["rot"] * 4,
                "flops": t * ((hq + hk) * case["rot"] * 3 + 2 * hk * dim * 4)}
    seen = [_pairs(q, kv, case["window"]) for q, kv in zip(*_lens(case))]
    rows = sum(_lens(case)[0])
    return {"bytes": sum(k for _, k in seen) * case["hk"] * (dim + dim // 16) + rows * case["hq"] * (2 * dim * size + 4),
            "flops": 4 * dim * case["hq"] * sum(p for p, _ in seen)}


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _table(max_pos, rot):
    """cos and sin of every position's angles, as a program keeps them: fp32 [max_pos, rot / 2, 2]."""
    w = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * w
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _views(pages, dim):
    """The pool's four parts: K codes [n, h, page, dim/2], V codes [n, h, page/4, dim/8, 4, 4], K scales [n, h, page, dim/32],
    V scales [n, h, dim/32, page]."""
    page = pages.shape[2] * 16 // (dim * 17)
    a, s = page * dim // 2, page * dim // 32
    return (pages[:, :, :a].unflatten(2, (page, dim // 2)), pages[:, :, a:2 * a].unflatten(2, (page // 4, dim // 8, 4, 4)),
            pages[:, :, 2 * a:2 * a + s].unflatten(2, (page, dim // 32)), pages[:, :, 2 * a + s:].unflatten(2, (dim // 32, page)))


def _encode(x):
    """Codes (two a byte) and scale bytes of fp32 x [..., dim]."""
    b = x.unflatten(-1, (-1, 32))
    m, ex = torch.frexp(b.abs().amax(-1, keepdim=True))  # amax = m 2^ex, .5 <= m < 1
    e = torch.where(m <= 0.875, ex - 3, ex - 2).clamp(-125, 125)
    y = torch.ldexp(b.abs(), -e)
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
            + 8 * torch.signbit(b).to(torch.uint8))
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] | (code[..., 1] << 4), (e + 127).squeeze(-1).to(torch.uint8)


def _decode(code, scale):
    """fp32 values of codes [..., dim / 2] and scale bytes [..., dim / 32]."""
    c = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=code.device)
    v = grid[(c & 7).int()] * (1 - 2 * (c >> 3).float())
    s = torch.ldexp(torch.ones((), device=code.device), scale.int() - 127)
    s = torch.where(scale == 255, torch.full_like(s, math.nan), s)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _pool(case, g, kv_lens):
    """A pool with spare pages, in no order, and its page table. What no token fills is left as random bytes."""
    page, dim, hk = case["page"], case["dim"], case["hk"]
    need = [-(-n // page) for n in kv_lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).int().cpu()
    table = torch.zeros(len(need), max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pages = torch.randint(0, 256, (n_pages, hk, page * dim * 17 // 16), generator=g, device=DEV, dtype=torch.uint8)
    return pages, table.to(DEV)


def prepare(case, seed):
    g = _generator(seed)
    dtype, dim, hq, hk = DTYPES[case["dtype"]], case["dim"], case["hq"], case["hk"]
    s = dict(case)
    if case["op"] == "rope":
        n = case["tokens"]
        s["table"] = _table(case["max_pos"], case["rot"])
        if n > 64:  # a sequence, or its last part
            s["positions"] = torch.arange(n, device=DEV, dtype=torch.int32) + (case["max_pos"] - n) // 2
        else:
            s["positions"] = torch.randint(0, case["max_pos"], (n,), generator=g, device=DEV, dtype=torch.int32)
        x = _randn(g, n, hq + 2 * hk, dim).to(dtype)  # the projection's output, values behind the keys
        s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
        return s
    q_lens, kv_lens = _lens(case)
    n = sum(q_lens)
    s["pages"], s["page_table"] = _pool(case, g, kv_lens)
    s["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    starts = [0]
    for x in q_lens:
        starts.append(starts[-1] + x)
    s["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["max_new"], s["max_kv"], s["rows"] = max(q_lens), max(kv_lens), n
    if case["op"] == "append":
        s["table"] = _table(max(kv_lens), case["rot"])
        x = _randn(g, n, hq + 2 * hk, dim).to(dtype)
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        return s
    # keys with a strong channel or two, as rotary heads have them; queries that make some keys stand out
    kc, vc, ks, vs = _views(s["pages"], dim)
    page = case["page"]
    loud = 1 + 3 * (torch.rand(hk, 1, dim, generator=g, device=DEV) > 0.95).float()
    step = max(1, (1 << 26) // (hk * page * dim))
    for i in range(0, s["pages"].shape[0], step):
        m = min(step, s["pages"].shape[0] - i)
        code, scale = _encode(_randn(g, m, hk, page, dim) * loud)
        kc[i:i + m], ks[i:i + m] = code, scale
        code, scale = _encode(_randn(g, m, hk, page, dim))
        vc[i:i + m] = code.view(m, hk, page // 4, 4, dim // 8, 4).transpose(3, 4)
        vs[i:i + m] = scale.transpose(2, 3)
    last = s["page_table"].cpu()
    for b, length in enumerate(kv_lens):  # NaN behind each sequence's last token
        if length % page:
            at = int(last[b, length // page])
            ks[at, :, length % page:], vs[at, :, :, length % page:] = 255, 255
    s["q"] = (1.5 * _randn(g, n, hq, dim)).to(dtype)
    s["scale"] = dim ** -0.5
    return s


# ------------------------------------------------------------------ plain forms


def _rotate(x, cs, interleaved, sign=1.0):
    """x fp32 [n, h, dim], cs [n, rot / 2, 2]."""
    rot = 2 * cs.shape[1]
    c, s = cs[:, None, :, 0], sign * cs[:, None, :, 1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _places(s):
    """(sequence, index among its tokens) of every new token."""
    n = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(s["q_starts"][1:].long(), n, right=True)
    return b, s["kv_lens"][b].long() - s["q_starts"][b + 1].long() + n


def _plain_append(s):
    dim, page = s["dim"], s["page"]
    b, j = _places(s)
    cs = s["table"][j]
    q = _rotate(s["q"].float(), cs, s["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cs, s["interleaved"])
    at, off = s["page_table"][b, j // page].long(), j % page
    kc, vc, ks, vs = _views(s["pages"], dim)
    code, scale = _encode(k)
    kc[at, :, off], ks[at, :, off] = code, scale
    code, scale = _encode(s["v"].float())
    vc[at, :, off // 4, :, off % 4], vs[at, :, :, off] = code.unflatten(-1, (-1, 4)), scale
    # read back
    k = _decode(kc[at, :, off], ks[at, :, off]).to(s["k"].dtype)
    v = _decode(vc[at, :, off // 4, :, off % 4].flatten(-2), vs[at, :, :, off]).to(s["v"].dtype)
    return {"q": q, "k": k, "v": v}


def _plain_attention(s):
    dim, hq, hk, batch = s["dim"], s["hq"], s["hk"], s["batch"]
    group, new, length = hq // hk, s["max_new"], s["max_kv"]
    kc, vc, ks, vs = _views(s["pages"], dim)
    at = s["page_table"].long()  # [b, p]
    kv, starts = s["kv_lens"].long(), s["q_starts"].long()
    have = torch.arange(length, device=DEV) < kv[:, None]  # [b, j]
    k = _decode(kc[at], ks[at]).transpose(1, 2).flatten(2, 3)[:, :, :length]  # [b, h, j, dim]
    k = torch.where(have[:, None, :, None], k, 0.0)
    v = _decode(vc[at].transpose(4, 5).flatten(5, 6).flatten(3, 4), vs[at].transpose(3, 4))
    v = v.transpose(1, 2).flatten(2, 3)[:, :, :length]
    v = torch.where(have[:, None, :, None], v, 0.0)
    # the rows, padded to the longest sequence's
    t = torch.arange(new, device=DEV)
    n = (starts[1:] - starts[:-1])[:, None]
    row = (starts[:-1, None] + t).clamp(max=s["rows"] - 1)
    q = s["q"].float()[row].view(batch, new, hk, group, dim).permute(0, 2, 3, 1, 4).flatten(2, 3).contiguous()
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"]).unflatten(2, (group, new))
    del k
    p = kv[:, None] - n + t  # [b, t] the row's position
    j = torch.arange(length, device=DEV)
    see = (j <= p[:, :, None]) & have[:, None]
    if s["window"]:
        see &= j > p[:, :, None] - s["window"]
    x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    x.sub_(m0).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v).unflatten(2, (group, new)) / torch.where(z == 0, 1.0, z)
    lse = (m0 + z.log()).squeeze(-1)
    # the rows back in their places
    b, j = _places(s)
    t = torch.arange(s["rows"], device=DEV) - starts[b]
    o, lse = o[b, :, :, t], lse[b, :, :, t]
    return {"o": o.flatten(1, 2).to(s["q"].dtype), "lse": lse.flatten(1, 2)}


def run(s):
    if own:
        import test_layer_gate_amd as ttt
        if s["op"] == "rope":
            f = ttt.rope_backward if s["backward"] else ttt.rope_forward
            q, k = f(s["q"], s["k"], s["table"], positions=s["positions"], interleaved=s["interleaved"])
            return {"q": q, "k": k}
        if s["op"] == "append":
            q = ttt.kv_append(s["pages"], s["page_table"], s["kv_lens"], s["k"], s["v"], q=s["q"], q_starts=s["q_starts"],
                              rope_table=s["table"], interleaved=s["interleaved"])
            k, v = ttt.kv_read(s["pages"], s["page_table"], s["kv_lens"], s["rows"], s["dim"], s["k"].dtype,
                               q_starts=s["q_starts"])
            return {"q": q, "k": k, "v": v}
        o, lse = ttt.kv_attention(s["q"], s["pages"], s["page_table"], s["kv_lens"], q_starts=s["q_starts"],
                                  max_new=s["max_new"], max_kv=s["max_kv"], scale=s["scale"], window=s["window"], with_lse=True)
        return {"o": o, "lse": lse}
    if s["op"] == "rope":
        cs, sign = s["table"][s["positions"].long()], -1.0 if s["backward"] else 1.0
        return {"q": _rotate(s["q"].float(), cs, s["interleaved"], sign).to(s["q"].dtype),
                "k": _rotate(s["k"].float(), cs, s["interleaved"], sign).to(s["k"].dtype)}
    return _plain_append(s) if s["op"] == "append" else _plain_attention(s)


# ------------------------------------------------------------------ in 64 bits


def _turned(x, table, at, interleaved, back):
    """Each pair of x as a complex number, times its angle's (or, back, its conjugate)."""
    rot = 2 * table.shape[1]
    z = torch.view_as_complex(table.double())[at][:, None]
    z = z.conj() if back else z
    y = x.double().clone()
    i = torch.arange(rot // 2, device=DEV)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    w = torch.complex(y[..., one], y[..., two]) * z
    y[..., one], y[..., two] = w.real, w.imag
    return y


def _held(x):
    """What the cache holds of x (fp64 [n, h, dim]), from the format's definition."""
    out = torch.empty_like(x)
    steps = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    for i in range(0, x.shape[0], 4096):
        b = x[i:i + 4096].unflatten(-1, (-1, 32))
        top = b.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top / 7)).clamp(-125, 125)
        e = torch.where(top > 7 * 2.0 ** e, e + 1, torch.where(top <= 7 * 2.0 ** (e - 1), e - 1, e)).clamp(-125, 125)
        y = b.abs() / 2.0 ** e
        lo = (torch.searchsorted(steps, y, right=True) - 1).clamp(0, 6)  # steps[lo] <= y
        down, up = y - steps[lo], steps[lo + 1] - y
        pick = torch.where((up < down) | ((up == down) & (lo % 2 == 1)), lo + 1, lo)
        out[i:i + 4096] = (torch.sign(b) * steps[pick] * 2.0 ** e).flatten(-2)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    dim, hk = s["dim"], s["hk"]
    if s["op"] == "rope":
        at = s["positions"].long()
        return {n: _turned(s[n], s["table"], at, s["interleaved"], s["backward"]) for n in ("q", "k")}
    q_lens, kv_lens = _lens(case)
    if s["op"] == "append":
        at = torch.cat([torch.arange(n - m, n, device=DEV) for m, n in zip(q_lens, kv_lens)])
        return {"q": _turned(s["q"], s["table"], at, s["interleaved"], False),
                "k": _held(_turned(s["k"], s["table"], at, s["interleaved"], False)), "v": _held(s["v"].double())}
    page = s["page"]
    steps = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEV)
    n_code = page * dim // 2
    o = torch.zeros(s["rows"], s["hq"], dim, dtype=torch.float64, device=DEV)
    lse = torch.full((s["rows"], s["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    group, row = s["hq"] // hk, 0
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        raw = s["pages"][s["page_table"][b, :-(-n // page)].long()].long()
        d = torch.arange(dim, device=DEV)
        tok = torch.arange(page, device=DEV)[:, None]
        k_at, v_at = tok * (dim // 2) + d // 2, n_code + (tok // 4) * (dim * 2) + (d // 8) * 16 + (tok % 4) * 4 + d % 8 // 2
        ks_at, vs_at = 2 * n_code + tok * (dim // 32) + d // 32, 2 * n_code + page * (dim // 32) + (d // 32) * page + tok
        p = torch.arange(n - m, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)
        see = (j <= p) & (j > p - (s["window"] or n + 1))
        for h in range(hk):
            k, v = (steps[(raw[:, h][:, c] >> (d % 2 * 4)) & 15] * 2.0 ** (raw[:, h][:, e] - 127).double()
                    for c, e in ((k_at, ks_at), (v_at, vs_at)))
            k, v = k.flatten(0, 1)[:n], v.flatten(0, 1)[:n]
            for i in range(group):
                x = (s["q"][row:row + m, h * group + i].double() @ k.T) * s["scale"]
                x = x.masked_fill(~see, -math.inf)
                lse[row:row + m, h * group + i] = torch.logsumexp(x, -1)
                o[row:row + m, h * group + i] = torch.softmax(x, -1) @ v
        row += m
    return {"o": o, "lse": lse}
