"""The cases on which three operators around a decoder block are measured:
the norms before and after a block with its gate and residual scale (norm),
linear attention with a decay for each head (linear), and an AdamW step over
many tensors (adamw).

norm     n = f, or f / rms(f) * post;  r = x + scale * gate * n, kept in x's
         type;  h = r / rms(r) * pre. The gate is one vector, one a sequence,
         one a row, or none. Backward: the gradients of x, f, gate and both
         weights from those of r and h.
linear   S_t = exp(log_decay) S_{t-1} + k_t v_t^T for every head of k and v,
         o_t = scale q_t S_t for every head of q of its group; sequences of
         ragged lengths between q_starts; the states are updated in place.
adamw    m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2, and the decoupled
         step on the weights. States of N values (every tensor padded to a
         multiple of 256) are held as m [N], v [N] in fp32, or in 8 bits as m
         codes [N], r codes [N], m scales [N / 256], r scales [N / 256], r =
         sqrt(v): code times its block's fp32 scale. m's codes are e4m3, the
         scale max|m| / 448; r's have 4 exponent and 4 fraction bits and no
         sign, the scale max r / 496; no r above 0 becomes 0.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases


def _norm(name, rows, d, dtype, res, gate, seqs, post, pre, backward):
    """gate: none, one (a vector), seq (one for each of `seqs` sequences) or row; res: the residual's type."""
    return {"name": name, "op": "norm", "rows": rows, "d": d, "dtype": dtype, "res": res, "gate": gate, "seqs": seqs,
            "post": post, "pre": pre, "backward": backward}


def _linear(name, batch, new, hk, group, dk, dv, dtype, lens, backward):
    """Up to `new` tokens for each of `batch` sequences; lens 0: every sequence has just those."""
    return {"name": name, "op": "linear", "batch": batch, "new": new, "hk": hk, "group": group, "dk": dk, "dv": dv,
            "dtype": dtype, "lens": lens, "backward": backward}


def _adamw(name, tensors, total, dtype, grad, master, bits, clip, layer=0):
    """`tensors` of about `total` values together, or, with layer > 0, a gated MLP's of that d_model and `total` d_ff."""
    return {"name": name, "op": "adamw", "tensors": tensors, "total": total, "dtype": dtype, "grad": grad,
            "master": master, "bits": bits, "clip": clip, "layer": layer}


def listed():
    return [
        # one token each of four sequences being decoded: the norm behind attention and the one before the MLP
        _norm("norm_step", 4, 2560, "bf16", "bf16", "none", 1, True, True, False),
        # a training sequence of 64k tokens, with a learned gate vector
        _norm("norm_train_64k", 65536, 2560, "bf16", "bf16", "one", 1, False, True, False),
        # the gradients of eight packed sequences, each with its own gate, both norms
        _norm("norm_backward_8x2k", 16384, 4096, "bf16", "bf16", "seq", 8, True, True, True),
        # an odd number of rows, an fp32 residual stream, a gate for every row, fp32 throughout
        _norm("norm_backward_f32", 5001, 1384, "f32", "f32", "row", 1, True, False, True),
        # one token each of 48 sequences
        _linear("linear_step_48", 48, 1, 8, 4, 128, 128, "bf16", 0, False),
        # a prompt of 64k tokens, grouped heads
        _linear("linear_prompt_64k", 1, 65536, 8, 4, 128, 128, "bf16", 0, False),
        # ragged prompts in fp32, small heads
        _linear("linear_ragged_f32", 7, 3001, 4, 1, 64, 64, "f32", 3, False),
        # the gradients of two training sequences of 8k tokens
        _linear("linear_backward_2x8k", 2, 8192, 16, 1, 128, 128, "bf16", 0, True),
        # norms, biases and small projections, where latency counts
        _adamw("adamw_small", 60, 150_000, "f32", "f32", False, 32, False),
        # the fast-weight MLP of the 64k configuration: bf16 weights with fp32 masters, fp32 gradients and states
        _adamw("adamw_layer_32", 5, 9728, "bf16", "f32", True, 32, False, 2560),
        # the same with states in 8 bits and the gradients' norm limited
        _adamw("adamw_layer_8", 5, 9728, "bf16", "f32", True, 8, True, 2560),
        # odd sizes, bf16 gradients, no masters, 8 bits
        _adamw("adamw_ragged_8", 37, 4_000_001, "bf16", "bf16", False, 8, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "norm":
        d = 8 * _log(rng, 16, 1024)
        rows = _log(rng, 1, min(65536, 2_400_000_000 // (d * (24 if dtype == "bf16" else 32))))
        gate = rng.choice(["none", "one", "seq", "row"])
        seqs = 1
        if gate == "seq":
            seqs = rng.randint(1, 16)
            rows = max(1, rows // seqs) * seqs
        res = "f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "f32"])
        c = _norm("", rows, d, dtype, res, gate, seqs, rng.random() < 0.6, rng.random() < 0.8, rng.random() < 0.5)
    elif op == "linear":
        dk, dv = rng.choice([64, 128, 128, 256]), rng.choice([64, 128, 128, 256])
        hk, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 4, 5])
        most = 65536 * 32 * 128 * 128 // (hk * group * dk * dv * (4 if dtype == "f32" else 1))
        if rng.random() < 0.4:  # single tokens, or a few
            batch = _log(rng, 1, max(1, min(256, 256 * 8 * 128 * 128 // (hk * dk * dv))))
            c = _linear("", batch, rng.choice([1, 1, 1, 2, 4, 7]), hk, group, dk, dv, dtype, 0, False)
        else:
            back = rng.random() < 0.4
            batch = rng.randint(1, 8)
            new = _log(rng, 16, max(16, min(65536, most // (batch * (3 if back else 1)))))
            c = _linear("", batch, new, hk, group, dk, dv, dtype, rng.choice([0, rng.randrange(1, 1000)]), back)
    else:
        grad = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        c = _adamw("", rng.randint(1, 62), _log(rng, 1000, 60_000_000), dtype, grad, dtype == "bf16" and rng.random() < 0.5,
                   rng.choice([8, 8, 32]), rng.random() < 0.5)
    del c["name"]
    return c


def _lens(case):
    """New tokens of every sequence: the case's own, so that its work is known."""
    if not case["lens"]:
        return [case["new"]] * case["batch"]
    r = random.Random(case["lens"])
    return [r.randint(1, case["new"]) for _ in range(case["batch"])]


def _shapes(case):
    """The tensors' shapes, likewise."""
    if case["layer"]:
        d, f = case["layer"], case["total"]
        return [(f, d), (f, d), (d, f), (4, d), (d, d)]
    r = random.Random(case["total"] * 64 + case["tensors"])
    w = [math.exp(r.uniform(0, 6)) for _ in range(case["tensors"])]
    return [(max(1, int(case["total"] * x / sum(w))),) for x in w]


def _offsets(shapes):
    """Where each tensor's values start among N, and N."""
    at, out = 0, []
    for s in shapes:
        out.append(at)
        at += -(-math.prod(s) // 256) * 256
    return out, at


def work(case):
    if case["op"] == "norm":
        n, d, s, res = case["rows"], case["d"], SIZE[case["dtype"]], SIZE[case["res"]]
        gate = n * d * s if case["gate"] == "row" else 0
        if case["backward"]:  # r, dr and dx; f and df; dh; the gate and its gradient
            return {"bytes": n * d * (3 * res + (2 + case["pre"]) * s) + 2 * gate, "flops": 20 * n * d}
        return {"bytes": n * d * (2 * res + (1 + case["pre"]) * s) + gate, "flops": 10 * n * d}
    if case["op"] == "linear":
        n, hk, dk, dv, s = sum(_lens(case)), case["hk"], case["dk"], case["dv"], SIZE[case["dtype"]]
        hq = hk * case["group"]
        states = case["batch"] * hk * dk * dv * 4
        if case["backward"]:  # q, k, v, do, and the gradients of the first three; the states' two
            return {"bytes": n * s * (2 * hq * dk + 2 * hk * (dk + dv) + hq * dv) + 3 * states,
                    "flops": 2 * n * dk * dv * (2 * hq + 3 * hk)}
        return {"bytes": n * s * (hq + hk) * (dk + dv) + 2 * states, "flops": 2 * n * dk * dv * (hq + hk)}
    n = sum(math.prod(s) for s in _shapes(case))
    each = 2 * SIZE[case["dtype"]] + SIZE[case["grad"]] + (8 - SIZE[case["dtype"]] if case["master"] else 0)
    # in 8 bits the two codes and what they stand for afterwards
    return {"bytes": n * (each + (16 if case["bits"] == 32 else 4 + 4)), "flops": 16 * n}


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "norm":
        n, d, res = case["rows"], case["d"], DTYPES[case["res"]]
        # a residual stream is larger than what a block adds to it, and has a few large channels
        loud = 1 + 20 * (torch.rand(d, generator=g, device=DEV) > 0.998).float()
        s["x"] = (2 * _randn(g, n, d) * loud).to(res)
        s["f"] = _randn(g, n, d).to(dtype)
        for w in ("w_post", "w_pre"):
            s[w] = (1 + 0.2 * _randn(g, d)).to(dtype)
        gates = {"none": 0, "one": 1, "seq": case["seqs"], "row": n}[case["gate"]]
        s["g"] = (0.5 + 0.3 * _randn(g, gates, d)).to(dtype) if gates else None
        s["scale"], s["eps"] = 0.7, 1e-6
        if case["backward"]:  # x is the stored sum then
            s["dr"], s["dh"] = (_randn(g, n, d)).to(res), (_randn(g, n, d)).to(dtype) if case["pre"] else None
        return s
    if case["op"] == "linear":
        hk, dk, dv = case["hk"], case["dk"], case["dv"]
        hq, lens = hk * case["group"], _lens(case)
        n = sum(lens)
        x = _randn(g, n, hq * dk + hk * (dk + dv)).to(dtype)  # one projection's output
        s["q"] = x[:, :hq * dk].unflatten(1, (hq, dk))
        s["k"] = x[:, hq * dk:(hq + hk) * dk].unflatten(1, (hk, dk))
        s["v"] = x[:, (hq + hk) * dk:].unflatten(1, (hk, dv))
        # memories from some four tokens to some thousand
        s["log_decay"] = -torch.exp2(-torch.linspace(2, 10, hk, device=DEV))
        s["state"] = _randn(g, case["batch"], hk, dk, dv)
        starts = [0]
        for m in lens:
            starts.append(starts[-1] + m)
        s["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        s["max_new"], s["scale"] = max(lens), dk ** -0.5
        if case["backward"]:
            s["do"] = _randn(g, n, hq, dv).to(dtype)
            s["d_state"] = _randn(g, case["batch"], hk, dk, dv)
        return s
    shapes = _shapes(case)
    at, total = _offsets(shapes)

    def tensors(flat):
        return [flat[a:a + math.prod(z)].view(z) for a, z in zip(at, shapes)]
    held = torch.zeros(total, dtype=torch.bool, device=DEV)
    for t in tensors(held):
        t.fill_(True)
    # gradients of a few sizes, as the tensors of a model have them
    size = torch.exp(torch.empty(total // 256, 1, device=DEV).uniform_(-9, -5, generator=g)).expand(-1, 256).reshape(-1)
    grad = torch.where(held, _randn(g, total) * size, 0.0)
    weight = torch.where(held, _randn(g, total) * 0.02, 0.0)
    s["flat_g"], s["flat_p"] = grad.to(DTYPES[case["grad"]]), weight.to(dtype)
    s["flat_master"] = weight if case["master"] else None
    m, v = 0.5 * torch.where(held, _randn(g, total) * size, 0.0), torch.where(held, size.square(), 0.0) * (0.5 + torch.rand(total, generator=g, device=DEV))
    s["total"] = total
    if case["bits"] == 32:
        s["state"] = torch.cat([m, v]).view(torch.uint8)
    else:
        s["state"] = torch.cat([x.view(torch.uint8) for x in _pack(m, v.sqrt())])
    s["params"], s["grads"] = tensors(s["flat_p"]), tensors(s["flat_g"])
    s["masters"] = tensors(s["flat_master"]) if case["master"] else None
    s["hyper"] = {"lr": 3e-4, "step": 1000, "betas": (0.9, 0.95), "eps": 1e-8, "weight_decay": 0.1}
    s["max_norm"] = 1.0 if case["clip"] else 0.0
    return s


# ------------------------------------------------------------------ plain forms


def _rms(x, eps):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)


def _gate(s):
    """The rows' gates, fp32: [rows, d], or broadcast over them."""
    if s["g"] is None:
        return 1.0
    return s["g"].float().repeat_interleave(s["rows"] // s["g"].shape[0], 0) if s["gate"] == "seq" else s["g"].float()


def _plain_norm(s):
    f = s["f"].float()
    if s["post"]:
        f = f * _rms(f, s["eps"]) * s["w_post"].float()
    r = (s["x"].float() + s["scale"] * _gate(s) * f).to(s["x"].dtype)
    out = {"r": r}
    if s["pre"]:
        y = r.float()
        out["h"] = (y * _rms(y, s["eps"]) * s["w_pre"].float()).to(s["f"].dtype)
    return out


def _plain_norm_backward(s):
    r, f, d = s["x"].float(), s["f"].float(), s["dr"].float()
    out = {}
    if s["pre"]:
        rho, dh = _rms(r, s["eps"]), s["dh"].float()
        t = dh * s["w_pre"].float()
        d = d + rho * (t - r * rho.square() * (r * t).mean(-1, keepdim=True))
        out["dpre"] = (dh * r * rho).sum(0)
    phi = _rms(f, s["eps"]) if s["post"] else 1.0
    n = f * phi * (s["w_post"].float() if s["post"] else 1.0)
    dn = s["scale"] * _gate(s) * d
    if s["g"] is not None and s["g"].shape[0] == s["rows"]:  # one a row: no sums
        out["dgate"] = (s["scale"] * n * d).to(s["g"].dtype)
    elif s["g"] is not None:
        out["dgate"] = (s["scale"] * n * d).unflatten(0, (s["g"].shape[0], -1)).sum(1)
    if s["post"]:
        u = dn * s["w_post"].float()
        out["dpost"] = (dn * f * phi).sum(0)
        dn = phi * (u - f * phi.square() * (f * u).mean(-1, keepdim=True))
    return out | {"dx": d.to(s["x"].dtype), "df": dn.to(s["f"].dtype)}


def _chunks(x, c):
    """[B, H, G, T, a] -> [B, H, T / c, G c, a]."""
    return x.unflatten(3, (-1, c)).permute(0, 1, 3, 2, 4, 5).flatten(3, 4).contiguous()


def _decayed(q, k, v, ld, state, lead, s_in, s_out, s_up):
    """Rows [B, H, G, T, .] (zero behind a sequence's end) in chunks: for row t the sum over j <= t of s_in g^(t - j)
    (q_t k_j) v_j, over every head of k, and s_out g^(t + lead) q_t state, the chunks' sums of s_up g^. k v^T with it."""
    t = q.shape[3]
    c = min(128, t)
    pad = (0, 0, 0, -t % c)
    q, k, v = (_chunks(torch.nn.functional.pad(x, pad), c) for x in (q, k, v))
    gq, gk, nc = q.shape[3] // c, k.shape[3] // c, q.shape[2]
    i = torch.arange(c, device=DEV, dtype=torch.float32)
    ld = ld[:, None]
    far = (i[:, None] - i).repeat(gq, gk)
    d = torch.where(far >= 0, torch.exp(ld[:, None] * far.clamp(min=0)), 0.0) * s_in  # [H, Gq c, Gk c]
    p = torch.matmul(q, k.transpose(3, 4).contiguous()) * d[:, None]
    o = torch.matmul(p, v)
    del p
    # the chunks' own sums, then what stands before each chunk
    up = torch.exp(ld * (c - lead - i)).repeat(1, gk) * s_up
    u = torch.matmul((k * up[:, None, :, None]).transpose(3, 4).contiguous(), v)  # [B, H, nc, a, b]
    n = torch.arange(nc, device=DEV, dtype=torch.float32)
    gap = n[:, None] - 1 - n
    w = torch.where(gap >= 0, torch.exp(ld[:, None] * c * gap.clamp(min=0)), 0.0)
    e = torch.matmul(w.expand(q.shape[0], -1, -1, -1), u.flatten(3)).unflatten(3, u.shape[3:])
    e += torch.exp(ld * c * n)[:, :, None, None] * state[:, :, None]
    row = torch.exp(ld * (i + lead)).repeat(1, gq) * s_out
    o = o + torch.matmul(q, e) * row[:, None, :, None]
    return o.unflatten(3, (gq, c)).permute(0, 1, 3, 2, 4, 5).flatten(3, 4)[:, :, :, :t]


def _whole(k, v, ld, lens, state, lead, scale):
    """g^len state + scale times the sum of g^(len - lead - t) k_t v_t^T, over every head of k [B, H, G, T, .]."""
    t = torch.arange(k.shape[3], device=DEV, dtype=torch.float32)
    far = (lens[:, None] - lead - t)[:, None]
    w = torch.where(far >= 0, torch.exp(ld[:, None] * far.clamp(min=0)), 0.0)[:, :, None, :, None]
    u = torch.matmul((k * w).flatten(2, 3).transpose(2, 3).contiguous(), v.flatten(2, 3).contiguous())
    return torch.exp(ld * lens[:, None])[:, :, None, None] * state + scale * u


def _rows_of(s, back):
    """For every sequence and index the row (from its end, if back), and whether there is one."""
    starts = s["q_starts"].long()
    lens = (starts[1:] - starts[:-1])[:, None]
    t = torch.arange(s["max_new"], device=DEV)
    at = starts[:-1, None] + (lens - 1 - t if back else t)
    return torch.where(t < lens, at, 0), t < lens


def _padded(s, x, back=False):
    """Rows [n, heads, a] as fp32 [B, hk, heads / hk, T, a]."""
    at, have = _rows_of(s, back)
    x = torch.where(have[:, :, None, None], x.float()[at], 0.0)
    return x.unflatten(2, (s["hk"], -1)).permute(0, 2, 3, 1, 4).contiguous()


def _unpadded(s, x, back=False):
    """The rows back in their places, [n, heads, a]."""
    starts = s["q_starts"].long()
    n = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(starts[1:], n, right=True)
    t = starts[b + 1] - 1 - n if back else n - starts[b]
    return x[b, :, :, t].flatten(1, 2)


def _plain_linear(s):
    ld, state, scale = s["log_decay"], s["state"], s["scale"]
    if s["max_new"] == 1:  # a token each: the recurrence itself
        k, v = s["k"].float(), s["v"].float()
        state.mul_(torch.exp(ld)[:, None, None]).add_(k[..., None] * v[:, :, None])
        o = scale * torch.matmul(s["q"].float().unflatten(1, (s["hk"], -1)), state)
        return {"o": o.flatten(1, 2).to(s["q"].dtype), "state": state}
    q, k, v = (_padded(s, s[n]) for n in ("q", "k", "v"))
    lens = (s["q_starts"][1:] - s["q_starts"][:-1]).float()
    o = _decayed(q, k, v, ld, state, 1, scale, scale, 1.0)
    state.copy_(_whole(k, v, ld, lens, state, 1, 1.0))
    return {"o": _unpadded(s, o).to(s["q"].dtype), "state": state}


def _plain_linear_backward(s):
    ld, state, d_state, scale, dtype = s["log_decay"], s["state"], s["d_state"], s["scale"], s["q"].dtype
    q, k, v, do = (_padded(s, s[n]) for n in ("q", "k", "v", "do"))
    turned = state.transpose(2, 3)
    dq = _unpadded(s, _decayed(do, v, k, ld, turned, 1, scale, scale, 1.0)).to(dtype)
    q, k, v, do = (_padded(s, s[n], True) for n in ("q", "k", "v", "do"))
    dk = _unpadded(s, _decayed(v, do, q, ld, d_state.transpose(2, 3), 0, scale, 1.0, scale), True).to(dtype)
    dv = _unpadded(s, _decayed(k, q, do, ld, d_state, 0, scale, 1.0, scale), True).to(dtype)
    lens = (s["q_starts"][1:] - s["q_starts"][:-1]).float()
    return {"dq": dq, "dk": dk, "dv": dv, "d_state0": _whole(q, do, ld, lens, d_state, 0, scale)}


def _pack(m, r):
    """Codes and scales of fp32 m and r [N]."""
    m, r = m.view(-1, 256), r.view(-1, 256)
    sm = (m.abs().amax(1, keepdim=True) / 448).clamp(min=2.0 ** -126)
    sr = (r.amax(1, keepdim=True) / 496).clamp(min=2.0 ** -126)
    y = r / sr
    e = (torch.frexp(y)[1] - 1).clamp(min=-6)  # 2^e <= y < 2^(e + 1), or the least normal's
    code = (e + 6) * 16 + torch.round(torch.ldexp(y, 4 - e)).int()
    code = torch.maximum(code, (r > 0).int())
    return ((m / sm).to(torch.float8_e4m3fn).view(torch.uint8).flatten(), code.to(torch.uint8).flatten(),
            sm.flatten(), sr.flatten())


def _parts(s):
    """The four parts of 8-bit states."""
    n = s["total"]
    x = s["state"]
    return x[:n], x[n:2 * n], x[2 * n:2 * n + n // 64].view(torch.float32), x[2 * n + n // 64:].view(torch.float32)


def _unpack(s):
    """fp32 m and r of 8-bit states."""
    m, r, sm, sr = _parts(s)
    c = r.int()
    y = torch.where(c < 16, torch.ldexp(c.float(), torch.full_like(c, -10)),
                    torch.ldexp((16 + (c & 15)).float(), (c >> 4) - 11))
    return ((m.view(torch.float8_e4m3fn).float().view(-1, 256) * sm[:, None]).flatten(),
            (y.view(-1, 256) * sr[:, None]).flatten())


def _plain_adamw(s):
    h, n, out = s["hyper"], s["total"], {}
    (b1, b2), lr = h["betas"], h["lr"]
    g = s["flat_g"].float()
    if s["max_norm"]:
        out["norm"] = g.square().sum().sqrt()
        g = g * (s["max_norm"] / out["norm"]).clamp(max=1.0)
    if s["bits"] == 32:
        m, v = s["state"].view(torch.float32).view(2, n)
    else:
        m, v = _unpack(s)
        v = v * v
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    p = s["flat_p"].float() if s["flat_master"] is None else s["flat_master"]
    den = v.sqrt() * (1 / math.sqrt(1 - b2 ** h["step"])) + h["eps"]
    p = p * (1 - lr * h["weight_decay"]) - m / den * (lr / (1 - b1 ** h["step"]))
    s["flat_p"].copy_(p)
    if s["flat_master"] is not None:
        s["flat_master"].copy_(p)
        out["master"] = s["flat_master"]
    if s["bits"] == 32:
        s["state"].view(torch.float32).view(2, n).copy_(torch.stack([m, v]))
        m, v = s["state"].view(torch.float32).view(2, n)
    else:
        for a, b in zip(_parts(s), _pack(m, v.sqrt())):
            a.copy_(b)
        m, v = _unpack(s)
        m, v = m.bfloat16(), (v * v).bfloat16()
    return out | {"p": s["flat_p"], "m": m, "v": v}


def _own(s):
    import test_layer_gate_amd as ttt
    if s["op"] == "norm":
        post, pre = s["w_post"] if s["post"] else None, s["w_pre"] if s["pre"] else None
        if s["backward"]:
            d = ttt.block_norm_backward(s["dr"], s["dh"], s["x"], s["f"], post=post, pre=pre, gate=s["g"],
                                        scale=s["scale"], eps=s["eps"])
            return {k: x for k, x in d.items() if x is not None}
        r, h = ttt.block_norm(s["x"], s["f"], post=post, pre=pre, gate=s["g"], scale=s["scale"], eps=s["eps"])
        return {"r": r, "h": h} if s["pre"] else {"r": r}
    if s["op"] == "linear":
        if s["backward"]:
            dq, dk, dv, d0 = ttt.linear_attention_backward(
                s["do"], s["q"], s["k"], s["v"], s["log_decay"], state=s["state"], d_state=s["d_state"],
                q_starts=s["q_starts"], max_new=s["max_new"], scale=s["scale"])
            return {"dq": dq, "dk": dk, "dv": dv, "d_state0": d0}
        o = ttt.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], state=s["state"], q_starts=s["q_starts"],
                                 max_new=s["max_new"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    out = {}
    if s["max_norm"]:
        out["norm"] = ttt.grad_norm(s["grads"])
    ttt.adamw_step(s["params"], s["grads"], s["state"], bits=s["bits"], masters=s["masters"], norm=out.get("norm"),
                   max_norm=s["max_norm"], **s["hyper"])
    m, v = ttt.adamw_read(s["state"], s["bits"], dtype=torch.float32 if s["bits"] == 32 else torch.bfloat16)
    if s["flat_master"] is not None:
        out["master"] = s["flat_master"]
    return out | {"p": s["flat_p"], "m": m, "v": v}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "norm":
        return _plain_norm_backward(s) if s["backward"] else _plain_norm(s)
    if s["op"] == "linear":
        return _plain_linear_backward(s) if s["backward"] else _plain_linear(s)
    return _plain_adamw(s)


# ------------------------------------------------------------------ in 64 bits


def _exact_norm(s):
    """Block of rows by block; the gradients by the chain rule through x / |x|."""
    eps, scale, out = s["eps"], s["scale"], {}
    d = s["d"]
    sums = {k: torch.zeros(d, dtype=torch.float64, device=DEV) for k in ("dpre", "dpost")}
    gates = None if s["g"] is None else s["g"].shape[0]
    sums["dgate"] = None if gates is None else torch.zeros(gates, d, dtype=torch.float64, device=DEV)
    w_post, w_pre = s["w_post"].double(), s["w_pre"].double()
    parts = {}
    for a in range(0, s["rows"], 4096):
        rows = torch.arange(a, min(a + 4096, s["rows"]), device=DEV)
        x, f = s["x"][rows].double(), s["f"][rows].double()
        which = None if gates is None else rows * gates // s["rows"]
        gate = torch.ones((), dtype=torch.float64, device=DEV) if gates is None else s["g"].double()[which]
        length = torch.sqrt((f * f).sum(-1, keepdim=True) / d + eps)
        unit = f / length
        n = unit * w_post if s["post"] else f
        got = {}
        if not s["backward"]:
            r = x + scale * gate * n
            got["r"] = r
            r = r.to(s["x"].dtype).double()  # h is of the sum as it is stored
            if s["pre"]:
                got["h"] = w_pre * r / torch.sqrt((r * r).sum(-1, keepdim=True) / d + eps)
        else:
            dr = s["dr"][rows].double()
            if s["pre"]:
                dh = s["dh"][rows].double()
                size = torch.sqrt((x * x).sum(-1, keepdim=True) / d + eps)
                u = x / size
                dr = dr + (dh * w_pre - u * ((dh * w_pre * u).sum(-1, keepdim=True) / d)) / size
                sums["dpre"] += (dh * u).sum(0)
            got["dx"] = dr
            if gates is not None:
                sums["dgate"].index_add_(0, which, scale * dr * n)
            dn = scale * gate * dr
            if s["post"]:
                sums["dpost"] += (dn * unit).sum(0)
                dn = (dn * w_post - unit * ((dn * w_post * unit).sum(-1, keepdim=True) / d)) / length
            got["df"] = dn
        for k, v in got.items():
            parts.setdefault(k, []).append(v)
    out = {k: torch.cat(v) for k, v in parts.items()}
    if s["backward"]:
        out |= {"dpre": sums["dpre"]} if s["pre"] else {}
        out |= {"dpost": sums["dpost"]} if s["post"] else {}
        out |= {"dgate": sums["dgate"]} if gates is not None else {}
    return out


def _exact_linear(s):
    """Every pair of rows of a head, without states: o = scale (q k^T . decays) v and what the first state gives."""
    q, k, v, ld = s["q"].double(), s["k"].double(), s["v"].double(), s["log_decay"].double()
    n, scale, group, starts = q.shape[0], s["scale"], s["group"], s["q_starts"].tolist()
    s0 = s["state"].double()
    z = {m: torch.zeros(t.shape, dtype=torch.float64, device=DEV) for m, t in (("q", q), ("k", k), ("v", v))}
    o = torch.zeros(n, q.shape[1], s["dv"], dtype=torch.float64, device=DEV)
    end = torch.zeros_like(s0)
    for b, (lo, hi) in enumerate(zip(starts, starts[1:])):
        for h in range(s["hk"]):
            t = torch.arange(hi - lo, dtype=torch.float64, device=DEV)
            kk, vv, first = k[lo:hi, h], v[lo:hi, h], s0[b, h]
            at = torch.exp(ld[h] * (t + 1))[:, None]
            left = torch.exp(ld[h] * (hi - lo - 1 - t))[:, None]  # of a row's product at the end
            if s["backward"]:
                dlast = s["d_state"][b, h].double()
                end[b, h] = torch.exp(ld[h] * (hi - lo)) * dlast
                z["k"][lo:hi, h] += left * (vv @ dlast.T)
                z["v"][lo:hi, h] += left * (kk @ dlast)
            else:
                end[b, h] = torch.exp(ld[h] * (hi - lo)) * first + (left * kk).T @ vv
            for i in range(0, hi - lo, 2048):
                j = min(i + 2048, hi - lo)
                d = torch.exp(ld[h] * (t[i:j, None] - t[:j]).clamp(min=0)).tril_(i) * scale
                for c in range(h * group, (h + 1) * group):
                    qq = q[lo + i:lo + j, c]
                    p = (qq @ kk[:j].T) * d
                    if not s["backward"]:
                        o[lo + i:lo + j, c] = p @ vv[:j] + scale * at[i:j] * (qq @ first)
                        continue
                    do = s["do"][lo + i:lo + j, c].double()
                    dp = (do @ vv[:j].T) * d
                    z["q"][lo + i:lo + j, c] = dp @ kk[:j] + scale * at[i:j] * (do @ first.T)
                    z["k"][lo:lo + j, h] += dp.T @ qq
                    z["v"][lo:lo + j, h] += p.T @ do
                    end[b, h] += scale * (at[i:j] * qq).T @ do
    if s["backward"]:
        return {"dq": z["q"], "dk": z["k"], "dv": z["v"], "d_state0": end}
    return {"o": o, "state": end}


def _nearest(y, values):
    """The nearest of ascending `values`, ties to the even index."""
    hi = torch.searchsorted(values, y).clamp(1, len(values) - 1)
    lo = hi - 1
    up, down = values[hi] - y, y - values[lo]
    return values[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]


def _exact_adamw(s):
    h, n, out = s["hyper"], s["total"], {}
    b1, b2 = h["betas"]
    e4m3 = torch.tensor([math.ldexp(c % 8 + 8 * (c >= 8), max(c // 8, 1) - 10) for c in range(127)], dtype=torch.float64, device=DEV)
    e4m4 = torch.tensor([math.ldexp(c % 16 + 16 * (c >= 16), max(c // 16, 1) - 11) for c in range(256)], dtype=torch.float64, device=DEV)
    g = s["flat_g"].double()
    if s["max_norm"]:
        out["norm"] = torch.linalg.vector_norm(g)
        g = g * min(1.0, s["max_norm"] / float(out["norm"]))
    if s["bits"] == 32:
        m, v = s["state"].view(torch.float32).double().view(2, n)
    else:
        cm, cr, sm, sr = (x.long() if x.dtype == torch.uint8 else x.double().repeat_interleave(256) for x in _parts(s))
        m = e4m3[(cm & 127).clamp(max=126)] * (1 - 2 * (cm >> 7)) * sm
        v = (e4m4[cr] * sr) ** 2
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    p = (s["flat_p"] if s["flat_master"] is None else s["flat_master"]).double()
    step = (m / (1 - b1 ** h["step"])) / (torch.sqrt(v / (1 - b2 ** h["step"])) + h["eps"])
    p = p - h["lr"] * (h["weight_decay"] * p + step)
    if s["bits"] == 8:
        mb, rb = m.view(-1, 256), v.sqrt().view(-1, 256)
        sm = (mb.abs().amax(1, keepdim=True) / 448).float().double().clamp(min=2.0 ** -126)
        sr = (rb.amax(1, keepdim=True) / 496).float().double().clamp(min=2.0 ** -126)
        m = (_nearest((mb / sm).abs(), e4m3) * torch.sign(mb) * sm).flatten()
        r = torch.where(rb > 0, _nearest(rb / sr, e4m4).clamp(min=float(e4m4[1])), 0.0) * sr
        v = (r * r).flatten()
    if s["flat_master"] is not None:
        out["master"] = p
    return out | {"p": p, "m": m, "v": v}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "adamw": _exact_adamw}[s["op"]](s)
