"""The example of a trained block (norms, linear attention, fast-weight layer,
AdamW) on the GPU: its gradients against the chain of float64 oracles, and its
steps against the oracle's AdamW of those gradients. The chain itself is held
against differences on the CPU.

Tolerance, relative in the 2-norm. fp32: the layer's backward takes bf16 operands,
a few roundings of 2^-9 along its chain, 2e-2 at most as in its own tests; all
other kernels and products are fp32's. bf16: some 20 roundings of rms 2^-9.6
forwards and backwards, amplified at most as the layer's fifth power: sqrt(20)
1.3e-3 5 = 2.9e-2, and the layer's own 2e-2: 5e-2."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle.block_oracle as bo
import oracle.ttt_oracle as ora

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EPS = 1e-6


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def host(t):
    return t.detach().double().cpu().numpy()


def forward(w, x, decay, eta, chunk, heads, kv_heads, dim):
    B, T, d = x.shape
    n = bo.pre_norm(x, w["norm1"], EPS)
    qkv = (n @ w["Wqkv"].T).reshape(B, T, -1, dim)
    parts = [np.split(qkv[b], [heads, heads + kv_heads], 1) for b in range(B)]
    o = np.stack([bo.linear(*p, decay, dim ** -0.5)[0] for p in parts]).reshape(B, T, -1)
    f = o @ w["Wo"].T
    x1 = x + f
    n2 = bo.pre_norm(x1, w["norm2"], EPS)
    y2, _ = ora.ttt_prefill(
        n2, x, w["Wg"], w["Wu"], w["W_down0"], w["taps"], w["W_target"], eta, chunk)
    return x1 + y2, (n, parts, o, f, x1, n2)


def reference(w, x, target, decay, eta, chunk, heads, kv_heads, dim):
    """loss, gradients of w and x."""
    B, T, d = x.shape
    y, (n, parts, o, f, x1, n2) = forward(w, x, decay, eta, chunk, heads, kv_heads, dim)
    dy = (y - target) / (B * T)
    loss = ((y - target) ** 2).sum() / (2 * B * T)
    g = ora.ttt_prefill_backward(n2, x, w["Wg"], w["Wu"], w["W_down0"], w["taps"], w["W_target"], eta, chunk, dy)
    b = bo.norm_backward(dy, g.pop("dH"), x1, f, None, w["norm2"], None, 1.0, EPS, False, True)
    dx0 = g.pop("dX0")
    g["dnorm2"] = b["dpre"].sum((0, 1))
    g["dWo"] = np.einsum("btd,bto->do", b["df"], o)
    do = (b["df"] @ w["Wo"]).reshape(B, T, heads, dim)
    dqkv = np.stack([np.concatenate(bo.linear_backward(do[i], *parts[i], decay, dim ** -0.5)[:3], 1)
                     for i in range(B)]).reshape(B, T, -1)
    g["dWqkv"] = np.einsum("bto,btd->od", dqkv, n)
    b = bo.norm_backward(b["dx"], dqkv @ w["Wqkv"], x, None, None, w["norm1"], None, 1.0, EPS, False, True)
    g["dnorm1"] = b["dpre"].sum((0, 1))
    return loss, {k: g["d" + k] for k in w}, b["dx"] + dx0


def test_the_chain_of_oracles_against_differences():
    rng = np.random.default_rng(5)
    B, T, d, f, heads, kv_heads, dim, chunk = 2, 8, 6, 10, 4, 2, 4, 4

    def t(*s, by=0.4):
        return rng.standard_normal(s) * by
    w = dict(Wqkv=t(32, d), Wo=t(d, 16), norm1=1 + t(d), norm2=1 + t(d), Wg=t(f, d), Wu=t(f, d), W_down0=t(d, f),
             taps=t(3, d), W_target=t(d, d))
    x, target = t(B, T, d, by=1), t(B, T, d, by=1)
    rest = (np.array([0.9, 0.6]), 0.1, chunk, heads, kv_heads, dim)
    _, g, dx = reference(w, x, target, *rest)

    def loss(w, x):
        return ((forward(w, x, *rest)[0] - target) ** 2).sum() / (2 * B * T)
    for k in w:
        D, h = t(*w[k].shape, by=1), 1e-5
        slope = (loss({**w, k: w[k] + h * D}, x) - loss({**w, k: w[k] - h * D}, x)) / (2 * h)
        assert abs(slope - (g[k] * D).sum()) <= 1e-7 * (1 + abs(slope)), k
    D = t(*x.shape, by=1)
    slope = (loss(w, x + 1e-5 * D) - loss(w, x - 1e-5 * D)) / 2e-5
    assert abs(slope - (dx * D).sum()) <= 1e-7 * (1 + abs(slope))


@pytest.mark.gpu
@pytest.mark.parametrize("config,T,heads,kv_heads,dim,bits,tol", [
    ("tiny", 192, 4, 2, 64, 32, 2e-2), ("tiny", 256, 2, 2, 128, 8, 2e-2), ("mid_amp", 768, 4, 1, 64, 8, 5e-2)])
def test_gradients_and_steps(example, config, T, heads, kv_heads, dim, bits, tol):
    block, x = example.random_block(config, 2, T, heads, kv_heads, dim, seed=4, bits=bits)
    target = torch.roll(x, -1, 1)
    rest = (np.exp(host(block.log_decay)), block.eta, block.chunk, heads, kv_heads, dim)
    loss, got, dx = block.gradients(x, target)
    w = {k: host(v) for k, v in block.w.items()}
    want_loss, want, want_dx = reference(w, host(x), host(target), *rest)
    errs = {k: np.linalg.norm(host(got[k]) - want[k]) / np.linalg.norm(want[k]) for k in want}
    errs["x"] = np.linalg.norm(host(dx) - want_dx) / np.linalg.norm(want_dx)
    print(f"{config}: " + "  ".join(f"{k} {e:.1e}" for k, e in errs.items()), flush=True)
    assert abs(float(loss) / want_loss - 1) <= tol
    assert max(errs.values()) <= tol, errs

    # a step from fresh states, of the block's own gradients: what the weights
    # become is AdamW's, whose update of step 1 is lr sign(g) where |g| >> eps
    masters = list(map(host, block.masters or block.w.values()))
    norm = np.sqrt(sum((host(v) ** 2).sum() for v in got.values()))
    kw = dict(lr=1e-3, max_norm=0.5 * norm, betas=(0.9, 0.99), weight_decay=0.1)
    assert torch.equal(block.step(x, target, **kw), loss)
    for p, before, g, held in zip(block.masters or block.w.values(), masters, got.values(), block.w.values()):
        ref = bo.adamw(before, 0.5 * host(g), 0.0, 0.0, 1e-3, 1, 0.9, 0.99, 1e-8, 0.1)[0]
        # two roundings of p, some 20 of an update of at most lr
        assert (np.abs(host(p) - ref) <= 2.0 ** -22 * (np.abs(before) + 20e-3)).all()
        assert torch.equal(held, p.to(held.dtype))
    for _ in range(2):
        assert torch.isfinite(block.step(x, target, **kw))
