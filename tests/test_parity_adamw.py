"""GPU parity of the AdamW step, its states in 32 and 8 bits, and the
gradients' norm, against the float64 oracle.

Tolerances, u = 2^-24. m and v are two rounded products, of factors that are
rounded themselves, and their sum: 4 u of its magnitudes. The update m / (sqrt(v)
rs + eps) a: 10 roundings, those of m and v with it; p k - update: 2 more of p. A
bf16 weight adds half a step, 2^-8. An 8-bit value is within half a step of its
code's grid (its block's scale rounded), which the oracle gives; codes decode
exactly. The norm: sums in 64 bits, rounded once, the root once."""
import math

import numpy as np
import pytest
import torch

import oracle.block_oracle as bo

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def host(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def make(sizes, dtype, grad, masters, seed=0):
    rng = np.random.default_rng(seed)
    ms = [torch.from_numpy(rng.standard_normal(n)).float().cuda() for n in sizes]
    ps = [m.to(dtype) if dtype == BF else m for m in ms]
    gs = [torch.from_numpy(rng.standard_normal(n) * math.exp(rng.uniform(-12, 2))).to(grad).cuda() for n in sizes]
    return ps, gs, (ms if masters else None)


def parts(flat, sizes):
    at = 0
    for n in sizes:
        yield flat[at:at + n]
        at += -(-n // 256) * 256


def held_states(ttt, state, bits):
    """(m, v) float64 of the whole buffer."""
    if bits == 32:
        return tuple(map(host, ttt.adamw_read(state)))
    m, r = bo.read_states(state.cpu().numpy(), state.numel() // 520 * 256)
    return m, r * r


def check_steps(ttt, sizes, dtype, grad, masters, bits, steps=3, clip=0.0, **kw):
    ps, _, ms = make(sizes, dtype, grad, masters)
    state = ttt.adamw_state(ps, bits)
    assert state.numel() == ttt.adamw_state_size(sizes, bits)
    for step in range(1, steps + 1):
        gs = make(sizes, dtype, grad, masters, seed=step)[1]
        before = [host(p) for p in (ms or ps)]
        m0, v0 = held_states(ttt, state, bits)
        norm = ttt.grad_norm(gs) if clip else None
        c = 1.0
        if clip:
            want = math.sqrt(sum(float((host(g) ** 2).sum()) for g in gs))
            assert abs(float(norm) - want) <= 2 * U * want
            c = min(1.0, clip / want)
        ttt.adamw_step(ps, gs, state, step=step, bits=bits, masters=ms, norm=norm, max_norm=clip, **HYPER, **kw)
        m1, v1 = held_states(ttt, state, bits)
        ref_m, ref_r = np.zeros_like(m0), np.zeros_like(m0)
        for i, (g, m, v, rm, rr) in enumerate(zip(gs, parts(m0, sizes), parts(v0, sizes), parts(ref_m, sizes), parts(ref_r, sizes))):
            b1, b2 = HYPER["betas"]
            gh = c * host(g)
            p, m2, v2, u = bo.adamw(before[i], gh, m, v, HYPER["lr"], step, b1, b2, HYPER["eps"], HYPER["weight_decay"])
            rm[:], rr[:] = m2, np.sqrt(v2)
            ms_size = b1 * np.abs(m) + (1 - b1) * np.abs(gh)
            u_room = 12 * U * np.abs(u) * np.where(m2 != 0, ms_size / np.maximum(np.abs(m2), 1e-300), 1) + 2.0 ** -126
            room = 3 * U * np.abs(before[i]) + 8 * u_room
            if ms:
                assert (np.abs(host(ms[i]) - p) <= room).all(), i
                assert torch.equal(ps[i], ms[i].to(BF))
            else:
                half = 2.0 ** -8 * np.abs(p) if dtype == BF else 0.0
                assert (np.abs(host(ps[i]) - p) <= room + half).all(), i
        # (a tensor's states, of zeros behind its end)
        for x1, ref, most, bits_, least, size in ((m1, ref_m, 448, 3, 2.0 ** -9, 4), (np.sqrt(v1), ref_r, 496, 4, 2.0 ** -10, 8)):
            room = 2 * size * U * np.maximum(np.abs(ref), np.abs(m0) if x1 is m1 else 0)
            if bits == 8:
                half = bo.held(ref, most, bits_, least)
                # an r above 0 that would round to 0 takes the least code
                room = room + half * (1 + 2.0 ** -20) + (np.where((ref > 0) & (ref < half * (1 + 2.0 ** -20)), half, 0) if x1 is not m1 else 0)
            else:
                room = room + 4 * U * np.abs(ref)
            if x1 is m1:
                g_size = np.zeros_like(ref)
                for i, part in enumerate(parts(g_size, sizes)):
                    part[:] = np.abs(c * host(gs[i])) * (1 - HYPER["betas"][0])
                room = room + 8 * U * g_size
            assert (np.abs(x1 - ref) <= room + 2.0 ** -126).all(), (bits, most, float((np.abs(x1 - ref) - room).max()))
    return ps, ms, state


SIZES = [1, 7, 255, 256, 257, 2047, 2048, 2049, 5000]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,grad,masters", [(BF, BF, False), (BF, F32, False), (BF, BF, True), (BF, F32, True), (F32, F32, False),
                                                (F32, BF, False)])
def test_steps(ttt, bits, dtype, grad, masters):
    check_steps(ttt, SIZES, dtype, grad, masters, bits)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(ttt, bits):
    """More than one launch takes, empty ones among them, limited by the norm."""
    check_steps(ttt, [0, 3] + [17 * i % 700 for i in range(150)] + [0], BF, F32, False, bits, clip=0.5)


def test_the_norm_limits_and_does_not_lift(ttt):
    for clip in (1e-3, 1e6):
        check_steps(ttt, [300, 5], F32, F32, False, 32, clip=clip)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_norm_that_is_not_finite_changes_nothing(ttt, bad, bits):
    ps, gs, ms = make([300, 40], BF, F32, True)
    state = ttt.adamw_state(ps, bits)
    ttt.adamw_step(ps, gs, state, step=1, bits=bits, masters=ms, **HYPER)
    keep = [t.clone() for t in (*ps, *ms, state)]
    gs[1][7] = bad
    norm = ttt.grad_norm(gs)
    assert not torch.isfinite(norm)
    ttt.adamw_step(ps, gs, state, step=2, bits=bits, masters=ms, norm=norm, max_norm=1.0, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(keep, (*ps, *ms, state)))


def test_a_nan_takes_its_block_of_8_bits_and_no_more(ttt):
    ps, gs, _ = make([700], F32, F32, False)
    for bad in (float("nan"), float("inf")):
        state = ttt.adamw_state(ps, 8)
        g = gs[0].clone()
        g[300] = bad
        ttt.adamw_step([ps[0].clone()], [g], state, step=1, bits=8, **HYPER)
        m, v = ttt.adamw_read(state, 8)
        assert torch.isnan(m[256:512]).all() and torch.isnan(v[256:512]).all()
        assert torch.isfinite(m[:256]).all() and torch.isfinite(v[512:]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_code_reads_exactly(ttt, dtype):
    n = 512
    state = torch.zeros(2 * n + 2 * n // 256 * 4, dtype=torch.uint8)
    state[:n] = state[n:2 * n] = torch.arange(n) % 256
    state[2 * n:].view(F32).copy_(torch.tensor([1.0, 2.0 ** -20, 1.0, 2.0 ** 10]))
    m, v = ttt.adamw_read(state.cuda(), 8, dtype=dtype)
    rm, rr = bo.read_states(state.numpy(), n)
    assert np.array_equal(host(m), torch.from_numpy(rm).to(dtype).double().numpy(), equal_nan=True)
    assert np.array_equal(host(v), torch.from_numpy(rr * rr).to(dtype).double().numpy())


def test_a_block_that_only_decays_keeps_its_codes(ttt):
    """Without gradients the scales fall and the codes stay, where rounding to a
    fixed grid would hold values whose decay is less than half a step."""
    p, g, _ = make([512], F32, F32, False)
    state = ttt.adamw_state(p, 8)
    ttt.adamw_step(p, g, state, step=1, bits=8, **HYPER)
    codes, v0 = state[:1024].clone(), ttt.adamw_read(state, 8)[1]
    for step in range(2, 60):
        ttt.adamw_step(p, [torch.zeros_like(g[0])], state, step=step, bits=8, lr=0.0, betas=(0.9, 0.999), eps=1e-8)
    assert torch.equal(state[512:1024], codes[512:])
    v1 = ttt.adamw_read(state, 8)[1]
    kept = v0 > v0.max() * 1e-6
    assert torch.allclose(v1[kept] / v0[kept], torch.full_like(v1[kept], 0.999 ** 58), rtol=1e-4)


def test_far_from_one(ttt):
    """Gradients whose squares leave fp32's range, and none at all."""
    p = [torch.ones(300, device="cuda"), torch.ones(300, device="cuda")]
    g = [torch.full((300,), 1e-30, device="cuda"), torch.zeros(300, device="cuda")]
    for bits in (32, 8):
        q = [t.clone() for t in p]
        ttt.adamw_step(q, g, ttt.adamw_state(q, bits), step=1, bits=bits, lr=1e-3, eps=1e-8)
        assert torch.isfinite(q[0]).all() and torch.equal(q[1], p[1])
    big = [torch.full((5,), 1e30, device="cuda")]
    assert abs(float(ttt.grad_norm(big)) / (1e30 * math.sqrt(5)) - 1) < 1e-6


def test_captured_with_step_and_rate_on_the_gpu(ttt):
    sizes = [1000, 257]
    ps, gs, _ = make(sizes, F32, F32, False)
    eager = [p.clone() for p in ps]
    state, estate = ttt.adamw_state(ps, 8), ttt.adamw_state(ps, 8)
    step, lr = torch.ones((), dtype=torch.int32, device="cuda"), torch.full((), 1e-2, device="cuda")
    held = [g.clone() for g in gs]

    def call():
        norm = ttt.grad_norm(held)
        ttt.adamw_step(ps, held, state, lr=lr, step=step, betas=(0.9, 0.95), weight_decay=0.1, bits=8, norm=norm, max_norm=0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in range(1, 5):
        new = make(sizes, F32, F32, False, seed=n)[1]
        for a, b in zip(held, new):
            a.copy_(b)
        step.fill_(n)
        lr.fill_(1e-2 / n)
        graph.replay()
        before = [e.clone() for e in eager]
        ttt.adamw_step(eager, new, estate, lr=1e-2 / n, step=n, betas=(0.9, 0.95), weight_decay=0.1, bits=8,
                       norm=ttt.grad_norm(new), max_norm=0.5)
        torch.cuda.synchronize()
        # the two corrections are computed in 32 bits on the GPU, in 64 on the host
        for a, b, c in zip(ps, eager, before):
            assert (a - b).abs().max() <= 2.0 ** -18 * (b - c).abs().max() + 2.0 ** -22
        for a, b in zip(ps, eager):
            a.copy_(b)
        state.copy_(estate)


def test_on_another_stream(ttt):
    ps, gs, _ = make(SIZES, BF, BF, False)
    want = [p.clone() for p in ps]
    ttt.adamw_step(want, gs, ttt.adamw_state(want, 8), step=3, bits=8, **HYPER)
    side = torch.cuda.Stream()
    state = ttt.adamw_state(ps, 8)
    side.wait_stream(torch.cuda.current_stream())
    norm = ttt.grad_norm(gs, stream=side)
    ttt.adamw_step(ps, gs, state, step=3, bits=8, norm=norm, max_norm=1e9, stream=side, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ps, want))
