"""GPU parity of the norms before and after a block, their gate and residual
scale, and their gradients, against the float64 oracle.

Tolerances, u = 2^-24. A sum of d squares: each lane adds at most 32 values of
fp32, the wave 6 times, at most 16 waves: 54 roundings, all terms positive, so
within 54 u; its root half of that, with the division, the root and the products
40 u of a normed value. r: those of the other part, and of the sum. A bf16 result
adds half a step, 2^-8 of the value. h is compared with the norm of the stored r.
Gradients: dx and df are differences of three terms, each within 64 u of its
magnitude where sums of d terms with signs enter (54 roundings of the sum of
magnitudes). Sums over n rows: n more roundings of the sum of magnitudes, at
most."""
import numpy as np
import pytest
import torch

import oracle.block_oracle as bo

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def host(t):
    return t.detach().double().cpu().numpy()


def tensor(rng, *shape, dtype=BF):
    return torch.from_numpy(rng.standard_normal(shape)).to(dtype).cuda()


def near(got, ref, room, what):
    got = host(got).reshape(ref.shape)
    room = room + (2.0 ** -8 * np.abs(ref) if what[1] == BF else 0.0)
    bad = ~(np.abs(got - ref) <= room + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - ref)[bad].max()))


def gate_rows(gate, rows):
    return None if gate is None else np.repeat(host(gate).reshape(-1, gate.shape[-1]), rows // max(1, gate.numel() // gate.shape[-1]), 0)


def check_forward(ttt, x, f, post, pre, gate, scale, eps, **kw):
    rows, d = x.numel() // x.shape[-1], x.shape[-1]
    r, h = ttt.block_norm(x, f, post=post, pre=pre, gate=gate, scale=scale, eps=eps, **kw)
    xh, at = host(x).reshape(rows, d), (lambda w: None if w is None or w is True else host(w))
    if f is not None:
        ref, size = bo.residual(xh, host(f).reshape(rows, d), at(post), gate_rows(gate, rows), scale, eps, post is not None)
        near(r, ref, 48 * U * size, ("r", x.dtype))
        xh = host(r).reshape(rows, d)
    if pre is not None:
        ref = bo.pre_norm(xh, at(pre), eps)
        near(h, ref, 48 * U * np.abs(ref), ("h", h.dtype))
    else:
        assert h is None
    return r, h


# each width's lanes, vectors and waves: a part of a wave, whole waves, both vectors of a lane, the widest
@pytest.mark.parametrize("d", [8, 16, 504, 512, 520, 1000, 2560, 4096, 4104, 8192, 8200, 16384])
@pytest.mark.parametrize("dtype,res", [(BF, BF), (BF, F32), (F32, F32)])
def test_forward_widths(ttt, d, dtype, res):
    rng = np.random.default_rng(d)
    rows = 5
    x, f = tensor(rng, rows, d, dtype=res), tensor(rng, rows, d, dtype=dtype)
    check_forward(ttt, x, f, tensor(rng, d, dtype=dtype), tensor(rng, d, dtype=dtype), tensor(rng, 1, d, dtype=dtype), 0.7, 1e-6)


@pytest.mark.parametrize("parts", ["r", "rp", "rq", "rpq", "rg", "rpqg", "q", "Q", "PQ"])
@pytest.mark.parametrize("rows", [1, 7])
def test_forward_parts(ttt, parts, rows):
    """p: norm behind the block, q: before the next, P, Q: without a weight, g: a gate, r: a block at all."""
    rng = np.random.default_rng(rows)
    d = 264
    x = tensor(rng, rows, d)
    f = tensor(rng, rows, d) if "r" in parts or "P" in parts else None
    w = {c: tensor(rng, d) if c in parts else True if c.upper() in parts else None for c in "pq"}
    check_forward(ttt, x, f, w["p"], w["q"], tensor(rng, rows, d) if "g" in parts else None, -1.5, 0.5)


def test_forward_gates_and_layouts(ttt):
    rng = np.random.default_rng(1)
    B, T, d = 3, 4, 72
    wide = tensor(rng, B, T, 3 * d)
    x, f = wide[..., :d], wide[..., 2 * d:]                 # parts of wider rows
    for gate in (tensor(rng, d), tensor(rng, B, 1, d), tensor(rng, B, T, d), tensor(rng, 6, 2 * d)[:, d:],
                 tensor(rng, 1, d).expand(12, d)):
        check_forward(ttt, x, f, True, tensor(rng, d, dtype=F32), gate, 1.0, 1e-6)
    x = tensor(rng, 12, d)
    keep = x.clone()
    r, h = ttt.block_norm(x, f.reshape(12, d), pre=True, r=x)
    assert r is x
    want = ttt.block_norm(keep, f.reshape(12, d), pre=True)
    assert torch.equal(r, want[0]) and torch.equal(h, want[1])
    out = torch.full((12, 2 * d), 7.0, dtype=BF, device="cuda")
    ttt.block_norm(keep, f.reshape(12, d), pre=True, r=out[:, :d], h=torch.empty_like(keep))
    assert torch.equal(out[:, :d], want[0]) and (out[:, d:] == 7).all()


def test_extreme_rows(ttt):
    """Rows of zeros, of the largest values, and a NaN: its row alone."""
    x = torch.zeros(4, 64, device="cuda")
    x[1] = 1e18
    x[2, 5] = float("nan")
    h = ttt.block_norm(x, pre=True, eps=1e-6)[1]
    assert (h[0] == 0).all() and torch.allclose(h[1], torch.ones_like(h[1]), rtol=1e-6)
    assert torch.isnan(h[2]).all() and (h[3] == 0).all()
    e = ttt.block_norm(torch.zeros(0, 64, device="cuda"), torch.zeros(0, 64, device="cuda"), pre=True)
    assert e[0].shape == (0, 64)


def check_backward(ttt, rows, d, dtype, res, post, pre, gates, dr=True, f=True, w_dtype=None, scale=0.7, eps=1e-6, **kw):
    rng = np.random.default_rng(rows * 7 + d)
    w_dtype = w_dtype or dtype
    r, fv = tensor(rng, rows, d, dtype=res), tensor(rng, rows, d, dtype=dtype) if f else None
    post, pre = (tensor(rng, d, dtype=w_dtype) if w == 1 else True if w else None for w in (post, pre))
    gate = tensor(rng, gates, d, dtype=dtype) if gates else None
    dr = tensor(rng, rows, d, dtype=res) if dr else None
    dh = tensor(rng, rows, d, dtype=dtype) if pre is not None else None
    got = ttt.block_norm_backward(dr, dh, r if pre is not None else None, fv, post=post, pre=pre, gate=gate, scale=scale,
                                  eps=eps, dx=torch.empty_like(r) if dr is None else None, **kw)
    at = (lambda w: None if w is None or w is True else host(w))
    ref = bo.norm_backward(np.zeros((rows, d)) if dr is None else host(dr), None if dh is None else host(dh), host(r),
                           None if fv is None else host(fv), at(post), at(pre), gate_rows(gate, rows), scale, eps,
                           post is not None, pre is not None)
    near(got["dx"], ref["dx"], 128 * U * ref["dx_size"], ("dx", res))
    if f:
        near(got["df"], ref["df"], 192 * U * ref["df_size"], ("df", dtype))
    if gates == rows:
        near(got["dgate"], ref["dgate"], 192 * U * ref["dgate_size"], ("dgate", dtype))
    elif gates:
        many = rows // gates
        cut = (lambda a: a.reshape(gates, many, d).sum(1))
        near(got["dgate"], cut(ref["dgate"]), (192 + many) * U * cut(ref["dgate_size"]), ("dgate", F32))
    if at(post) is not None:
        near(got["dpost"], ref["dpost"].sum(0), (192 + rows) * U * ref["dpost_size"].sum(0), ("dpost", F32))
    if at(pre) is not None:
        near(got["dpre"], ref["dpre"].sum(0), (64 + rows) * U * np.abs(ref["dpre"]).sum(0), ("dpre", F32))
    return got


@pytest.mark.parametrize("d", [8, 512, 520, 2560, 4096, 8192, 8200, 16384])
@pytest.mark.parametrize("dtype,res", [(BF, BF), (BF, F32), (F32, F32)])
def test_backward_widths(ttt, d, dtype, res):
    check_backward(ttt, 12, d, dtype, res, 1, 1, 3)


@pytest.mark.parametrize("post", [0, 1, 2])
@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("gates", [0, 1, 6, 18])
def test_backward_parts(ttt, post, pre, gates):
    check_backward(ttt, 18, 136, BF, F32, post, pre, gates, w_dtype=F32)


def test_backward_without_a_block_or_dr(ttt):
    check_backward(ttt, 9, 64, BF, BF, 0, 1, 0, f=False)
    check_backward(ttt, 9, 64, BF, BF, 1, 1, 9, dr=False)
    check_backward(ttt, 9, 64, F32, F32, 0, 1, 0, f=False, dr=False)


@pytest.mark.parametrize("rows,gates", [(1, 1), (5000, 1), (5000, 2), (5000, 10), (5000, 500), (5000, 2500), (5000, 5000)])
def test_backward_sums_over_rows(ttt, rows, gates):
    """Gates of one row to all: sums in slices of a gate, of several gates a workgroup, of rows alone."""
    check_backward(ttt, rows, 72, BF, BF, 1, 1, gates)


def test_backward_is_the_same_every_time_and_in_place(ttt):
    a = check_backward(ttt, 3000, 264, BF, BF, 1, 1, 2)
    b = check_backward(ttt, 3000, 264, BF, BF, 1, 1, 2)
    assert all(torch.equal(a[k], b[k]) for k in a)
    rng = np.random.default_rng(0)
    dr, r, dh = (tensor(rng, 33, 64) for _ in range(3))
    want = ttt.block_norm_backward(dr, dh, r, pre=True)["dx"]
    assert ttt.block_norm_backward(dr, dh, r, pre=True, dx=dr)["dx"] is dr and torch.equal(dr, want)


def test_backward_of_no_rows_gives_zero_sums(ttt):
    e = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    got = ttt.block_norm_backward(e, e, e, e, post=w, pre=w, gate=torch.ones(1, 64, device="cuda"))
    for k in ("dpost", "dpre", "dgate"):
        assert (got[k] == 0).all() and got[k].numel() == 64


def test_captured_and_on_another_stream(ttt):
    rng = np.random.default_rng(3)
    x, f, w, dr, dh = (tensor(rng, *s) for s in ((40, 264), (40, 264), (264,), (40, 264), (40, 264)))

    def both(**kw):
        r, h = ttt.block_norm(x, f, post=w, pre=w, **kw)
        return (r, h, *(t for t in ttt.block_norm_backward(dr, dh, r, f, post=w, pre=w, **kw).values() if t is not None))
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for _ in range(3):
        f.copy_(tensor(rng, 40, 264))
        graph.replay()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
