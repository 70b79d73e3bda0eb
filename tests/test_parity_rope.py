"""GPU parity of the rotary positions: the table of every scaling, and the
rotation and its gradient for both pair layouts, parts of the head, strided
and in-place tensors.

Tolerances. A rotated value is fl(fl(a c) - fl(b s)): three roundings, at
most 2^-24 (|a c| + |b s|) for the products and as much again for the sum;
a bf16 result (8 significant bits) adds half a unit in the last place, at
most 2^-8 of the value. The
table is rounded once from float64 angles of up to 1e5 rad whose own error
is below 1e5 * 2^-50."""
import numpy as np
import pytest
import torch

import oracle.serve_oracle as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def close(y, x, cs, inter, transposed, dtype, what):
    ref = so.rotate(x, cs, inter, transposed)
    room = 2 ** -23 * (so.rotate(np.abs(x), np.abs(cs), inter, True))   # |a c| + |b s| for one of
    room = np.maximum(room, 2 ** -23 * so.rotate(np.abs(x), np.abs(cs), inter))  # the pair's two
    rot = 2 * cs.shape[1]
    room[..., rot:] = 0
    if dtype == BF:
        room = room + 2 ** -8 * np.abs(ref) * (np.arange(x.shape[-1]) < rot)
    err = np.abs(y - ref)
    assert (err <= room + 1e-37).all(), (what, float((err - room).max()))


@pytest.mark.parametrize("kind,kw", [
    (None, {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
    ("yarn", dict(factor=4.0, original=4096, low=1, high=32)),
    ("yarn", dict(factor=16.0, original=64, low=1, high=32)),
    ("bands", dict(factor=8.0, original=8192, low=1, high=4))])
@pytest.mark.parametrize("rot,base", [(16, 1e4), (128, 5e5), (96, 1e6)])
def test_table(ttt, kind, kw, rot, base):
    t = ttt.rope_table(3000, rot, base, scaling=kind, amplitude=1.25, **kw)
    ref = so.table(3000, rot, base, amplitude=1.25, kind=kind, **kw)
    assert t.shape == (3000, rot // 2, 2)
    assert np.abs(host(t) - ref).max() <= 2 ** -24 * 1.25 + 1e-9


def test_table_far_positions(ttt):
    t = ttt.rope_table(131072, 16, 1e4)
    ref = so.table(131072, 16, 1e4)
    assert np.abs(host(t) - ref)[-100:].max() <= 2 ** -24 + 1e-9
    yarn = ttt.rope_table(8, 16, 1e4, scaling="yarn", factor=4.0, original=4096)
    assert abs(float(yarn[0, 0, 0]) - (0.1 * np.log(4) + 1)) < 1e-6


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hk,dim,rot", [
    (1, 1, 1, 16, 16), (3, 5, 1, 64, 32), (7, 4, 2, 80, 32), (257, 32, 8, 128, 128),
    (33, 3, 3, 96, 96), (65, 2, 1, 256, 64), (2, 1, 1, 1024, 1024), (4097, 8, 2, 64, 16)])
def test_rotation_and_gradient(ttt, dtype, inter, n, hq, hk, dim, rot):
    g = torch.Generator().manual_seed(n * dim + rot)
    x = torch.randn(n, hq + 2 * hk, dim, generator=g).to(dtype).cuda()
    q, k = x[:, :hq], x[:, hq:hq + hk]          # parts of one projection
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32)
    table = ttt.rope_table(5000, rot, 1e4)
    cs = host(table)[pos.numpy()]
    for f, back in ((ttt.rope_forward, False), (ttt.rope_backward, True)):
        before = x.clone()
        yq, yk = f(q, k, table, positions=pos.cuda(), interleaved=inter)
        torch.cuda.synchronize()
        assert torch.equal(x, before)
        close(host(yq), host(q), cs, inter, back, dtype, "q")
        close(host(yk), host(k), cs, inter, back, dtype, "k")
        only, none = f(q, None, table, positions=pos.cuda(), interleaved=inter)
        assert none is None and torch.equal(only, yq)
        into = dict(dq=q, dk=k) if back else dict(q_out=q, k_out=k)
        f(q, k, table, positions=pos.cuda(), interleaved=inter, **into)     # in place
        torch.cuda.synchronize()
        assert torch.equal(x[:, :hq], yq) and torch.equal(x[:, hq:hq + hk], yk)
        assert torch.equal(x[:, hq + hk:], before[:, hq + hk:])
        x.copy_(before)


def test_gradient_is_that_of_differences(ttt):
    """d/dx_i of <dy, R x>, by central differences of the forward in fp32. The
    map is linear, so a difference of width 2 has no truncation error; its
    rounding is 2^-23 of the sum's terms, for 64 of them below 64 * 2^-22."""
    g = torch.Generator().manual_seed(5)
    n, dim, rot = 3, 64, 32
    table = ttt.rope_table(100, rot, 1e4)
    x, dy = torch.randn(2, n, 1, dim, generator=g).cuda()
    pos = torch.tensor([0, 17, 99], dtype=torch.int32, device="cuda")
    for inter in (False, True):
        dx, _ = ttt.rope_backward(dy, None, table, positions=pos, interleaved=inter)
        for i in range(dim):
            e = torch.zeros_like(x)
            e[..., i] = 1.0
            up, _ = ttt.rope_forward(x + e, None, table, positions=pos, interleaved=inter)
            dn, _ = ttt.rope_forward(x - e, None, table, positions=pos, interleaved=inter)
            num = ((up - dn) * dy).sum((1, 2)) / 2
            assert (num - dx[:, 0, i]).abs().max() <= 64 * 2 ** -22


def test_batches_head_major_and_default_positions(ttt):
    g = torch.Generator().manual_seed(6)
    table = ttt.rope_table(40, 64, 1e4)
    q = torch.randn(3, 40, 4, 64, generator=g).to(BF).cuda()
    yq, _ = ttt.rope_forward(q, None, table)      # positions restart in every sequence
    cs = np.tile(host(table), (3, 1, 1))
    close(host(yq).reshape(120, 4, 64), host(q).reshape(120, 4, 64), cs, False, False, BF, "batch")
    hm = torch.randn(4, 40, 64, generator=g).cuda()   # [heads, tokens, dim]
    out = torch.empty_like(hm)
    ttt.rope_forward(hm.transpose(0, 1), None, table, q_out=out.transpose(0, 1))
    close(host(out.transpose(0, 1)), host(hm.transpose(0, 1)), host(table), False, False, F32, "hm")
    one = torch.randn(1, 1, 64, generator=g).cuda().expand(40, 2, 64)  # broadcast input
    y, _ = ttt.rope_forward(one, None, table)
    close(host(y), host(one), host(table), False, False, F32, "broadcast")


def test_positions_outside_the_table_are_nan_and_empty_calls(ttt):
    table = ttt.rope_table(10, 32, 1e4)
    q = torch.ones(3, 1, 64, device="cuda")
    pos = torch.tensor([9, 10, -1], dtype=torch.int32, device="cuda")
    y, _ = ttt.rope_forward(q, None, table, positions=pos)
    y = y.cpu()
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1:, :, :32]).all()
    assert (y[1:, :, 32:] == 1).all()
    e, _ = ttt.rope_forward(q[:0], None, table)
    assert e.shape == (0, 1, 64)


def test_another_stream(ttt):
    table = ttt.rope_table(600, 128, 1e4)
    q = torch.randn(600, 8, 128, device="cuda")
    ref, _ = ttt.rope_forward(q, None, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    ttt.rope_forward(q, None, table, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
