"""GPU parity of bf16 linear attention, beyond its result's own rounding: weights
and states enter their products as two bf16 terms.

Tolerances, relative to the same sums with every term's magnitude (size). A bf16
rounding leaves at most half a step, 2^-8 of its value, and the second term's
2^-8 of that again: 2^-16 of each weight or state, of which every term of a result
holds one. What fp32 sums leave is test_parity_linear's `coef`. The result is
rounded once (2^-8 of itself). Of all values together (2-norm) those roundings are
spread evenly over a step of at most 2^-7 of the value: 2^-7 / sqrt(12) of it (one
term of the state leaves 0.0023 to 0.0024, more than that)."""
import math

import numpy as np
import pytest
import torch

import oracle.block_oracle as bo
from test_parity_linear import Case, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def close(got, ref, size, coef, what):
    room = coef * size
    room = room + 2.0 ** -8 * (np.abs(ref) + room) + 1e-37
    err = np.abs(got - ref)
    assert (err <= room).all(), (what, float((err / room).max()))
    if ref.size:
        e, r = np.linalg.norm(err), np.linalg.norm(ref)
        assert e <= 2.0 ** -7 / math.sqrt(12) * r + 1e-30, (what, e / r)


def forward(ttt, c, terms=2.0 ** -16, **kw):
    s = None if c.state is None else c.state.clone()
    o = c.run(ttt, s, **kw)
    for b in range(len(c.lens)):
        at = c.rows(b)
        args = [host(x[at]) for x in (c.q, c.k, c.v)]
        s0 = None if s is None else host(c.state[b])
        ref, last = bo.linear(*args, c.g, c.scale, s0)
        size, state_size = bo.linear(*map(np.abs, args), c.g, c.scale, None if s0 is None else np.abs(s0))
        close(host(o[at]), ref, size, c.coef + terms, ("o", b))
        if s is not None:
            assert (np.abs(host(s[b]) - last) <= c.coef * state_size + 1e-37).all(), b


def backward(ttt, c):
    got = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, q_starts=c.starts, scale=c.scale, max_new=max(c.lens),
                                        state=c.state, d_state=c.d_state)
    coef = c.coef * (c.hq // c.hk) + 2.0 ** -16
    for b in range(len(c.lens)):
        at = c.rows(b)
        args = [host(x[at]) for x in (c.do, c.q, c.k, c.v)]
        s0, ds = (None if x is None else host(x[b]) for x in (c.state, c.d_state))
        ref = bo.linear_backward(*args, c.g, c.scale, s0, ds)
        size = bo.linear_backward(*map(np.abs, args), c.g, c.scale, *(None if x is None else np.abs(x) for x in (s0, ds)))
        for i, name in enumerate(("dq", "dk", "dv")):
            close(host(got[i][at]), ref[i], size[i], coef, (name, b))
        if got[3] is not None:
            assert (np.abs(host(got[3][b]) - ref[3]) <= c.coef * (c.hq // c.hk) * size[3] + 1e-37).all(), b


@pytest.mark.parametrize("lens", [[9], [33], [64], [200], [0, 130, 1, 0, 64], [1400, 300, 0, 513]])
@pytest.mark.parametrize("group", [1, 3])
def test_outputs(ttt, lens, group):
    forward(ttt, Case(lens, group=group))
    forward(ttt, Case(lens, group=group, state=False, decays=[-0.01]))


@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128), (128, 256), (256, 64), (256, 256)])
def test_outputs_of_dims(ttt, dk, dv):
    forward(ttt, Case([100, 37], dk=dk, dv=dv, group=2, scale=dk ** -0.5))


@pytest.mark.parametrize("which", ["state", "weights"])
def test_each_part_alone(ttt, which):
    """A state that no row adds to, and rows without a state."""
    c = Case([150], dk=128, dv=128, group=2, decays=[-1e-4], state=which == "state")
    if which == "state":
        c.k = torch.zeros_like(c.k)
    forward(ttt, c)


@pytest.mark.parametrize("lens", [[9], [65], [0, 130, 1, 0, 64], [1100, 300, 0, 513]])
@pytest.mark.parametrize("group", [1, 2])
def test_gradients(ttt, lens, group):
    backward(ttt, Case(lens, group=group))


@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128), (128, 256), (256, 64)])
def test_gradients_of_dims(ttt, dk, dv):
    backward(ttt, Case([100, 37], dk=dk, dv=dv, scale=dk ** -0.5))
