"""GPU parity of linear attention for few rows a sequence, token by token and in
one short chunk, which are fp32 throughout for either type of rows.

Tolerances: test_parity_linear's of fp32 sums (`coef`), and a bf16 result's one
rounding, 2^-8 of it. Two cases have results that need every one of 24 bits, and
hold them exactly: sums of 1 + 2^-8 + 2^-20 and -(1 + 2^-8), powers of two whose
partial sums fit fp32, so 2^-20 in any order; a part of two bf16 terms loses the
2^-20, which lies 12 bits below the 2^-8 that the first term leaves."""
import pytest
import torch

from test_parity_linear import BF, F32, Case
from test_parity_linear_terms import forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def parity(ttt, lens, dtype=BF, **kw):
    c = Case(lens, dtype=dtype, **kw)
    if dtype == BF:
        forward(ttt, c, terms=0.0)
    else:
        c.check(ttt)


# token by token whatever the rule is (1, 2), and on both sides of it
LENS = [[1], [2, 1], [2, 0, 1], [3], [6, 5], [7, 1], [8, 2, 0, 1], [31], [32, 9]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("group", [1, 2, 3, 5, 9])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_groups(ttt, lens, group, dtype):
    parity(ttt, lens, dtype, group=group, hk=3 if group < 5 else 1)
    parity(ttt, lens, dtype, group=group, state=False)


@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("dv", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dims(ttt, dk, dv, dtype):
    for group in (1, 4):
        parity(ttt, [2, 1], dtype, dk=dk, dv=dv, group=group)
        parity(ttt, [7, 0, 3], dtype, dk=dk, dv=dv, group=group)


@pytest.mark.parametrize("rows", [1, 3, 4, 6, 7])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_sequences(ttt, rows, dtype):
    parity(ttt, [rows] * 40 + [0, 1], dtype, dv=256)


@pytest.mark.parametrize("decays", [[0.0], [-1e-5, -20.0], [-float("inf"), -0.01], [-200.0]])
@pytest.mark.parametrize("lens", [[1], [2], [7]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decays(ttt, decays, lens, dtype):
    parity(ttt, lens, dtype, decays=decays, state=decays[0] != -float("inf"))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,at", [([2, 1], 1), ([7, 3], 4), ([20, 3], 11)])
def test_what_is_not_finite_reaches_no_earlier_row(ttt, bad, which, dtype, lens, at):
    """Rows and heads that it does not reach are those of a clean run (which the
    other tests hold to the oracle): each is within its own bound of the same
    exact value, so within both of the other."""
    c = Case(lens, dtype=dtype, group=2)
    s0 = c.state.clone()
    clean = c.run(ttt, s0).double()
    size = Case.__new__(Case)
    size.__dict__.update({k: (v.abs() if k in ("q", "k", "v") else v) for k, v in c.__dict__.items()})
    size = size.run(ttt, c.state.abs()).double() * 1.01          # the sums of magnitudes, to bf16's 2^-8
    x = getattr(c, which).clone()
    x[at, 0, 5] = bad
    setattr(c, which, x)
    s = c.state.clone()
    o = c.run(ttt, s)
    hit = torch.zeros(c.n, c.hq, dtype=torch.bool, device="cuda")
    if which == "q":
        hit[at, 0] = True
    else:
        hit[at:lens[0], :2] = True
    coef = c.coef + 2.0 ** -16
    room = 2 * coef * size + (2.0 ** -7 * (clean.abs() + coef * size) if dtype == BF else 0) + 1e-37
    assert ((o.double() - clean).abs() <= room)[~hit].all()
    assert not torch.isfinite(o[hit]).all() and torch.isfinite(s[1]).all() and torch.isfinite(s[0, 1]).all()
    assert torch.isfinite(s).all() == (which == "q")


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 7, 8, 32])
def test_every_bit_of_a_state(ttt, rows):
    dk, dv = 128, 64
    q = torch.zeros(rows, 1, dk, dtype=BF, device="cuda")
    q[:, :, 3], q[:, :, 77] = 1, -1
    k, v = torch.zeros(rows, 1, dk, dtype=BF, device="cuda"), torch.ones(rows, 1, dv, dtype=BF, device="cuda")
    state = torch.zeros(1, 1, dk, dv, device="cuda")
    state[0, 0, 3], state[0, 0, 77] = 1 + 2.0 ** -8 + 2.0 ** -20, 1 + 2.0 ** -8
    o = ttt.linear_attention(q, k, v, torch.zeros(1, device="cuda"), state=state, scale=1.0)
    assert (o == 2.0 ** -20).all()


@pytest.mark.parametrize("rows", [2, 3, 5, 7, 8, 32])
def test_every_bit_of_a_weight(ttt, rows):
    dk, dv = 64, 64
    q, k = torch.zeros(2, rows, 1, dk, dtype=BF, device="cuda")
    q[:, 0, 0], q[:, 0, 1], q[:, 0, 2] = 1, 2.0 ** -8, 2.0 ** -20
    k[0, 0, :3] = 1
    k[1, 0, :2] = -1
    v = torch.ones(rows, 1, dv, dtype=BF, device="cuda")
    o = ttt.linear_attention(q, k, v, torch.zeros(1, device="cuda"), scale=1.0)
    assert (o[1:] == 2.0 ** -20).all()
