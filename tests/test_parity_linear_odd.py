"""GPU: an infinity or a NaN in linear attention's inputs reaches what depends on
it, and nothing else: everything else has the bits of a clean run (what is masked
away takes no part in it). o and the state after row `at` depend on a row of k and
v, o of its row and heads on one of q. Of the gradients,

  dq_t  on do_t, and on k_j and v_j of j <= t
  dk_j  on v_j, and on q_t and do_t of t >= j (of the state's heads)
  dv_j  on k_j, and likewise
  the first state's  on every q and do"""
import pytest
import torch

from test_parity_linear import BF, F32, Case

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def spoiled(c, which, at, bad):
    x = getattr(c, which).clone()
    x[at, 0, 5] = bad
    setattr(c, which, x)


def same(got, want, hit, what):
    assert torch.equal(got[~hit], want[~hit]), what


@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("group", [1, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,at", [([130, 70], 77), ([900], 450), ([20, 3], 11), ([5, 2], 2)])
def test_outputs(ttt, which, bad, group, dtype, lens, at):
    c = Case(lens, group=group, dtype=dtype, dv=128)
    s0, s1 = c.state.clone(), c.state.clone()
    want = c.run(ttt, s0)
    spoiled(c, which, at, bad)
    got = c.run(ttt, s1)
    hit = torch.zeros(c.n, c.hq, dtype=torch.bool, device="cuda")
    if which == "q":
        hit[at, 0] = True
        assert torch.equal(s0, s1)
    else:
        hit[at:lens[0], :group] = True
        assert not torch.isfinite(s1[0, 0]).all() and torch.equal(s0[1:], s1[1:]) and torch.equal(s0[0, 1:], s1[0, 1:])
    same(got, want, hit, "o")
    rows = got.flatten(2)[hit]
    assert not torch.isfinite(rows).all(-1).any()               # every row that depends on it


@pytest.mark.parametrize("which", ["do", "q", "k", "v"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("group", [1, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,at", [([130, 70], 77), ([900], 450), ([20, 3], 11)])
def test_gradients(ttt, which, bad, group, dtype, lens, at):
    c = Case(lens, group=group, dtype=dtype, dv=128)
    kw = dict(q_starts=c.starts, scale=c.scale, max_new=max(lens), state=c.state, d_state=c.d_state)
    want = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, **kw)
    spoiled(c, which, at, bad)
    got = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, **kw)
    dq = torch.zeros(c.n, c.hq, dtype=torch.bool, device="cuda")
    dk, dv = (torch.zeros(c.n, c.hk, dtype=torch.bool, device="cuda") for _ in range(2))
    if which == "do":
        dq[at, 0] = True
    if which in ("do", "q"):
        dk[:at + 1, 0] = dv[:at + 1, 0] = True
        assert not torch.isfinite(got[3][0, 0]).all() and torch.equal(got[3][:, 1:], want[3][:, 1:])
        assert torch.equal(got[3][1:], want[3][1:])
    else:
        dq[at:lens[0], :group] = True
        (dv if which == "k" else dk)[at, 0] = True
        assert torch.equal(got[3], want[3])
    for g, w, hit, name in zip(got, want, (dq, dk, dv), ("dq", "dk", "dv")):
        same(g, w, hit, name)
        if hit.any():
            assert not torch.isfinite(g.flatten(2)[hit]).all(-1).any(), name
