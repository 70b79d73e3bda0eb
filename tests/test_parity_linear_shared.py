"""GPU parity of linear attention's gradients where query heads share a state, in
every pair of dimensions (their own kernels, and with dim_k != dim_v launches of
their own), and of long sequences' parts in every dimension, forward and backward.
Tolerances as in test_parity_linear (fp32) and test_parity_linear_terms (bf16)."""
import pytest
import torch

from test_parity_linear import BF, F32, Case
from test_parity_linear_terms import backward, forward

pytestmark = pytest.mark.gpu
DIMS = [64, 128, 256]


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def gradients(ttt, c):
    if c.dtype == BF:
        backward(ttt, c)
    else:
        c.check_backward(ttt)


@pytest.mark.parametrize("dk", DIMS)
@pytest.mark.parametrize("dv", DIMS)
@pytest.mark.parametrize("group", [2, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_of_shared_states(ttt, dk, dv, group, dtype):
    gradients(ttt, Case([100, 37], dk=dk, dv=dv, group=group, dtype=dtype, scale=dk ** -0.5))
    gradients(ttt, Case([5, 0, 1], dk=dk, dv=dv, group=group, dtype=dtype, scale=dk ** -0.5, state=False))


@pytest.mark.parametrize("dk,dv", [(128, 128), (256, 256), (64, 256), (256, 128)])
@pytest.mark.parametrize("group", [1, 2])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_parts_of_dims(ttt, dk, dv, group, dtype):
    c = Case([700, 200, 0, 321], hk=1, dk=dk, dv=dv, group=group, dtype=dtype, scale=dk ** -0.5)
    if dtype == BF:
        forward(ttt, c)
    else:
        c.check(ttt)
    gradients(ttt, c)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 256), (128, 64)])
@pytest.mark.parametrize("group", [1, 3])
@pytest.mark.parametrize("lens", [[50], [900]])
def test_the_state_gradient_in_its_place(ttt, dk, dv, group, lens):
    """d_state0 in d_state, with one part and with several: what it is apart."""
    c = Case(lens, hk=1, dk=dk, dv=dv, group=group)
    kw = dict(q_starts=c.starts, scale=c.scale, max_new=lens[0], state=c.state)
    want = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, d_state=c.d_state, **kw)
    d = c.d_state.clone()
    got = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, d_state=d, d_state0=d, **kw)
    assert got[3] is d and all(map(torch.equal, got, want))
