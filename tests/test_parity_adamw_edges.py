"""GPU: AdamW steps at the edges of their ranges."""
import pytest
import torch

from test_parity_adamw import BF, F32, HYPER, SIZES, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,masters", [(BF, True), (F32, False)])
@pytest.mark.parametrize("lr", ["host", "device"])
def test_a_step_on_the_device_counts_from_one(ttt, bits, dtype, masters, lr):
    """Below 1 nothing changes; a captured loop whose counter starts at 0 takes its
    first step at 1."""
    hyper = dict(HYPER, bits=bits)
    if lr == "device":
        hyper["lr"] = torch.tensor(HYPER["lr"], dtype=F32, device="cuda")
    ps, gs, ms = make(SIZES, dtype, F32, masters)
    state = ttt.adamw_state(ps, bits)
    step = torch.ones(1, dtype=torch.int32, device="cuda")
    ttt.adamw_step(ps, gs, state, step=step, masters=ms, **hyper)       # states that are not zero
    held = [[t.clone() for t in x] for x in (ps, ms or [], [state])]
    for n in (0, -1, -(1 << 31)):
        step.fill_(n)
        ttt.adamw_step(ps, gs, state, step=step, masters=ms, **hyper)
        for x, y in zip((ps, ms or [], [state]), held):
            assert all(map(torch.equal, x, y)), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ttt.adamw_step(ps, gs, state, step=step, masters=ms, **hyper)
        step.add_(1)
    step.fill_(0)
    graph.replay()
    for x, y in zip((ps, ms or [], [state]), held):
        assert all(map(torch.equal, x, y))
    graph.replay()
    assert int(step) == 2
    ps2, ms2, state2 = held
    step.fill_(1)
    ttt.adamw_step(ps2, gs, state2[0], step=step, masters=ms2 or None, **hyper)
    assert all(map(torch.equal, ps, ps2)) and torch.equal(state, state2[0])
    assert all(torch.isfinite(p).all() for p in ps)
