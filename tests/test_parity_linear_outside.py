"""GPU: the gradients of rows that no sequence claims are zero, written by the
library itself (the outputs hold something else before), and no other row's are."""
import ctypes

import pytest
import torch

from test_parity_linear import BF, F32, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def rows(t):
    from test_layer_gate_amd import _serve as sv
    return ctypes.byref(sv.Rows(t.data_ptr(), t.stride(0), t.stride(1), t.shape[1], 0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [1, 2])
@pytest.mark.parametrize("before,lens,behind", [(0, [40, 70], 13), (9, [3, 0, 65], 0), (1, [64], 700), (5, [0, 0], 7), (0, [33], 0)])
def test_the_library_writes_every_row(ttt, dtype, group, before, lens, behind):
    from test_layer_gate_amd import _block as bl
    c = Case([before + sum(lens) + behind], dtype=dtype, group=group, dv=128)
    B, n = len(lens), c.n
    starts = torch.tensor([before + sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    dt = 0 if dtype == BF else 1
    desc = bl.Linear(c.ld.data_ptr(), starts.data_ptr(), B, n, max(1, *lens), dt, c.hk, c.hq, c.dk, c.dv, c.scale, 0)
    need = ctypes.c_size_t(0)
    L = bl._L()
    assert L.ttt_linear_attention_backward_workspace_size(ctypes.byref(desc), ctypes.byref(need)) == 0
    ws = torch.empty(max(256, need.value), dtype=torch.uint8, device="cuda")

    def filled(heads, dim):     # heads apart by more than their values
        return torch.full((n, heads, dim + 16), 3.0, dtype=dtype, device="cuda")[..., :dim]
    got = filled(c.hq, c.dk), filled(c.hk, c.dk), filled(c.hk, c.dv)
    st = L.ttt_linear_attention_backward(ctypes.byref(desc), rows(c.do), rows(c.q), rows(c.k), rows(c.v), None, None,
                                         *map(rows, got), None, ws.data_ptr(), ws.nbytes,
                                         torch.cuda.current_stream().cuda_stream)
    assert st == 0, L.ttt_last_error()
    inside = slice(before, before + sum(lens))
    cut = [x[inside].contiguous() for x in (c.do, c.q, c.k, c.v)]
    want = ttt.linear_attention_backward(*cut, c.ld, q_starts=starts - before, scale=c.scale, max_new=max(1, *lens))
    for g, w in zip(got, want):
        assert torch.equal(g[inside], w)
        out = torch.cat([g[:before], g[inside.stop:]])
        assert out.shape[0] == before + behind and (out == 0).all()
        assert (g.as_strided((n, g.shape[1], 16), g.stride(), g.storage_offset() + g.shape[2]) == 3).all()


def test_starts_out_of_order(ttt):
    """Sequences that are cut short by their starts: every row is a gradient or zero."""
    c = Case([100], dtype=F32)
    starts = torch.tensor([60, 90, 20, 30], dtype=torch.int32, device="cuda")    # rows 60..89 and 20..29
    got = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, q_starts=starts, scale=c.scale)
    for g in got[:3]:
        assert (g[:20] == 0).all() and (g[30:60] == 0).all() and (g[90:] == 0).all()
        assert (g[20:30] != 0).any() and (g[60:90] != 0).any()
