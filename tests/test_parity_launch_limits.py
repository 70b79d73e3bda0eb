"""GPU: calls whose kernels have more threads than one launch holds (fewer than
2^32), and calls on either side of where launches are cut (2^21 workgroups)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
CUT = 1 << 21


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def test_norm_rows_behind_the_first_launch(ttt):
    """The last rows and the first ones are those of calls of their own."""
    rows, d = CUT + 1003, 64
    g = torch.Generator("cuda").manual_seed(1)
    x, f = (torch.randn(rows, d, generator=g, device="cuda").to(BF) for _ in range(2))
    gate = torch.randn(rows // 3, d, generator=g, device="cuda").to(BF)      # a gate for three rows
    assert rows % 3 == 0
    w = torch.randn(d, generator=g, device="cuda").to(BF)
    r, h = ttt.block_norm(x, f, post=w, pre=w, gate=gate, scale=0.5)
    for rows_, gates in ((slice(0, 300), slice(0, 100)), (slice(rows - 3000, rows), slice(rows // 3 - 1000, rows // 3))):
        r2, h2 = ttt.block_norm(x[rows_], f[rows_], post=w, pre=w, gate=gate[gates], scale=0.5)
        assert torch.equal(r[rows_], r2) and torch.equal(h[rows_], h2)
    at = slice(CUT - 2 - (CUT - 2) % 3, CUT + 31 - (CUT + 31) % 3)           # over the cut
    r2, h2 = ttt.block_norm(x[at], f[at], post=w, pre=w, gate=gate[at.start // 3:at.stop // 3], scale=0.5)
    assert torch.equal(r[at], r2) and torch.equal(h[at], h2)


def test_norm_of_more_threads_than_a_launch_holds(ttt):
    """2^23 + 3 rows, 512 threads each (60 GB of results; all rows are one)."""
    rows, d = (1 << 23) + 3, 3592
    one = torch.randn(1, d, device="cuda").to(BF)
    want = ttt.block_norm(one, pre=True)[1]
    h = ttt.block_norm(one.expand(rows, d), pre=True)[1]
    assert h.shape == (rows, d)
    for lo in range(0, rows, 1 << 19):
        part = h[lo:lo + (1 << 19)]
        assert torch.equal(part, want.expand_as(part)), lo


def test_norm_sums_of_no_rows(ttt):
    """More gates than one launch's workgroups, and no row: sums of zero."""
    gates, d = 16385, 16384
    empty = torch.zeros(0, d, dtype=BF, device="cuda")
    gate = torch.ones(1, d, dtype=BF, device="cuda").expand(gates, d)
    held = torch.full((gates, d), 7.0, device="cuda")      # whose memory the sums get
    del held
    got = ttt.block_norm_backward(empty, None, None, empty, gate=gate)
    assert got["dgate"].shape == (gates, d) and got["dgate"].dtype is F32 and not got["dgate"].any()


def linear_inputs(batch, rows, heads, dk, dv):
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v = (torch.empty(batch * rows, heads, d, dtype=BF, device="cuda").normal_(generator=g) for d in (dk, dk, dv))
    return q, k, v, -torch.rand(heads, generator=g, device="cuda")


@pytest.mark.parametrize("rows", [1, 8])
def test_linear_sequences_behind_the_first_launch(ttt, rows):
    """2^22 - 64 states of 8 slices (token by token: more than 2^32 threads) or 2:
    some sequences from all over are those of calls of their own."""
    batch, heads, dk, dv = 65535, 64, 64, 256 if rows == 1 else 64
    q, k, v, ld = linear_inputs(batch, rows, heads, dk, dv)
    out = torch.full((batch * rows, heads, dv), 7.0, dtype=BF, device="cuda")
    ttt.linear_attention(q, k, v, ld, q_starts=torch.arange(0, batch * rows + 1, rows, dtype=torch.int32, device="cuda"),
                         max_new=rows, out=out)
    for lo in (0, 4000, 32767, 32768, 65500):
        cut = slice(lo * rows, min(lo + 40, batch) * rows)
        n = (cut.stop - cut.start) // rows
        want = ttt.linear_attention(q[cut], k[cut], v[cut], ld,
                                    q_starts=torch.arange(0, n * rows + 1, rows, dtype=torch.int32, device="cuda"), max_new=rows)
        assert torch.equal(out[cut], want), lo
    assert not (out == 7).all(-1).any()


def test_linear_gradients_of_more_threads_than_a_launch_holds(ttt):
    """2^22 - 64 states of heads of 256: three roles of two slices, 1.5 times 2^32 threads."""
    batch, heads, d = 65535, 64, 256
    q, k, v, ld = linear_inputs(batch, 1, heads, d, d)
    do = torch.empty_like(v).normal_(generator=torch.Generator("cuda").manual_seed(4))
    dq, dk, dv, _ = ttt.linear_attention_backward(do, q, k, v, ld, q_starts=torch.arange(batch + 1, dtype=torch.int32, device="cuda"),
                                                  max_new=1, scale=0.0625)
    for lo in (0, 4000, 32767, 43000, 65500):
        cut = slice(lo, min(lo + 30, batch))
        n = cut.stop - lo
        want = ttt.linear_attention_backward(do[cut], q[cut], k[cut], v[cut], ld,
                                             q_starts=torch.arange(n + 1, dtype=torch.int32, device="cuda"), max_new=1, scale=0.0625)
        for g, w in zip((dq, dk, dv), want):
            assert torch.equal(g[cut], w), lo
    # dv of one row: scale (k q) do, of dq and dk likewise: none is left as it was
    for g in (dq, dk, dv):
        assert all(bool((part != 0).any(-1).all()) for part in g.split(8192))


def need_memory(gb):
    if torch.cuda.mem_get_info()[0] < gb * 10 ** 9:
        pytest.skip(f"needs {gb} GB of GPU memory")


def test_adamw_values_behind_the_first_launch(ttt):
    """2^32 + 12345 values: steps and states read back, beside a call for the last ones."""
    n = (1 << 32) + 12345
    last = n - (1 << 32) + (1 << 20)          # whole chunks and blocks before them
    gen = torch.Generator("cuda").manual_seed(5)
    p, g = (torch.empty(n, dtype=BF, device="cuda").normal_(generator=gen) for _ in range(2))
    p2, g2 = p[-last:].clone(), g[-last:].clone()
    kw = dict(lr=1e-2, weight_decay=0.1, bits=8)
    state, state2 = ttt.adamw_state([p], 8), ttt.adamw_state([p2], 8)
    for step in (1, 2):
        ttt.adamw_step([p], [g], state, step=step, **kw)
        ttt.adamw_step([p2], [g2], state2, step=step, **kw)
    assert torch.equal(p[-last:], p2)
    del p, g
    for x, y in zip(ttt.adamw_read(state, 8, dtype=BF), ttt.adamw_read(state2, 8, dtype=BF)):
        assert torch.equal(x[-y.numel():], y) and bool(y[:last].any())


def test_adamw_of_more_threads_than_a_launch_holds(ttt):
    """17 tensors of 2^31 values with one gradient (144 GB): each becomes what the first does."""
    need_memory(160)
    n, count = 1 << 31, 17
    g = torch.empty(n, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(6))
    ps = [torch.ones(n, dtype=BF, device="cuda") for _ in range(count)]
    state = ttt.adamw_state(ps, 8)
    ttt.adamw_step(ps, [g] * count, state, lr=0.1, step=1, bits=8)
    one = torch.ones(1 << 20, dtype=BF, device="cuda")
    ttt.adamw_step([one], [g[:1 << 20]], ttt.adamw_state([one], 8), lr=0.1, step=1, bits=8)
    assert torch.equal(ps[0][:1 << 20], one) and not (one == 1).any()
    codes = state[:n * count].view(count, n)
    for i in range(1, count):
        for lo in range(0, n, n // 4):
            at = slice(lo, lo + n // 4)
            assert torch.equal(ps[i][at], ps[0][at]) and torch.equal(codes[i, at], codes[0, at]), (i, lo)
