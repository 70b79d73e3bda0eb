"""GPU parity of linear attention and its gradients against the float64 oracle
(token by token), in chunks and for few tokens.

Tolerances, u = 2^-24, relative to the same sums with every term's magnitude
(A). fp32: a sum over dim_k, over at most 64 rows of a chunk, and a state that
each chunk multiplies once and adds to twice: dim_k + 64 + 3 chunks roundings;
g^n is 2^(n lg): the exponent is within 3 u of itself, so g^n within 3 u n
|log_decay| + 2 u of itself, and where that passes 64 u the term is below 2^-30 of
the others. bf16 rows in chunks: the weights or the state are rounded (half a step,
2^-8 of their part of A each, so of A together), and the result (2^-8 of it).
Those roundings are spread evenly, so of all values together (2-norm) the error is
within sqrt(2 / 3) 2^-8 < 2^-8; fp32's is within 16 sqrt(dim_k) u of it. States
have fp32's in either type (v times its decay enters as 24 bits)."""
import math

import numpy as np
import pytest
import torch

import oracle.block_oracle as bo

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
FEW = 2      # rows a sequence that are taken one by one, in fp32: no weights are rounded


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Case:
    def __init__(self, lens, hk=2, group=1, dk=64, dv=64, dtype=BF, decays=None, state=True, seed=0, gap=0, scale=0.2):
        rng = np.random.default_rng(seed)
        self.lens, self.dtype, self.scale = lens, dtype, scale
        self.hk, self.hq, self.dk, self.dv = hk, hk * group, dk, dv
        n = self.n = sum(lens) + gap

        def t(*s, dtype=dtype):
            return torch.from_numpy(rng.standard_normal(s)).to(dtype).cuda()
        x = t(n, self.hq * dk + hk * (dk + dv))          # one projection's output
        self.q = x[:, :self.hq * dk].unflatten(1, (self.hq, dk))
        self.k = x[:, self.hq * dk:(self.hq + hk) * dk].unflatten(1, (hk, dk))
        self.v = x[:, (self.hq + hk) * dk:].unflatten(1, (hk, dv))
        self.do = t(n, self.hq, dv)
        decays = [-0.002, -0.3] if decays is None else decays
        self.ld = torch.tensor([decays[h % len(decays)] for h in range(hk)], dtype=F32, device="cuda")
        B = len(lens)
        self.state = t(B, hk, dk, dv, dtype=F32) if state else None
        self.d_state = t(B, hk, dk, dv, dtype=F32) if state else None
        self.starts = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
        self.g = np.exp(host(self.ld))
        self.coef = (dk + 64 + 3 * math.ceil(max(lens) / 32) + 128) * U

    def run(self, ttt, state, **kw):
        kw.setdefault("max_new", max(self.lens))
        return ttt.linear_attention(self.q, self.k, self.v, self.ld, state=state, q_starts=self.starts, scale=self.scale, **kw)

    def rows(self, b):
        lo = sum(self.lens[:b])
        return slice(lo, lo + self.lens[b])

    def check(self, ttt, few=None, **kw):
        s = None if self.state is None else self.state.clone()
        o = self.run(ttt, s, **kw)
        few = max(self.lens) <= FEW if few is None else few
        for b in range(len(self.lens)):
            at = self.rows(b)
            args = [host(x[at]) for x in (self.q, self.k, self.v)]
            s0 = None if s is None else host(self.state[b])
            ref, last = bo.linear(*args, self.g, self.scale, s0)
            size, state_size = bo.linear(*map(np.abs, args), self.g, self.scale, None if s0 is None else np.abs(s0))
            close(host(o[at]), ref, size, self.coef, self.dtype, "few" if few else "o", self.dk)
            if s is not None:
                room = self.coef * state_size
                assert (np.abs(host(s[b]) - last) <= room + 1e-37).all(), (b, float((np.abs(host(s[b]) - last) / room).max()))
        return o, s

    def check_backward(self, ttt, **kw):
        kw = dict(dict(max_new=max(self.lens), state=self.state, d_state=self.d_state), **kw)
        keep = None if kw["d_state"] is None else kw["d_state"].clone()
        got = ttt.linear_attention_backward(self.do, self.q, self.k, self.v, self.ld, q_starts=self.starts, scale=self.scale, **kw)
        for b in range(len(self.lens)):
            at = self.rows(b)
            args = [host(x[at]) for x in (self.do, self.q, self.k, self.v)]
            s0, ds = (None if x is None else host(x[b]) for x in (kw["state"], keep))
            ref = bo.linear_backward(*args, self.g, self.scale, s0, ds)
            size = bo.linear_backward(*map(np.abs, args), self.g, self.scale, None if s0 is None else np.abs(s0),
                                      None if ds is None else np.abs(ds))
            for i, name in enumerate(("dq", "dk", "dv")):
                close(host(got[i][at]), ref[i], size[i], self.coef * (self.hq // self.hk), self.dtype, name, max(self.dk, self.dv))
            if got[3] is not None:
                room = self.coef * (self.hq // self.hk) * size[3]
                assert (np.abs(host(got[3][b]) - ref[3]) <= room + 1e-37).all(), b
        return got


def close(got, ref, size, coef, dtype, what, dim):
    room = coef * size + 1e-37
    if dtype == BF:
        room = room + 2.0 ** -8 * np.abs(ref) + (0.0 if what == "few" else (2.0 ** -8 + 2.0 ** -16) * size)
    err = np.abs(got - ref)
    assert (err <= room).all(), (what, float((err / room).max()))
    if ref.size:
        all_together = 2.0 ** -8 if dtype == BF else 16 * math.sqrt(dim) * U
        assert np.linalg.norm(err) <= all_together * np.linalg.norm(ref) + 1e-30, (what, np.linalg.norm(err) / np.linalg.norm(ref))


# chunks of 64 rows (bf16) and 32 (fp32): less than one, whole ones, one more; empty sequences between
LENS = [[9], [31], [32], [33], [63], [64], [65], [200], [0, 130, 1, 0, 64]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths(ttt, lens, dtype):
    Case(lens, group=2, dtype=dtype).check(ttt)


@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("dv", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dims(ttt, dk, dv, dtype):
    Case([100, 37], dk=dk, dv=dv, dtype=dtype).check(ttt)
    Case([3, 1], dk=dk, dv=dv, dtype=dtype, group=3).check(ttt)


@pytest.mark.parametrize("group", [1, 2, 3, 5])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_groups(ttt, group, dtype):
    Case([140], group=group, dtype=dtype, hk=3).check(ttt)
    Case([8, 2, 0, 1], group=group, dtype=dtype, hk=3).check(ttt)
    Case([5], group=9, dtype=dtype, hk=1).check(ttt)


@pytest.mark.parametrize("decays", [[0.0], [-1e-5, -20.0], [-float("inf"), -0.01], [-200.0]])
@pytest.mark.parametrize("lens", [[70], [4]])
def test_decays(ttt, decays, lens):
    """No decay, next to none, at once, and all there can be: g^0 is 1 whatever g is."""
    for dtype in (BF, F32):
        Case(lens, decays=decays, dtype=dtype, state=decays[0] != -float("inf")).check(ttt)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_parts_of_long_sequences(ttt, dtype):
    """Long enough for several parts, of which the last is short or missing."""
    Case([1400, 300, 0, 513], hk=1, dtype=dtype).check(ttt)
    Case([700], hk=1, group=2, dtype=dtype, state=False).check(ttt)


@pytest.mark.parametrize("max_new", [1, 2, 8, 64, 5000])
def test_a_wrong_bound_changes_no_result(ttt, max_new):
    Case([333, 20], group=2, dtype=F32).check(ttt, max_new=max_new)
    Case([333, 20], group=2).check(ttt, max_new=max_new, few=max_new <= FEW)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_segments_then_tokens_continue_a_prompt(ttt, dtype):
    c = Case([150], dtype=dtype, group=2)
    s = c.state.clone()
    o, at = [], 0
    for n in (64, 65, 9, 8, 1, 1, 2):
        cut = slice(at, at + n)
        o.append(ttt.linear_attention(c.q[cut], c.k[cut], c.v[cut], c.ld, state=s, scale=c.scale))
        at += n
    ref, last = bo.linear(host(c.q), host(c.k), host(c.v), c.g, c.scale, host(c.state[0]))
    size, state_size = bo.linear(*(np.abs(host(x)) for x in (c.q, c.k, c.v)), c.g, c.scale, np.abs(host(c.state[0])))
    close(host(torch.cat(o)), ref, size, c.coef, dtype, "o", c.dk)
    assert (np.abs(host(s[0]) - last) <= c.coef * state_size).all()


def test_rows_behind_the_last_sequence_are_left(ttt):
    for lens in ([40, 70], [3, 1]):
        c = Case(lens, gap=13)
        out = torch.full((c.n, c.hq, c.dv), 3.0, dtype=BF, device="cuda")
        assert c.run(ttt, None, out=out) is out
        assert (out[sum(lens):] == 3).all() and torch.equal(out[:sum(lens)], c.run(ttt, None)[:sum(lens)])
        got = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, q_starts=c.starts)
        assert all((g[sum(lens):] == 0).all() for g in got[:3])


def test_layouts(ttt):
    """Head-major rows, [B, T, heads, dim], broadcast heads, strided outputs."""
    c = Case([60, 60], hk=2, group=2)
    want = c.run(ttt, c.state.clone())
    q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (c.q, c.k, c.v))
    kw = dict(scale=c.scale, state=c.state.clone())
    assert torch.equal(ttt.linear_attention(q, k, v, c.ld, **kw), want)
    four = [x.reshape(2, 60, *x.shape[1:]) for x in (c.q, c.k, c.v)]
    kw["state"] = c.state.clone()
    assert torch.equal(ttt.linear_attention(*four, c.ld, **kw).reshape(want.shape), want)
    out = torch.zeros(120, 4, 96, dtype=BF, device="cuda")[..., :64]
    kw["state"] = c.state.clone()
    ttt.linear_attention(c.q, c.k, c.v, c.ld, out=out, **kw)
    assert torch.equal(out, want)
    one = c.k[:, :1].expand(-1, 2, -1)
    kw["state"] = c.state.clone()
    a = ttt.linear_attention(c.q, one, c.v, c.ld, **kw)
    kw["state"] = c.state.clone()
    assert torch.equal(a, ttt.linear_attention(c.q, one.contiguous(), c.v, c.ld, **kw))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_what_is_not_finite_reaches_no_earlier_row(ttt, dtype, bad, which):
    """Rows that it must not reach are the oracle's of clean inputs. (Their bits
    may differ from a clean run's: a chunk with such a v is taken row by row, and
    each of two results is within the elementwise bound of the exact one, whose
    terms of either sign cancel: no bound relative to the result alone holds, with
    o = a - b, a = b (1 + d), |error| up to 2^-8 (a + b) = (2 / d + 1) 2^-8 |o|.)"""
    for lens, at in (([130, 70], 77), ([5, 3], 2)):
        c = Case(lens, dtype=dtype, group=2)
        refs = []
        for b in range(2):
            args = [host(x[c.rows(b)]) for x in (c.q, c.k, c.v)]
            refs.append((bo.linear(*args, c.g, c.scale, host(c.state[b]))[0],
                         bo.linear(*map(np.abs, args), c.g, c.scale, np.abs(host(c.state[b])))[0]))
        ref, size = (np.concatenate(x) for x in zip(*refs))
        x = getattr(c, which).clone()
        x[at, 0, 5] = bad
        setattr(c, which, x)
        s = c.state.clone()
        o = c.run(ttt, s)
        heads = c.hq // c.hk      # the heads that see state head 0
        clean = np.ones(c.n, bool)
        clean[at:lens[0]] = False
        for rows, hs in ((clean, slice(0, heads)), (np.ones(c.n, bool), slice(heads, None))):
            close(host(o)[rows, hs], ref[rows, hs], size[rows, hs], c.coef, dtype, "few" if lens[0] <= FEW else "o", c.dk)
        if which == "q":
            assert not torch.isfinite(o[at, 0]).all() and torch.isfinite(o[at + 1:]).all() and torch.isfinite(s).all()
        else:
            assert not torch.isfinite(o[at, :heads]).all() and not torch.isfinite(s[0, 0]).all() and torch.isfinite(s[1]).all()


def test_nothing_to_do(ttt):
    c = Case([0, 0])
    s = c.state.clone()
    assert c.run(ttt, s, max_new=1).shape == (0, c.hq, c.dv) and torch.equal(s, c.state)
    got = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, q_starts=c.starts, state=c.state, d_state=c.d_state)
    assert torch.equal(got[3], c.d_state) and got[0].shape == c.q.shape
    got = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, q_starts=c.starts, state=c.state)
    assert (got[3] == 0).all()


@pytest.mark.parametrize("lens", [[1], [8], [64], [65], [0, 130, 1, 0, 64]])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [1, 3])
def test_gradients_lengths(ttt, lens, dtype, group):
    Case(lens, dtype=dtype, group=group).check_backward(ttt)


@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("dv", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_dims(ttt, dk, dv, dtype):
    Case([100, 37], dk=dk, dv=dv, dtype=dtype).check_backward(ttt)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [1, 2])
def test_gradients_of_parts(ttt, dtype, group):
    Case([1100, 300, 0, 513], hk=1, dtype=dtype, group=group).check_backward(ttt)


@pytest.mark.parametrize("decays", [[0.0], [-1e-5, -20.0]])
def test_gradients_decays_and_missing_states(ttt, decays):
    c = Case([90], decays=decays, dtype=F32, group=2)
    c.check_backward(ttt)
    c.check_backward(ttt, state=None)
    c.check_backward(ttt, d_state=None)
    got = c.check_backward(ttt, state=None, d_state=None)
    assert got[3] is None
    d = c.d_state.clone()
    got = c.check_backward(ttt, d_state=d, d_state0=d)       # in its place
    assert got[3] is d
    long = Case([1100], hk=1, dtype=F32)
    d = long.d_state.clone()
    assert long.check_backward(ttt, d_state=d, d_state0=d)[3] is d


def test_gradients_against_differences(ttt):
    """Along a random direction of every input. The loss, summed in float64 from
    the kernel's outputs, is linear in each, so a difference over 0.2 has no error
    but the outputs' roundings: random ones of some 2^-22 each, 5 2^-22 |d loss / d o|
    |o| together, below 1e-4 of a gradient of the same sums."""
    c = Case([50], dtype=F32, dk=64, dv=64)
    got = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, state=c.state, d_state=c.d_state, scale=c.scale)

    def loss(x):
        s = x["state"].clone()
        o = ttt.linear_attention(x["q"], x["k"], x["v"], c.ld, state=s, scale=c.scale)
        return float((o.double() * c.do).sum() + (s.double() * c.d_state).sum())
    at = dict(q=c.q, k=c.k, v=c.v, state=c.state)
    for name, g in zip(("q", "k", "v", "state"), got):
        d = torch.randn_like(at[name])
        d /= d.norm()
        h = 0.1
        slope = (loss({**at, name: at[name] + h * d}) - loss({**at, name: at[name] - h * d})) / (2 * h)
        want = float((g.double() * d).sum())
        assert abs(slope - want) <= 1e-4 * float(g.double().norm()), (name, slope, want)


def test_the_same_every_time(ttt):
    c = Case([700, 90], hk=1, group=2)
    runs = []
    for _ in range(2):
        s = c.state.clone()
        runs.append((c.run(ttt, s), s, *ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, q_starts=c.starts, max_new=700)))
    assert all(torch.equal(a, b) for a, b in zip(*runs) if a is not None)


@pytest.mark.parametrize("lens", [[500, 60], [2, 1]])
def test_captured_and_on_another_stream(ttt, lens):
    c = Case(lens, hk=1, group=2)

    def both(**kw):
        s = c.state.clone()
        o = c.run(ttt, s, **kw)
        g = ttt.linear_attention_backward(c.do, c.q, c.k, c.v, c.ld, state=c.state, d_state=c.d_state, q_starts=c.starts,
                                          max_new=max(lens), **kw)
        return (o, s, *g)
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for _ in range(3):
        c.v.copy_(torch.randn_like(c.v))
        graph.replay()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
