"""GPU: large calls of rotary positions and the cache against the same rows in
small calls, bit for bit. A wave of a large call walks over several heads with
what it has loaded of its tokens; in small calls, which the other tests compare
with the oracle, it has one."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    import test_layer_gate_amd as m
    m.lib()
    return m


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rows(n, heads, dim, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, heads, dim, generator=g, device="cuda")
    x[n // 3, :, dim - 1] = float("inf")      # a token whose heads are NaN in the cache
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "neighbours"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 32), (80, 48)])
@pytest.mark.parametrize("backward", [False, True])
def test_rope_over_many_heads(ttt, dtype, inter, dim, rot, backward):
    """39 heads in strides of 20 or 10 (bf16 heads of 80: side by side): from the
    first tensor to the second within a walk."""
    n, hq, hk = 5301, 32, 7
    x = rows(n, hq + hk, dim, dtype, 1)
    q, k = x[:, :hq], x[:, hq:]
    table = ttt.rope_table(n + 5, rot, 1e4)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).contiguous()
    f = ttt.rope_backward if backward else ttt.rope_forward
    got = f(q, k, table, positions=pos, interleaved=inter)
    for a in range(0, n, 50):
        want = f(q[a:a + 50], k[a:a + 50], table, positions=pos[a:a + 50].contiguous(), interleaved=inter)
        for y, z in zip(got, want):
            assert torch.equal(y[a:a + 50].view(torch.uint8), z.view(torch.uint8)), a
    y = x.clone()      # in place, in the fused rows
    f(y[:, :hq], y[:, hq:], table, positions=pos, interleaved=inter, **dict(
        zip(("dq", "dk") if backward else ("q_out", "k_out"), (y[:, :hq], y[:, hq:]))))
    assert torch.equal(y[:, :hq].contiguous().view(torch.uint8), got[0].view(torch.uint8))
    assert torch.equal(y[:, hq:].contiguous().view(torch.uint8), got[1].view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "neighbours"])
@pytest.mark.parametrize("n,dim,rot", [(8193, 64, 64), (8193, 64, 32), (20001, 128, 128), (12001, 256, 96), (20001, 128, 0)])
def test_cache_over_many_heads(ttt, dtype, inter, n, dim, rot):
    """13 + 2 x 3 heads in strides of 10, 5 or 3: queries to keys to values
    within a walk, the last heads' waves with one fewer."""
    hq, hk, page = 13, 3, 48
    x = rows(n, hq + 2 * hk, dim, dtype, 2)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    news, before = [n - 5001, 1, 5000], [3, 100, 40]
    starts = np.concatenate([[0], np.cumsum(news)])
    need = [-(-(a + b) // page) for a, b in zip(news, before)]
    ids = np.random.default_rng(3).permutation(sum(need))
    table = np.full((3, max(need)), -1)
    for b, at in enumerate(np.concatenate([[0], np.cumsum(need)[:-1]])):
        table[b, :need[b]] = ids[at:at + need[b]]
    table[2, 7] = -1                          # a page that is none
    rope = dict(rope_table=ttt.rope_table(n + 200, rot, 1e4), interleaved=inter) if rot else {}

    def pool():
        return torch.full((len(ids), hk, page * dim * 17 // 16), 85, dtype=torch.uint8, device="cuda")
    big, small, place = pool(), pool(), pool()
    lens = np.array(news) + before
    args = (ints(table), ints(lens))
    got = ttt.kv_append(big, *args, k, v, q=q if rot else None, q_starts=ints(starts), **rope)
    read = ttt.kv_read(big, *args, n, dim, dtype, q_starts=ints(starts))
    for b in range(3):
        for a in range(0, news[b], 100):
            m = min(100, news[b] - a)
            r = slice(starts[b] + a, starts[b] + a + m)
            few = (ints(table[b:b + 1]), ints([before[b] + a + m]))
            y = ttt.kv_append(small, *few, k[r], v[r], q=q[r] if rot else None, **rope)
            if rot:
                assert torch.equal(y.view(torch.uint8), got[r].view(torch.uint8)), (b, a)
            for z, w in zip(read, ttt.kv_read(small, *few, m, dim, dtype)):
                assert torch.equal(z[r].view(torch.uint8), w.view(torch.uint8)), (b, a)
    assert torch.equal(big, small)
    if rot:      # queries rotated in place
        y = x.clone()
        ttt.kv_append(place, *args, k, v, q=y[:, :hq], q_out=y[:, :hq], q_starts=ints(starts), **rope)
        assert torch.equal(place, big)
        assert torch.equal(y[:, :hq].contiguous().view(torch.uint8), got.view(torch.uint8))
        assert torch.equal(y[:, hq:].contiguous().view(torch.uint8), x[:, hq:].contiguous().view(torch.uint8))
