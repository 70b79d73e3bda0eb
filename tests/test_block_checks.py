"""CPU-only: what the Python entry points of norms, linear attention and AdamW
refuse by themselves, before the library is asked. Nothing is launched: the
tensors say that they are on the GPU, and the library's functions only count
their calls."""
import pytest
import torch

from test_layer_gate_amd import _block as bl
from test_layer_gate_amd import _serve as sv

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class OnGpu(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


def gpu(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Methods:
    """torch.Tensor's, as they are mapped over lists, of each tensor's own class."""
    get_device = staticmethod(lambda t: t.get_device())
    is_contiguous = staticmethod(lambda t: t.is_contiguous())
    numel = staticmethod(lambda t: t.numel())
    data_ptr = staticmethod(lambda t: t.data_ptr())


class Library:
    """Every function succeeds, and is counted."""
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    L = Library()
    monkeypatch.setattr(bl, "_L", lambda: L)
    monkeypatch.setattr(sv, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(bl, "_norm_workspace", lambda *a: 0)
    monkeypatch.setattr(bl, "_linear_workspace", lambda *a: 0)
    monkeypatch.setattr(bl, "_grad_norm_workspace", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bl, "_T", Methods)
    return L


def test_norm_takes_views(lib):
    x, f = gpu(4, 6, 64), gpu(24, 128)[:, :64]
    r, h = bl.block_norm(x, f.unflatten(0, (4, 6)), post=True, pre=gpu(64), gate=gpu(4, 1, 64), scale=0.5)
    assert r.shape == h.shape == (4, 6, 64) and lib.calls == ["ttt_block_norm"]
    assert bl.block_norm(x, pre=True)[0] is None and bl.block_norm(x, f, gate=gpu(64))[1] is None
    d = bl.block_norm_backward(None, h, r, f, pre=gpu(64), gate=gpu(4, 64))
    assert d["dgate"].dtype is F32 and d["dgate"].shape == (4, 64) and d["dpost"] is None and d["dpre"].shape == (64,)
    assert bl.block_norm_backward(r, None, r, f, gate=gpu(24, 64))["dgate"].dtype is BF


@pytest.mark.parametrize("call,error", [
    (lambda: bl.block_norm(torch.zeros(4, 64), gpu(4, 64)), ValueError),               # in host memory
    (lambda: bl.block_norm(gpu(4, 64), gpu(4, 64, dtype=torch.float16)), TypeError),
    (lambda: bl.block_norm(gpu(4, 64), gpu(3, 64)), ValueError),
    (lambda: bl.block_norm(gpu(4, 64), gpu(4, 128)[:, ::2]), ValueError),
    (lambda: bl.block_norm(gpu(4, 6, 64).transpose(0, 1), gpu(24, 64)), ValueError),
    (lambda: bl.block_norm(gpu(4, 64), gpu(4, 64), pre=gpu(32)), ValueError),
    (lambda: bl.block_norm(gpu(4, 64), gpu(4, 64), pre=gpu(64), post=gpu(64, dtype=F32)), TypeError),
    (lambda: bl.block_norm(gpu(4, 64), gpu(4, 64), gate=gpu(3, 64)), ValueError),
    (lambda: bl.block_norm(gpu(4, 64), gpu(4, 64), gate=gpu(4, 64, dtype=F32)), TypeError),
    (lambda: bl.block_norm(gpu(4, 64), gpu(4, 64), h=gpu(4, 64)), ValueError),
    (lambda: bl.block_norm(gpu(4, 64), r=gpu(4, 64), pre=True), ValueError),
    (lambda: bl.block_norm_backward(gpu(4, 64), None, None, pre=True), ValueError),
    (lambda: bl.block_norm_backward(None, None, None), ValueError),
    (lambda: bl.block_norm_backward(gpu(4, 64), gpu(4, 64), gpu(4, 64), pre=True, df=gpu(4, 64)), ValueError),
    (lambda: bl.block_norm_backward(gpu(4, 64), gpu(4, 64), gpu(4, 64), pre=gpu(64), dx=gpu(4, 64, dtype=F32)), TypeError),
])
def test_norm_refuses(lib, call, error):
    with pytest.raises(error):
        call()
    assert not lib.calls


def attend(**kw):
    a = dict(q=gpu(12, 4, 64), k=gpu(12, 2, 64), v=gpu(12, 2, 128), log_decay=gpu(2, dtype=F32))
    a.update(kw)
    return bl.linear_attention(**a)


def test_linear_takes_its_arguments(lib):
    assert attend().shape == (12, 4, 128)
    assert attend(state=gpu(3, 2, 64, 128, dtype=F32)).shape == (12, 4, 128)       # three sequences of four
    assert attend(q_starts=gpu(4, dtype=I32), state=gpu(3, 2, 64, 128, dtype=F32)).shape == (12, 4, 128)
    o = bl.linear_attention(gpu(2, 6, 4, 64), gpu(2, 6, 2, 64), gpu(2, 6, 2, 64), gpu(2, dtype=F32))
    assert o.shape == (2, 6, 4, 64)
    assert lib.calls == ["ttt_linear_attention"] * 4
    back = bl.linear_attention_backward(gpu(12, 4, 128), gpu(12, 4, 64), gpu(12, 2, 64), gpu(12, 2, 128), gpu(2, dtype=F32))
    assert back[3] is None and back[2].shape == (12, 2, 128)


@pytest.mark.parametrize("kw", [
    dict(k=gpu(12, 4, 64)), dict(k=gpu(12, 2, 128)), dict(v=gpu(11, 2, 128)), dict(log_decay=gpu(4, dtype=F32)),
    dict(log_decay=gpu(2)), dict(log_decay=torch.zeros(2)), dict(state=gpu(1, 2, 64, 64, dtype=F32)),
    dict(state=gpu(1, 2, 64, 128)), dict(state=gpu(5, 2, 64, 128, dtype=F32)), dict(q_starts=torch.zeros(3, dtype=I32)),
    dict(q_starts=gpu(3)), dict(q_starts=gpu(1, dtype=I32)), dict(out=gpu(12, 2, 128)), dict(out=gpu(12, 4, 64)),
    dict(q=gpu(12, 4, 128)[..., ::2]), dict(workspace=torch.zeros(64, dtype=U8)), dict(max_new=1 << 32),
    dict(q=torch.zeros(12, 4, 64, dtype=BF)),
])
def test_linear_refuses(lib, kw):
    with pytest.raises((ValueError, TypeError)):
        attend(**kw)
    assert not lib.calls


def test_adamw_takes_its_arguments(lib):
    p, g = [gpu(3, 5), gpu(7)], [gpu(3, 5, dtype=F32), gpu(7, dtype=F32)]
    s = gpu(512 * 2 + 16, dtype=U8)
    bl.adamw_step(p, g, s, lr=1e-3, step=1, bits=8)
    bl.adamw_step(p, g, s, lr=gpu(1, dtype=F32), step=gpu(1, dtype=I32), bits=8, masters=[t.float() for t in p],
                  norm=gpu(1, dtype=F32), max_norm=1.0)
    bl.adamw_step([], [], s, lr=1e-3, step=1)
    assert lib.calls == ["ttt_adamw_step"] * 2
    assert bl.grad_norm(g).dtype is F32
    m, v = bl.adamw_read(gpu(512 * 8, dtype=U8))
    assert m.shape == v.shape == (512,) and len(lib.calls) == 3


@pytest.mark.parametrize("call", [
    lambda p, g, s: bl.adamw_step(p, g[:1], s, lr=1e-3, step=1),
    lambda p, g, s: bl.adamw_step(p, [gpu(5, 3).t(), g[1]], s, lr=1e-3, step=1),
    lambda p, g, s: bl.adamw_step([p[0], gpu(7, dtype=F32)], g, s, lr=1e-3, step=1),
    lambda p, g, s: bl.adamw_step(p, [g[0], gpu(8, dtype=F32)], s, lr=1e-3, step=1),
    lambda p, g, s: bl.adamw_step(p, g, s.float(), lr=1e-3, step=1),
    lambda p, g, s: bl.adamw_step(p, g, s, lr=gpu(2, dtype=F32), step=1),
    lambda p, g, s: bl.adamw_step(p, g, s, lr=1e-3, step=gpu(1, dtype=F32)),
    lambda p, g, s: bl.adamw_step(p, g, s, lr=1e-3, step=1 << 40),
    lambda p, g, s: bl.adamw_step(p, g, s, lr=1e-3, step=1, masters=p),
    lambda p, g, s: bl.adamw_step(p, g, s, lr=1e-3, step=1, norm=1.0, max_norm=1.0),
    lambda p, g, s: bl.adamw_read(gpu(100, dtype=U8)),
    lambda p, g, s: bl.adamw_read(gpu(520, dtype=U8), 16),
    lambda p, g, s: bl.adamw_read(gpu(2048, dtype=U8), 32, dtype=BF),
    lambda p, g, s: bl.grad_norm([]),
    lambda p, g, s: bl.grad_norm(g, out=gpu(2, dtype=F32)),
    lambda p, g, s: bl.grad_norm([gpu(8, dtype=torch.float16)]),
    lambda p, g, s: bl.grad_norm([torch.zeros(4)]),
])
def test_adamw_refuses(lib, call):
    with pytest.raises((ValueError, TypeError)):
        call([gpu(3, 5), gpu(7)], [gpu(3, 5, dtype=F32), gpu(7, dtype=F32)], gpu(4096, dtype=U8))
    assert not lib.calls
