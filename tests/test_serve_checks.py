"""CPU-only: what the Python entry points of the attention half of a block
refuse by themselves, before the library is asked. Nothing is launched: the
tensors say that they are on the GPU, and the library's functions only count
their calls."""
import pytest
import torch

from test_layer_gate_amd import _serve as sv

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


class OnGpu(torch.Tensor):
    is_cuda = True


def gpu(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


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
    monkeypatch.setattr(sv, "_L", lambda: L)
    monkeypatch.setattr(sv, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(sv, "_workspace", lambda *a: 0)
    return L


def attention(**kw):
    q, pages = gpu(6, 4, 64), gpu(3, 2, 16 * 68, dtype=U8)
    return sv.kv_attention(q, pages, gpu(2, 1, dtype=I32), gpu(2, dtype=I32), **kw)


def test_attention_takes_the_callers_buffers(lib):
    lse, ws = gpu(6, 4, dtype=F32), gpu(512, dtype=U8)
    o, got = attention(lse=lse, workspace=ws)
    assert got is lse and o.shape == (6, 4, 64) and lib.calls == ["ttt_kv_attention"]
    attention(workspace=gpu(64, dtype=F32))      # any type: its bytes count
    assert len(lib.calls) == 2


@pytest.mark.parametrize("kw", [
    dict(lse=torch.zeros(6, 4)),                               # in host memory
    dict(lse=gpu(6, 4)),                                       # bf16
    dict(lse=gpu(6, 8, dtype=F32)[:, :4]),                     # rows apart
    dict(lse=gpu(6, 3, dtype=F32)),
    dict(workspace=torch.zeros(512, dtype=U8)),                # in host memory
    dict(workspace=gpu(512, dtype=U8)[::2]),
    dict(workspace=gpu(1, dtype=U8).expand(4096)),             # more elements than bytes
])
def test_attention_refuses_buffers_that_the_kernels_cannot_write(lib, kw):
    with pytest.raises(ValueError):
        attention(**kw)
    assert not lib.calls


def test_rope_table_is_made_on_the_gpu(lib):
    with pytest.raises(ValueError):
        sv.rope_table(64, 32, device="cpu")
    assert not lib.calls


MANY = 2 ** 32 + 1       # 1 in 32 bits


@pytest.mark.parametrize("call", [
    lambda x: sv.kv_append(gpu(3, 2, 16 * 68, dtype=U8), gpu(1, 1, dtype=I32), gpu(1, dtype=I32), x, x),
    lambda x: sv.rope_forward(x, None, gpu(8, 16, 2, dtype=F32), positions=gpu(1, dtype=I32).expand(MANY), q_out=x),
    lambda x: sv.kv_attention(x, gpu(3, 2, 16 * 68, dtype=U8), gpu(1, 1, dtype=I32), gpu(1, dtype=I32), out=x,
                              max_new=1, workspace=gpu(512, dtype=U8)),
    lambda x: sv.kv_read(gpu(3, 2, 16 * 68, dtype=U8), gpu(1, 1, dtype=I32), gpu(1, dtype=I32), MANY, 64, k_out=x,
                         v_out=x),
], ids=["append", "rope", "attention", "read"])
def test_rows_past_32_bits_are_refused(lib, call):
    """The library counts rows in 32 bits: 2^32 + 1 of them would be one."""
    with pytest.raises(ValueError, match="rows"):
        call(gpu(1, 2, 64).expand(MANY, 2, 64))
    assert not lib.calls


@pytest.mark.parametrize("kw", [dict(max_pos=MANY, rot_dim=0), dict(max_pos=0, rot_dim=MANY)])
def test_rope_tables_past_32_bits_are_refused(lib, kw):
    with pytest.raises(ValueError, match="2\\^31"):
        sv.rope_table(**kw, device="meta")
    assert not lib.calls


@pytest.mark.parametrize("size", [sv.kv_attention_workspace_size, sv.kv_attention_plan])
def test_sizes_of_other_types_are_refused(size):
    """As the call itself refuses them."""
    for dtype in (torch.float16, torch.float64, None):
        with pytest.raises(TypeError):
            size(1, 1, 8, 32, 128, dtype, max_new=1, max_kv=1 << 17)
    assert size(1, 1, 8, 32, 128, F32, max_new=1, max_kv=1 << 17)
