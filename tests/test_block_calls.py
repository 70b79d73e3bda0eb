"""CPU-only: more calls that the Python entry points of norms, linear attention
and AdamW take or refuse by themselves (nothing is launched, see
test_block_checks)."""
import pytest

from test_block_checks import BF, F32, I32, U8, bl, gpu, lib  # noqa: F401


def gradients(**kw):
    a = dict(do=gpu(12, 4, 128), q=gpu(12, 4, 64), k=gpu(12, 2, 64), v=gpu(12, 2, 128), log_decay=gpu(2, dtype=F32))
    a.update(kw)
    return bl.linear_attention_backward(**a)


def test_sequences_are_known_from_the_state_gradient(lib):  # noqa: F811
    """Each of three may be the one state that is given."""
    s = gpu(3, 2, 64, 128, dtype=F32)
    for kw in (dict(state=s), dict(d_state=s), dict(d_state0=s)):
        out = gradients(**kw)
        assert out[3].shape == s.shape and (out[3] is s) == ("d_state0" in kw)
    assert lib.calls == ["ttt_linear_attention_backward"] * 3
    for kw in (dict(state=s, d_state0=gpu(1, 2, 64, 128, dtype=F32)), dict(d_state0=gpu(5, 2, 64, 128, dtype=F32))):
        with pytest.raises(ValueError):
            gradients(**kw)
    assert len(lib.calls) == 3


def test_a_gradient_that_would_be_left_out_is_refused(lib):  # noqa: F811
    x = gpu(4, 64)
    for pre in (None, False):
        with pytest.raises(ValueError, match="dh without pre"):
            bl.block_norm_backward(x, x, x, x, pre=pre)
    assert not lib.calls
    bl.block_norm_backward(x, x, x, x, pre=True)
    bl.block_norm_backward(x, None, x, x)
    assert lib.calls == ["ttt_block_norm_backward"] * 2


@pytest.mark.parametrize("step", [1.0, "1", None])
def test_a_step_is_a_whole_number(lib, step):  # noqa: F811
    p, g, s = [gpu(7)], [gpu(7, dtype=F32)], gpu(2048, dtype=U8)
    with pytest.raises(TypeError):
        bl.adamw_step(p, g, s, lr=1e-3, step=step)
    assert not lib.calls
    bl.adamw_step(p, g, s, lr=1e-3, step=gpu(1, dtype=I32))
    bl.adamw_step([gpu(7, dtype=BF)], g, s, lr=1e-3, step=True)
    assert len(lib.calls) == 2


def test_a_state_of_other_tensors_or_bits_is_refused(lib):  # noqa: F811
    p, g = [gpu(300), gpu(7)], [gpu(300, dtype=F32), gpu(7, dtype=F32)]
    for bits, each in ((32, 2048), (8, 520)):
        s = gpu(3 * each, dtype=U8)
        bl.adamw_step(p, g, s, lr=1e-3, step=1, bits=bits)
        for q, h in ((p[:1], g[:1]), (p[1:], g[1:]), (p + p, g + g)):
            with pytest.raises(ValueError, match="state must be"):
                bl.adamw_step(q, h, s, lr=1e-3, step=1, bits=bits)
        with pytest.raises(ValueError, match="state must be"):
            bl.adamw_step(p, g, s, lr=1e-3, step=1, bits=40 - bits)
    assert lib.calls == ["ttt_adamw_step"] * 2


@pytest.mark.parametrize("sizes", [(), (0,), (1, 256, 257), (5000, 0, 7, 2048)])
def test_state_sizes_are_the_librarys(sizes):
    for bits in (8, 32):
        assert bl._state_bytes(sizes, bits) == bl.adamw_state_size(sizes, bits)
