"""The example block (rotary positions, 4-bit cache, attention, fast-weight
layer) on the GPU: a prompt in segments, then single tokens, against the same
block in float64 with the oracle's quantisation.

Tolerance, relative in the Frobenius norm of what the block adds to its input.
fp32: the layer's own, and a code of the cache that fp32's rounding turns over
once in some 10^5 values. bf16: a projection's rounding (2^-8 at most, some
2^-9.5 rms of a value) crosses a code's boundary with probability twice that
over half a step; the value is then off by a step. With steps of about half a
value that is an rms error of sqrt(2 * 2^-9.5 * 0.5) = 4% of the keys and
values, of the attention's output likewise, and, where the attention adds a
third of its input's size, 1.3% of the layer's input; the layer's output is of
up to the fifth power of it (two gated products and the update). 10% holds
them and the layer's own."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle.serve_oracle as so
import oracle.ttt_oracle as ora
from test_parity import O_TOL

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a GPU")
    spec = importlib.util.spec_from_file_location("decoder_block", os.path.join(ROOT, "examples", "decoder_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def host(t):
    return t.detach().double().cpu().numpy()


def norm(x):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)


def reference(block, x0, base):
    x, w, m = host(x0), {k: host(v) for k, v in block.w.items()}, {k: host(v) for k, v in block.mlp.items()}
    B, T, d = x.shape
    cs = so.table(T, block.dim, base)
    x1 = x.copy()
    for b in range(B):
        q, k, v = ((norm(x[b]) @ w[n].T).reshape(T, -1, block.dim) for n in ("Wq", "Wk", "Wv"))
        q, k = so.rotate(q, cs, False), so.rotate(k, cs, False)
        o = so.attend(q, so.decode(*so.encode(k)), so.decode(*so.encode(v)), np.ones(T, bool), T, block.dim ** -0.5)[0]
        x1[b] += o.reshape(T, -1) @ w["Wo"].T
    O, W = ora.ttt_prefill(norm(x1), x, m["Wg"], m["Wu"], m["W_down0"], m["taps"], m["W_target"], block.eta,
                           block.chunk, pad="chunk")
    return x1 + O - x


@pytest.mark.parametrize("config,segments,new,heads,kv_heads,dim,tol", [
    ("tiny", [64, 128], 70, 2, 1, 64, O_TOL + 4e-3),
    ("tiny", [192], 1, 3, 3, 128, O_TOL + 4e-3),
    ("mid_amp", [512, 256], 40, 4, 2, 64, 0.1)])
def test_segments_then_single_tokens(example, config, segments, new, heads, kv_heads, dim, tol):
    T = sum(segments) + new
    block, x0 = example.random_block(config, 2, T, heads, kv_heads, dim, seed=3, seq_len=T, page=16, base=1e4)
    y, at = [], 0
    for n in segments:
        part = x0[:, at:at + n].contiguous()
        y.append(block.segment(part, part))
        at += n
    for t in range(at, T):
        part = x0[:, t].contiguous()
        y.append(block.step(part, part)[:, None])
    torch.cuda.synchronize()
    assert block.lens.tolist() == [T, T]
    ref = reference(block, x0, 1e4)
    added = host(torch.cat(y, 1)) - host(x0)
    err = np.linalg.norm(added - ref) / np.linalg.norm(ref)
    tail = np.linalg.norm((added - ref)[:, at:]) / np.linalg.norm(ref[:, at:])
    print(f"{config}: {err:.2e}, single tokens {tail:.2e}", flush=True)
    assert err <= tol and tail <= tol
    with pytest.raises(ValueError):
        block.segment(x0[:, :block.chunk].contiguous(), x0[:, :block.chunk].contiguous())
