"""CPU-only: how attention is launched, from sizes alone (ttt_kv_attention_plan
is host code)."""
import ctypes
import itertools

import pytest
import torch

import test_layer_gate_amd as ttt
from test_layer_gate_amd import _serve as sv

BF, F32 = torch.bfloat16, torch.float32
EDGE = 1 << 20      # workgroups that parts and tiles of rows are limited to


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_workgroups_stay_countable(dtype, dim):
    """The kernels number workgroups in 32 bits. max_kv and max_new are bounds
    that may be far too large: parts and tiles of rows stop at 2^20 workgroups,
    past which there is one a sequence and key head, 2^26 at most (of the
    many-row kernel, 2^20 a sequence)."""
    most = 0
    for batch, (hk, hq), max_new, max_kv, window in itertools.product(
            (1, 2, 255, 256, 257, 1000, 65535), ((1, 1), (1, 1024), (8, 32), (32, 32), (256, 256), (1024, 1024)),
            (1, 2, 33, 5000, 1 << 24), (1, 1024, 1025, 1 << 17, 1 << 24, 1 << 30, (1 << 31) - 1), (0, 1, 4096)):
        for tokens in (1, batch, 1 << 24):
            p = ttt.kv_attention_plan(batch, tokens, hk, hq, dim, dtype, max_new=max_new, max_kv=max_kv, window=window)
            case = (batch, hk, hq, max_new, max_kv, window, tokens, p)
            assert 1 <= p["workgroups"], case
            if p["many"]:
                assert p["parts"] * hk <= EDGE and p["workgroups"] // batch <= EDGE, case
            else:
                assert p["workgroups"] <= max(EDGE, batch * hk), case
                assert p["parts"] == 1 or p["parts"] * batch * hk <= EDGE, case
            most = max(most, p["workgroups"])
    assert most >= 65535 * 1024


def test_the_parts_that_pay_stay():
    """The limit is far from calls that need parts to fill the card."""
    assert ttt.kv_attention_plan(1, 1, 8, 40, 128, max_new=1, max_kv=131072)["parts"] == 64
    p = ttt.kv_attention_plan(300, 300, 8, 32, 128, max_new=1, max_kv=131072)
    assert p["parts"] == 1 and not p["slices"]
    assert ttt.kv_attention_plan(1, 1024, 8, 32, 128, max_new=1024, max_kv=65536)["many"]


def test_plan_refusals():
    p = sv.AttnPlan()
    a = sv.Attn(0.1, 0, 16, 1024, 0, 0)
    L = sv._L()
    assert L.ttt_kv_attention_plan(ctypes.byref(a), 1, 1, 0, 8, 32, 128, ctypes.byref(p)) == 0
    assert L.ttt_kv_attention_plan(ctypes.byref(a), 1, 1, 0, 8, 32, 128, None) == -1
    assert L.ttt_kv_attention_plan(None, 1, 1, 0, 8, 32, 128, ctypes.byref(p)) == -1
    assert L.ttt_kv_attention_plan(ctypes.byref(a), 0, 1, 0, 8, 32, 128, ctypes.byref(p)) == -1
    assert L.ttt_kv_attention_plan(ctypes.byref(a), 1, 1, 0, 8, 32, 96, ctypes.byref(p)) == -2
    assert ctypes.sizeof(sv.AttnPlan) == 32


def test_fp32_rows_of_wide_heads_share_long_keys():
    """A wave with a tile of its own pays where tiles are many; of fp32 rows with
    heads of 256, whose queries fill LDS, over short keys alone."""
    def waves(dim, dtype, batch, new, keys, window=0):
        return ttt.kv_attention_plan(batch, batch * new, 8, 32, dim, dtype, max_new=new, max_kv=keys, window=window)["waves"]
    for n in (2048, 8192):
        assert waves(256, F32, 2, n, n) == 4
        assert waves(256, BF, 2, n, n) == 1 and waves(128, F32, 2, n, n) == 1 and waves(64, F32, 2, n, n) == 1
    assert waves(256, F32, 4, 1024, 1024) == 1 and waves(256, F32, 2, 2048, 2048, window=64) == 1
    assert waves(256, F32, 1, 1024, 1024) == 4      # too few tiles
