"""The example block takes a segment's inputs as a view of longer sequences, whose
rows are not evenly apart."""
import pytest
import torch

from test_parity_block import example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_segment_of_longer_sequences(example):  # noqa: F811
    outs = []
    for dense in (True, False):
        block, x0 = example.random_block("tiny", 2, 128, 2, 1, 64, seed=3, seq_len=128, page=16, base=1e4)
        y = []
        for at in (0, 64):
            part = x0[:, at:at + 64]
            assert not part.is_contiguous()
            y.append(block.segment(part.contiguous() if dense else part, part.contiguous()))
        outs.append(torch.cat(y, 1))
    assert torch.equal(*outs)
