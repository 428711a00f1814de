"""Workspaces and plans of a recurrent block's operators, without a GPU."""
import pytest

from test_block_cpu import recur
from test_sequence_cpu import BF16C, OK, Stride, size


@pytest.mark.parametrize("row", [0, 4096, 1 << 20])
def test_one_token_sequences_take_little_workspace(row):
    """A dense batch of one-token sequences is as many rows, however the stride over its tokens is given: some tens of
    chunks, each with a handful of fp32 rows."""
    s = Stride(row, 4096)
    for seqs, most in ((1024, 1 << 20), (16384, 12 << 20), (150000, 120 << 20)):
        p = recur(seqs=seqs, len=1, tokens=seqs, d=4096, x=s, r=Stride(row, 8192), i=Stride(row, 8192), z=s, dy=s)
        assert size("gated_recurrence_workspace_size", p, BF16C) == (OK, 0)
        status, need = size("gated_recurrence_grad_workspace_size", p, BF16C)
        assert status == OK and need < most
