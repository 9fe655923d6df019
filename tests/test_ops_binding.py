"""Refusals of the binding in moe_ops.py that need no GPU."""
import pytest
import torch

from routed_expert_ffn_06_b200 import moe_ops

HOST = -1


def test_a_workspace_below_the_control_block_is_refused():
    """The products write an error word into the 256 bytes of the control block
    and have no size to check: the binding does."""
    assert moe_ops._workspace(None, HOST) is None
    ws = torch.zeros(256, dtype=torch.uint8)
    assert moe_ops._workspace(ws, HOST) == ws.data_ptr()
    for n in (0, 16, 255):
        with pytest.raises(ValueError, match="256"):
            moe_ops._workspace(ws[:n], HOST)
