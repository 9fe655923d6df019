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


def _layer(**kw):
    d, E, F = 64, 4, 32
    fp8 = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn)   # noqa: E731
    a = dict(router_w=torch.zeros(E, d), router_bias=None, gate_up=fp8(E, 2, F, d),
             gate_up_scales=torch.zeros(E, 2, 1, 1), down=fp8(E, d, F),
             down_scales=torch.zeros(E, 1, 1))
    a.update(kw)
    return moe_ops.make_fp8_layer(2, **a)


def test_what_is_no_tensor_of_the_right_rank_is_a_value_error(monkeypatch):
    """None, or a tensor of another rank, in place of each tensor whose shape the
    binding reads; the message names it."""
    monkeypatch.setattr(moe_ops, "_current", lambda: HOST)     # host tensors stand for the device's
    f8, f32 = torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(1, 1)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    assert moe_ops.make_fp8_mat(f8, f32).struct.n == 4
    assert _layer().struct.n_experts == 4
    for bad in (None, 3.0, torch.zeros(4)):
        with pytest.raises(ValueError, match="codes"):
            moe_ops.make_fp8_mat(bad, f32)
        with pytest.raises(ValueError, match="scales"):
            moe_ops.make_fp8_mat(f8, bad)
        with pytest.raises(ValueError, match="x"):
            moe_ops.moe_fp8_quant(bad, f8, f32)
        with pytest.raises(ValueError, match="codes"):
            moe_ops.moe_fp8_quant(x, bad, f32)
        for name in ("router_w", "gate_up", "gate_up_scales", "down", "down_scales"):
            with pytest.raises(ValueError, match=name):
                _layer(**{name: bad})
        with pytest.raises(ValueError, match="shared_gate_up"):
            _layer(shared_gate_up=3.0 if bad is None else bad)
        with pytest.raises(ValueError, match="shared_down"):
            _layer(shared_gate_up=torch.zeros(2, 32, 64, dtype=torch.float8_e4m3fn),
                   shared_gate_up_scales=torch.zeros(2, 1, 1), shared_down=bad,
                   shared_down_scales=torch.zeros(1, 1))
