"""Grid waits of moe_fp8_layer_forward that are not reached."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops
from _ops_ref import Layer64, gen

pytestmark = pytest.mark.gpu

ERR_WHERE, FREE = 4, 6          # words of the control block: first failing site, the grid's counters


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("T", [1, 4, 8])
@pytest.mark.parametrize("short", [1, None, 1 << 20])
def test_no_block_goes_on_before_the_last_one_has_arrived(T, short):
    """The counter of the router's barrier starts `short` below zero (by the
    number of blocks: None; by far more, so that it stays below zero), so that all
    arrivals together do not reach the number waited for.  Every block's wait runs out: nothing is selected, no
    expert runs, and the routing outputs stay as they were."""
    L = Layer64(256, 32, 4, 64, 64, seed=3)
    x = (torch.randn(T, 256, device="cuda", generator=gen(1))).to(torch.bfloat16)
    y, ids, w, ws = L.run(x)
    moe.moe_workspace_set_wait_limit(ws, 2000)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    words = ws[:256].view(torch.int32)
    words[FREE] = -(short or sms)
    y2, ids2, w2, _ = L.run(x, ws)
    torch.cuda.synchronize()
    assert words[ERR_WHERE].item() == 0x500
    assert moe.moe_workspace_error(ws) == (7, 1)          # timeout
    assert (ids2 == -1).all() and w2.isnan().all() and (y2 == 0).all()
    y3, ids3, w3, _ = L.run(x, ws)                        # the counters are back at zero
    assert moe.moe_workspace_error(ws) == (0, 0)
    assert torch.equal(y, y3) and torch.equal(ids, ids3) and torch.equal(w, w3)
