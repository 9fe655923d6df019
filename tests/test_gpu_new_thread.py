"""Calls of the block's entry points from a thread that has made no CUDA call yet,
in a process of its own."""
import os
import subprocess
import sys

import pytest

from routed_expert_ffn_06_b200 import build

pytestmark = pytest.mark.gpu

CODE = """
import sys
import threading
import torch
sys.path.insert(0, "tests")
from routed_expert_ffn_06_b200 import moe, synth
from _util import GpuBlock

what, T = "%s", %d
wl = synth.WORKLOADS["tiny"]
layer = synth.make_layer(wl["shape"], seed=1, device="cuda", bias=wl["bias"], slot=wl["slot"])
x = synth.make_tokens(T, wl["shape"].d, seed=2, device="cuda")
gb = GpuBlock(layer, T)
split = moe.moe_router_split(gb.L)
gb.L.router_w_split = split.data_ptr()
_, ids, w = gb.route(x)
out = [torch.zeros(T, wl["shape"].E, device="cuda") if what == "route" else torch.zeros_like(x)
       for _ in range(2)]
torch.cuda.synchronize()

def call(o):
    s = torch.cuda.default_stream().cuda_stream
    if what == "route":
        moe.moe_route_topk(gb.L, x, T, 0, o, ids, w, gb.ws, stream=s)
    elif what == "prefill":
        moe.moe_expert_ffn_prefill(gb.L, x, T, ids, w, o, None, None, 0, gb.ws, stream=s)
    else:
        moe.moe_block_forward(gb.L, x, T, o, 0, gb.ws, stream=s)

failed = []
def work():
    try:
        call(out[0])
    except Exception as e:
        failed.append(repr(e))

t = threading.Thread(target=work)
t.start()
t.join()
assert not failed, failed
call(out[1])
torch.cuda.synchronize()
assert torch.equal(out[0], out[1]) and out[0].float().abs().max() > 0
"""


@pytest.mark.parametrize("what,T", [("route", 64), ("route", 4), ("prefill", 64), ("block", 64),
                                    ("block", 4)])
def test_first_cuda_call_of_a_thread(what, T):
    build.build()
    out = subprocess.run([sys.executable, "-c", CODE % (what, T)], cwd=build.ROOT,
                         capture_output=True, text=True, timeout=300,
                         env=dict(os.environ, PYTHONPATH=build.ROOT))
    assert out.returncode == 0, out.stderr[-2000:]
