"""Calls from a thread that has made no CUDA call yet, in a process of its own."""
import os
import subprocess
import sys

import pytest

from routed_expert_ffn_06_b200 import build

pytestmark = pytest.mark.gpu

CODE = """
import threading
import torch
from routed_expert_ffn_06_b200 import moe, moe_ops, synth

what = "%s"
g = torch.Generator(device="cuda")
g.manual_seed(1)
M, N, K, G = dict(narrow=(4, 64, 512, 1), tiles=(300, 200, 512, 1), wide=(8192, 4096, 256, 1),
                  grouped=(60, 96, 512, 5)).get(what, (8, 256, 256, 1))
a = torch.randint(0, 100, (M, K), device="cuda", dtype=torch.uint8, generator=g)
w = torch.randint(0, 100, (G, N, K) if G > 1 else (N, K), device="cuda", dtype=torch.uint8, generator=g)
sa, sw = torch.ones(M, K // 128, device="cuda"), torch.ones(*w.shape[:-2], -(-N // 128), K // 128, device="cuda")
m = moe_ops.make_fp8_mat(w, sw)
off = (torch.arange(G + 1, device="cuda") * M // G).int()
x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
norm = moe_ops.make_norm(K)
E, F = 8, 64
fp8 = lambda *s: torch.randint(0, 100, s, device="cuda", dtype=torch.uint8, generator=g)
one = lambda *s: torch.full(s, 2.0 ** -6, device="cuda")
layer = moe_ops.make_fp8_layer(2, torch.randn(E, K, device="cuda", generator=g), None, fp8(E, 2, F, K),
                               one(E, 2, 1, -(-K // 128)), fp8(E, K, F), one(E, -(-K // 128), 1))
c = [torch.zeros(M, N if what in ("narrow", "tiles", "wide", "grouped") else K, device="cuda",
                 dtype=torch.bfloat16) for _ in range(2)]
codes, scales = torch.zeros(M, K, device="cuda", dtype=torch.uint8), torch.zeros(M, K // 128, device="cuda")
ws = torch.zeros(1 << 22, device="cuda", dtype=torch.uint8)
ws = ws[(-ws.data_ptr()) %% 256:][:1 << 21]
torch.cuda.synchronize()

def call(o):
    s = torch.cuda.default_stream().cuda_stream
    if what == "norm":
        moe_ops.moe_norm_block(norm, x, None, None, M, None, o, stream=s)
    elif what == "quant":
        moe_ops.moe_fp8_quant(x, codes, scales, stream=s)
        o.view(torch.uint8)[:, :K].copy_(codes)
    elif what == "layer":
        moe_ops.moe_fp8_layer_forward(layer, x, M, o, ws, stream=s)
    elif G > 1:
        moe_ops.moe_fp8_gemm_grouped(m, a, sa, M, off, o, stream=s)
    else:
        moe_ops.moe_fp8_gemm(m, a, sa, M, o, stream=s)

failed = []
def work():
    try:
        call(c[0])
    except Exception as e:
        failed.append(repr(e))

t = threading.Thread(target=work)
t.start()
t.join()
assert not failed, failed
call(c[1])
torch.cuda.synchronize()
assert torch.equal(c[0], c[1]) and c[0].float().abs().max() > 0
"""


@pytest.mark.parametrize("what", ["norm", "quant", "narrow", "tiles", "wide", "grouped", "layer"])
def test_first_cuda_call_of_a_thread(what):
    build.build()
    out = subprocess.run([sys.executable, "-c", CODE % what], cwd=build.ROOT, capture_output=True,
                         text=True, timeout=300, env=dict(os.environ, PYTHONPATH=build.ROOT))
    assert out.returncode == 0, out.stderr[-2000:]
