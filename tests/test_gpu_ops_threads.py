"""First calls of a process from several threads at once."""
import os
import subprocess
import sys

import pytest

from routed_expert_ffn_06_b200 import build

pytestmark = pytest.mark.gpu

CODE = """
import threading
import torch
from routed_expert_ffn_06_b200 import moe_ops

M, N, K, n = 40, 300, 512, 8
codes = torch.randint(0, 100, (M, K), device="cuda", dtype=torch.uint8)
w = torch.randint(0, 100, (N, K), device="cuda", dtype=torch.uint8)
sa, sw = torch.rand(M, K // 128, device="cuda"), torch.rand(-(-N // 128), K // 128, device="cuda")
m = moe_ops.make_fp8_mat(w, sw)
c = [torch.zeros(M, N, device="cuda", dtype=torch.bfloat16) for _ in range(n)]
torch.cuda.synchronize()
meet, failed = threading.Barrier(n), []

def work(i):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            meet.wait()
            moe_ops.moe_fp8_gemm(m, codes, sa, M, c[i])
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        failed.append(repr(e))

ts = [threading.Thread(target=work, args=(i,)) for i in range(n)]
for t in ts:
    t.start()
for t in ts:
    t.join()
assert not failed, failed
r = [torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128]
A = codes.view(torch.float8_e4m3fn).double() * sa.double()[:, r[1]]
W = w.view(torch.float8_e4m3fn).double() * sw.double()[r[0]][:, r[1]]
# 128 products and 4 blocks, each addition off by at most a whole fp32 step, 2^-23;
# all terms are positive; then half a step of bf16
ref = A @ W.T
assert ((c[0].double() - ref).abs() <= (2 ** -8 + 140 * 2 ** -23) * ref).all()
assert all(torch.equal(o, c[0]) for o in c)
"""


def test_products_called_first_by_eight_threads():
    build.build()
    out = subprocess.run([sys.executable, "-c", CODE], cwd=build.ROOT, capture_output=True, text=True,
                         timeout=300, env=dict(os.environ, PYTHONPATH=build.ROOT))
    assert out.returncode == 0, out.stderr[-2000:]
