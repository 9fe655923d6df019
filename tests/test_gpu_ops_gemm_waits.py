"""Waits of the e4m3 products that run out, without a fault: the last word of the
workspace's control block makes one role of thread block 0 issue nothing (1: the
MMAs, so that the copies of a whole ring are in flight when the loader's wait for a
free stage gives up; 2: the copies)."""
import time

import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops
from _ops_ref import gen, quant_rows, rand_weights

pytestmark = pytest.mark.gpu

HOLD = 63           # word of the control block: 1 no MMAs, 2 no copies
LIMIT_US = 2000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# few rows, some rows, wide tiles; one weight matrix, and one for each of many groups;
# thread block 0 has more blocks of K than the ring has stages in every case
@pytest.mark.parametrize("who", [1, 2])
@pytest.mark.parametrize("M,N,K,G", [(4, 512, 8192, 1), (100, 640, 8192, 1), (2048, 4096, 2048, 1),
                                     (20, 2048, 4096, 40), (4096, 1024, 2048, 300)])
def test_a_wait_that_runs_out_ends_the_call_and_the_next_is_clean(M, N, K, G, who):
    a, sa = quant_rows(torch.randn(M, K, device="cuda", generator=gen(1)))
    shape = (N, K) if G == 1 else (G, N, K)
    w, sw = rand_weights(shape, 2)
    m = moe_ops.make_fp8_mat(w, sw)
    off = (torch.arange(G + 1, device="cuda") * M // G).int()
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:256]
    words = ws.view(torch.int32)

    def call():
        c = torch.full((M, N), float("nan"), device="cuda", dtype=torch.bfloat16)
        if G == 1:
            moe_ops.moe_fp8_gemm(m, a, sa, M, c, ws)
        else:
            moe_ops.moe_fp8_gemm_grouped(m, a, sa, M, off, c, ws)
        return c

    ref = call()
    assert moe.moe_workspace_error(ws) == (0, 0) and not ref.isnan().any()
    moe.moe_workspace_set_wait_limit(ws, LIMIT_US)
    words[HOLD] = who
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 0.5                 # a few limits, not the default second
    # the wait for a free stage, for a full one, or for an accumulator; no copy was lost
    assert words[4].item() & ~0x10 in (0x401, 0x404, 0x406)
    assert moe.moe_workspace_error(ws) == (7, 1)          # timeout
    words[HOLD] = 0
    assert torch.equal(call(), ref)
    assert moe.moe_workspace_error(ws) == (0, 0)
