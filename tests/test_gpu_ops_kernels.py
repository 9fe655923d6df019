"""Every kernel of the e4m3 products against 64-bit products."""
import pytest
import torch

from _ops_cases import DENSE, GROUPED
from _ops_ref import BF16, gen, product64, quant_rows, rand_weights
from routed_expert_ffn_06_b200 import build, moe, moe_ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def acts(M, K, seed):
    x = torch.randn(M, K, device="cuda", generator=gen(seed))
    x[:, :: max(1, K // 3)] *= 20
    return quant_rows(x)


def compare(c, ref, bound):
    err, tol = (c.double() - ref).abs(), bound * (1 + BF16) + BF16 * ref.abs()
    assert (err <= tol).all(), f"worst {(err / tol.clamp_min(1e-300)).max().item():.3f} of the bound"


def workspace():
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    return ws[(-ws.data_ptr()) % 256:][:256]


def ids(cases):
    return [f"{'x'.join(map(str, c[3]))}-{i}" for i, c in enumerate(cases)]


@pytest.mark.parametrize("M,N,K,plan", DENSE, ids=ids(DENSE))
def test_dense(M, N, K, plan):
    a, sa = acts(M, K, M + N)
    w, sw = rand_weights((N, K), K)
    m = moe_ops.make_fp8_mat(w, sw)
    assert moe_ops.moe_fp8_gemm_plan(m, M) == plan
    buf = torch.full((M + 2, N), 7.0, device="cuda", dtype=torch.bfloat16)
    c, ws = buf[1:M + 1], workspace()
    moe_ops.moe_fp8_gemm(m, a, sa, M, c, ws)
    assert moe.moe_workspace_error(ws) == (0, 0)
    compare(c, *product64(a, sa, w, sw))
    assert (buf[0] == 7).all() and (buf[M + 1] == 7).all()


@pytest.mark.parametrize("lead", [0, 5])
@pytest.mark.parametrize("counts,N,K,plan", GROUPED, ids=ids(GROUPED))
def test_grouped(counts, N, K, plan, lead):
    G, tail = len(counts), lead
    off = (lead + torch.tensor([0] + counts).cumsum(0)).int().cuda()
    rows = sum(counts)
    M = lead + rows + (tail if rows + lead + tail <= 32 or rows > 32 else 0)
    a, sa = acts(M, K, G + N)
    w, sw = rand_weights((G, N, K), K)
    m = moe_ops.make_fp8_mat(w, sw)
    assert moe_ops.moe_fp8_gemm_plan(m, M, True) == plan
    buf = torch.full((M + 2, N), 7.0, device="cuda", dtype=torch.bfloat16)
    c, ws = buf[1:M + 1], workspace()
    moe_ops.moe_fp8_gemm_grouped(m, a, sa, M, off, c, ws)
    assert moe.moe_workspace_error(ws) == (0, 0)
    o = off.tolist()
    for g in range(G):
        if counts[g]:
            r = slice(o[g], o[g + 1])
            compare(c[r], *product64(a[r], sa[r], w[g], sw[g]))
    assert (c[:lead] == 7).all() and (c[o[G]:] == 7).all()      # rows of no group
    assert (buf[0] == 7).all() and (buf[M + 1] == 7).all()
