"""The tensor cores' sums of e4m3 products hold the 24 bits of fp32."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe_ops

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# the places of a large product, a small one and the negative of the large one among
# the 128 columns of a block: in one k-step of 32, and in different ones
@pytest.mark.parametrize("at", [(0, 1, 2), (0, 1, 40), (0, 40, 1), (0, 40, 80), (40, 0, 41)])
@pytest.mark.parametrize("M,N", [(4, 64), (4, 16384), (100, 64), (2048, 4096)])
def test_products(M, N, at):
    """2^16 + 2^-7 - 2^16: each partial sum has 24 bits at most, so fp32 gives 2^-7
    in any order."""
    a, w = torch.zeros(M, 128, device="cuda"), torch.zeros(N, 128, device="cuda")
    a[:, at[0]], w[:, at[0]] = 256, 256
    a[:, at[1]], w[:, at[1]] = 2.0 ** -3, 2.0 ** -4
    a[:, at[2]], w[:, at[2]] = 256, -256
    c = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    m = moe_ops.make_fp8_mat(w.to(FP8), torch.ones(-(-N // 128), 1, device="cuda"))
    moe_ops.moe_fp8_gemm(m, a.to(FP8), torch.ones(M, 1, device="cuda"), M, c)
    assert (c == 2.0 ** -7).all()


@pytest.mark.parametrize("at", [(1, 2, 3), (1, 17, 2), (1, 2, 17), (1, 40, 70), (129, 130, 131)])
@pytest.mark.parametrize("T", [1, 8])
def test_gate_and_up_of_the_layer(T, at):
    """up = 2^15 + 2^-6 - 2^15 from tokens of 128, 1 and 128, gate = 32 = silu(32) in
    fp32; one channel goes on, so y = 32 * 2^-6."""
    d, F = 256, 32
    gu, dn = torch.zeros(1, 2, F, d, device="cuda"), torch.zeros(1, d, F, device="cuda")
    gu[0, 0, :, 0] = 1
    gu[0, 1, :, at[0]], gu[0, 1, :, at[1]], gu[0, 1, :, at[2]] = 256, 2.0 ** -6, -256
    dn[0, :, 5] = 1
    x = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    x[:, 0], x[:, at[0]], x[:, at[1]], x[:, at[2]] = 32, 128, 1, 128
    L = moe_ops.make_fp8_layer(1, torch.zeros(1, d, device="cuda"), None, gu.to(FP8),
                               torch.ones(1, 2, 1, 2, device="cuda"), dn.to(FP8),
                               torch.ones(1, 2, 1, device="cuda"))
    y = torch.empty_like(x)
    moe_ops.moe_fp8_layer_forward(L, x, T, y, moe_ops.alloc_fp8_workspace(L, T))
    assert (y == 0.5).all()
