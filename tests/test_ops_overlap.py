"""Outputs that overlap inputs are refused on the host."""
import ctypes

import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe_ops

P = 0x7F0000000000          # made-up device addresses
# a call that passes the checks stops at the missing device; with a GPU it would run
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe_ops.load()


def layer_call(lib, x, y, T):
    names = ("router_w", "gate_up", "gate_up_scales", "down", "down_scales")
    L = moe_ops.moe_fp8_layer(d_model=64, n_experts=16, ffn=32, top_k=2, shared_ffn=0,
                              **{n: P + (1 << 28) + (i << 20) for i, n in enumerate(names)})
    return lib.moe_fp8_layer_forward(ctypes.addressof(L), x, T, y, None, None, P + (1 << 30), 1 << 26,
                                     None)


@pytest.mark.parametrize("T", [1, 9, 32])
def test_layer_rows(lib, T):
    n = T * 64 * 2
    for at in (0, 16, n - 16):
        assert layer_call(lib, P, P + at, T) == 1
        assert layer_call(lib, P + at, P, T) == 1


@no_gpu
def test_layer_rows_side_by_side(lib):
    assert layer_call(lib, P, P + 9 * 128, 9) == 8 and layer_call(lib, P + 9 * 128, P, 9) == 8
    assert layer_call(lib, P, P + 16, 0) == 8              # no rows, no overlap


def gemm_call(lib, a, sa, c, M, groups):
    m = moe_ops.moe_fp8_mat(n=100, k=256, groups=groups, codes=P + (1 << 28), scales=P + (1 << 29))
    if groups == 1:
        return lib.moe_fp8_gemm(ctypes.addressof(m), a, sa, M, c, None, None)
    return lib.moe_fp8_gemm_grouped(ctypes.addressof(m), a, sa, M, P + (1 << 30), c, None, None)


@pytest.mark.parametrize("groups", [1, 3])
def test_product(lib, groups):
    M = 7
    na, ns, nc = M * 256, M * 2 * 4, M * 100 * 2
    far = P + (1 << 24)
    for at in (0, na - 16):
        assert gemm_call(lib, P, far, P + at, M, groups) == 1
    for at in (0, ns - 4):
        assert gemm_call(lib, far, P, P + at, M, groups) == 1
    assert gemm_call(lib, P + nc - 8, far, P, M, groups) == 1
    assert gemm_call(lib, far, P + nc - 4, P, M, groups) == 1


@no_gpu
@pytest.mark.parametrize("groups", [1, 3])
def test_product_side_by_side(lib, groups):
    M, far = 7, P + (1 << 24)
    assert gemm_call(lib, P, far, P + M * 256, M, groups) == 8
    assert gemm_call(lib, far, P, P + M * 8, M, groups) == 8
    assert gemm_call(lib, P + M * 200 + 8, far, P, M, groups) == 8
    assert gemm_call(lib, P, far, P, 0, groups) == 8
