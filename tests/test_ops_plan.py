"""The kernel that a product takes (no GPU needed)."""
import ctypes

import pytest
import torch

from _ops_cases import DENSE, GROUPED
from routed_expert_ffn_06_b200 import build, moe_ops

P = 0x7F0000000000

ALL = {(bn, 32, s) for bn, s in ((16, 7), (32, 5), (64, 3), (128, 4))} | {
    (bn, 128, s) for bn, s in ((16, 5), (32, 4), (64, 4), (128, 3), (256, 4), (256, 3))}


@pytest.fixture(scope="module")
def lib():
    build.build()
    if torch.cuda.is_available():
        assert torch.cuda.get_device_properties(0).multi_processor_count == 148
    return moe_ops.load()


def plan(lib, M, n, k, groups=1, grouped=0):
    m = moe_ops.moe_fp8_mat(n=n, k=k, groups=groups, codes=P, scales=P)
    out = (ctypes.c_int32 * 3)()
    st = lib.moe_fp8_gemm_plan(ctypes.addressof(m), M, grouped, out)
    return tuple(out) if st == 0 else st


def test_the_cases_take_every_kernel(lib):
    seen = set()
    for M, n, k, want in DENSE:
        assert plan(lib, M, n, k) == want, (M, n, k)
        seen.add(want)
    assert seen == ALL - {(256, 128, 3)}       # which needs many groups
    for counts, n, k, want in GROUPED:
        for lead in (0, 5):
            assert plan(lib, sum(counts) + lead, n, k, len(counts), 1) == want, (sum(counts), n, k)
        seen.add(want)
    assert seen == ALL


def test_no_other_kernel_is_planned(lib):
    for M in (1, 5, 32, 33, 100, 640, 5000, 81920, 2**31 - 256):
        for n in (1, 100, 1000, 4096, 65536):
            for g in (1, 2, 60, 240, 241, 512, 1024):
                assert plan(lib, M, n, 16, g, 1) in ALL
            assert plan(lib, M, n, 65536) in ALL


@pytest.mark.parametrize("groups", [300, 512, 1024])
@pytest.mark.parametrize("n", [1, 40, 1000, 4096])
def test_the_most_rows_are_planned_as_a_few_less(lib, groups, n):
    """Rows and groups add up beyond 2^31 without harm."""
    want = plan(lib, 2**31 - 4096, n, 16, groups, 1)
    for M in (2**31 - 1000, 2**31 - 513, 2**31 - 256):
        assert plan(lib, M, n, 16, groups, 1) == want


def test_ring_of_the_wide_kernel(lib):
    """Four stages up to 240 groups."""
    for g, stages in ((1, 4), (240, 4), (241, 3), (1024, 3)):
        assert plan(lib, 160 * g + 128, 65536, 128, g, 1) == (256, 128, stages)


def test_arguments(lib):
    assert plan(lib, 0, 64, 128) == 1 and plan(lib, 2**31 - 1, 64, 128) == 2
    assert plan(lib, 5, 64, 128, 3, 0) == 1 and plan(lib, 5, 64, 24) == 2
    m = moe_ops.moe_fp8_mat(n=64, k=128, groups=1, codes=P, scales=P)
    assert lib.moe_fp8_gemm_plan(ctypes.addressof(m), 5, 0, None) == 1
    assert lib.moe_fp8_gemm_plan(None, 5, 0, (ctypes.c_int32 * 3)()) == 1
