"""Long runs of dependent operators without a wait in between, over buffers that are
written again and again: each kernel may start while the one before it ends, and
the results are those of the same calls with a wait after each."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops
from _ops_ref import Layer64, gen, nb, rand_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("T", [1, 8, 27])
def test_decoder_steps(T):
    """norm -> e4m3 product -> norm -> MoE layer -> norm, 24 steps on one stream."""
    d, n = 1024, 24
    L = Layer64(d, 64, 6, 256, 256, seed=1)
    w, sw = rand_weights((d, d), 2, std=0.03)
    mat = moe_ops.make_fp8_mat(w, sw)
    g = gen(3)
    pre = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
    norm = moe_ops.make_norm(d, pre, pre, True, branch_scale=0.5)
    x0 = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    x, h, c = (torch.empty_like(x0) for _ in range(3))
    codes = torch.empty(T, d, device="cuda", dtype=torch.uint8)
    scales = torch.empty(T, nb(d), device="cuda")
    ws = moe_ops.alloc_fp8_workspace(L.handle, T)

    def steps(wait):
        calls = [lambda: moe_ops.moe_norm_block(norm, x, None, None, T, None, None, codes, scales)]
        for _ in range(n):
            calls += [lambda: moe_ops.moe_fp8_gemm(mat, codes, scales, T, c, ws),
                      lambda: moe_ops.moe_norm_block(norm, x, c, None, T, x, h),
                      lambda: moe_ops.moe_fp8_layer_forward(L.handle, h, T, c, ws),
                      lambda: moe_ops.moe_norm_block(norm, x, c, None, T, x, h),
                      lambda: moe_ops.moe_fp8_quant(h, codes, scales)]
        for f in calls:
            f()
            if wait:
                torch.cuda.synchronize()

    def result(run):
        x.copy_(x0)
        run()
        torch.cuda.synchronize()
        assert moe.moe_workspace_error(ws) == (0, 0)
        return x.clone(), h.clone(), codes.clone(), scales.clone()

    ref = result(lambda: steps(True))
    assert torch.isfinite(ref[0].float()).all() and ref[0].float().std() > 0
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        steps(False)
    for _ in range(5):
        for run in (lambda: steps(False), graph.replay):
            for a, b in zip(result(run), ref):
                assert torch.equal(a, b)


def test_products_one_after_the_other():
    """Products of every kind of tile in turn, each reading what the one before
    wrote as its scales, 40 rounds."""
    K = 512
    sizes = [(4, 8192, 1), (300, 1000, 1), (2048, 4096, 1), (25, 2048, 30), (3000, 1024, 260)]
    runs = []
    for i, (M, N, G) in enumerate(sizes):
        w, sw = rand_weights((N, K) if G == 1 else (G, N, K), i, std=0.03)
        a = torch.randint(0, 100, (M, K), device="cuda", dtype=torch.uint8, generator=gen(i))
        runs.append((moe_ops.make_fp8_mat(w, sw), a, torch.empty(M, K // 128, device="cuda"), M,
                     (torch.arange(G + 1, device="cuda") * M // G).int(), G,
                     torch.empty(M, N, device="cuda", dtype=torch.bfloat16)))

    def go(wait, rounds=40):
        for *_, c in runs:
            c.fill_(0.01)
        for _ in range(rounds):
            prev = runs[-1][-1]
            for m, a, sa, M, off, G, c in runs:
                n = sa.numel()
                sa.copy_((prev.flatten()[:n].float().abs() * 1e-3 + 0.01).view_as(sa))
                if G == 1:
                    moe_ops.moe_fp8_gemm(m, a, sa, M, c)
                else:
                    moe_ops.moe_fp8_gemm_grouped(m, a, sa, M, off, c)
                if wait:
                    torch.cuda.synchronize()
                prev = c
        torch.cuda.synchronize()
        return [c.clone() for *_, c in runs]
    ref = go(True)
    assert all(torch.isfinite(c.float()).all() for c in ref)
    for _ in range(3):
        for a, b in zip(go(False), ref):
            assert torch.equal(a, b)
