"""Selection inside moe_fp8_layer_forward where values are equal or not finite."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops
from _ops_ref import Layer64, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def tokens(T, d, seed):
    return torch.randn(T, d, device="cuda", generator=gen(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("E", [16, 31, 32, 33, 64, 128, 129, 512, 513, 1024])
@pytest.mark.parametrize("T,k", [(1, 16), (4, 3), (8, 16), (9, 10)])
def test_equal_logits_go_to_the_lower_experts(E, T, k):
    """More equal candidates than a warp holds: the round-by-round selection for
    every range of experts, and keys staged a few tokens at a time above 512."""
    L = Layer64(64, E, k, 32, 0, seed=E, bias=False)
    L.router_w.zero_()
    x = tokens(T, 64, 1)
    y, ids, w, ws = L.run(x)
    assert moe.moe_workspace_error(ws) == (0, 0)
    assert (ids == torch.arange(k, device="cuda", dtype=torch.int32)).all()
    # k terms of e^0 = 1 add up exactly; one division rounds
    assert (w.double() - 1 / k).abs().max() <= 2.0 ** -24 / k
    L.check(x, y, ids, w)


@pytest.mark.parametrize("E,k,nan", [(16, 4, 9), (64, 10, 20), (512, 10, 300), (1024, 16, 1000),
                                     (40, 16, 23)])
@pytest.mark.parametrize("where", ["bias", "row"])
def test_nan_logits_come_last(E, k, nan, where):
    """`nan` experts have NaN logits and at least k have not: none of the former is
    selected, and the rest are ordered as without them."""
    L = Layer64(64, E, k, 32, 32, seed=E)
    x = tokens(8, 64, 2)
    out = torch.randperm(E, device="cuda", generator=gen(5))[:nan]
    ref = L.logits64(x)[0]
    (L.bias if where == "bias" else L.router_w)[out] = float("nan")
    y, ids, w, ws = L.run(x)
    assert moe.moe_workspace_error(ws) == (0, 0)
    assert not torch.isin(ids.long(), out).any()
    ref[:, out] = float("-inf")
    # the logits of these inputs lie further apart than fp32 errs (64 products)
    top = ref.sort(dim=1, descending=True, stable=True)
    gap = (top.values[:, :k] - top.values[:, 1:k + 1]).min()
    assert gap > 1e-4
    assert torch.equal(ids.long(), top.indices[:, :k])
    assert (w.double() - torch.softmax(top.values[:, :k], 1)).abs().max() <= 1e-5
    assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("E", [20, 40, 600])
def test_nan_logits_are_selected_where_nothing_else_is_left(E):
    """Two finite logits and k = 5: these two first, then the lowest experts of the
    rest; a weight over NaN is NaN, and so is the output."""
    k, T = 5, 3
    L = Layer64(64, E, k, 32, 0, seed=E)
    L.bias.fill_(float("nan"))
    L.bias[7], L.bias[11] = 50.0, 80.0
    y, ids, w, ws = L.run(tokens(T, 64, 3))
    assert ids.tolist() == [[11, 7, 0, 1, 2]] * T
    assert w.isnan().all() and y.isnan().all()


def test_experts_masked_by_an_infinite_bias():
    """A bias of -inf takes an expert out; where fewer than k are left the masked
    ones fill up in their order with weight 0."""
    E, k, T = 48, 6, 8
    L = Layer64(64, E, k, 32, 32, seed=4)
    L.bias.fill_(float("-inf"))
    L.bias[[3, 20, 41, 45]] = 0.0
    y, ids, w, _ = L.run(tokens(T, 64, 4))
    assert (ids[:, :4].sort(dim=1).values == torch.tensor([3, 20, 41, 45], device="cuda")).all()
    assert (ids[:, 4:] == torch.tensor([0, 1], device="cuda")).all()
    assert (w[:, 4:] == 0).all() and torch.isfinite(y.float()).all()


def test_eager_calls_beside_replayed_graphs():
    """Three captured graphs replay on streams and workspaces of their own while
    eager calls run on a fourth: the outputs are the same as alone."""
    L = Layer64(1024, 64, 6, 256, 256, seed=10)
    xs = [tokens(T, 1024, T) for T in (1, 5, 12)]
    refs = [L.run(x)[0] for x in xs]
    xe = tokens(8, 1024, 20)
    eager_ref, _, _, ws_e = L.run(xe)
    runs = []
    for x in xs:
        ws = moe_ops.alloc_fp8_workspace(L.handle, 32)
        y, s, gr = torch.empty_like(x), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(gr, stream=s):
            moe_ops.moe_fp8_layer_forward(L.handle, x, x.shape[0], y, ws)
        runs.append((gr, s, y, ws))
    se = torch.cuda.Stream()
    ye = [torch.empty_like(xe) for _ in range(10)]
    for _ in range(5):
        for _, _, y, _ in runs:
            y.zero_()
        for y in ye:
            y.zero_()
        torch.cuda.synchronize()
        for i in range(10):
            for gr, s, _, _ in runs:
                with torch.cuda.stream(s):
                    gr.replay()
            with torch.cuda.stream(se):
                moe_ops.moe_fp8_layer_forward(L.handle, xe, 8, ye[i], ws_e)
        torch.cuda.synchronize()
        for (_, _, y, _), r in zip(runs, refs):
            assert torch.equal(y, r)
        assert all(torch.equal(y, eager_ref) for y in ye)
    for *_, ws in runs + [(ws_e,)]:
        assert moe.moe_workspace_error(ws) == (0, 0)
