"""moe_fp8_layer_forward against the 64-bit layer."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops
from _ops_ref import BF16, Layer64, gen, norm64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def tokens(T, d, seed, scale=1.0):
    return (torch.randn(T, d, device="cuda", generator=gen(seed)) * scale).to(torch.bfloat16)


@pytest.mark.parametrize("d,E,k,F,Fs,Ts", [
    (64, 16, 2, 32, 32, (1, 4, 8, 9)),
    (32, 4, 4, 32, 0, (1, 3)),                 # every expert selected, the smallest widths
    (96, 5, 1, 64, 64, (2, 8)),                # d below one scale block
    (160, 40, 3, 160, 0, (7, 32)),             # ragged scale blocks
    (1056, 40, 3, 160, 416, (7, 17)),          # shared wider than routed
    (2048, 64, 10, 512, 512, (1, 2, 4, 8)),
    (2080, 24, 6, 96, 64, (5,)),               # two scale blocks per warp, ragged
    (4096, 20, 16, 32, 32, (1, 8)),
    (256, 1024, 16, 64, 0, (8, 32)),           # the most experts
    (128, 9, 2, 4096, 4096, (3,)),             # the widest experts
    (512, 129, 8, 288, 96, (6, 31))])
def test_parity(d, E, k, F, Fs, Ts):
    L = Layer64(d, E, k, F, Fs, seed=d + E)
    for T in Ts:
        x = tokens(T, d, seed=T)
        y, ids, w, ws = L.run(x)
        assert moe.moe_workspace_error(ws) == (0, 0)
        L.check(x, y, ids, w)


def test_full_size_layer():
    L = Layer64(2048, 512, 10, 512, 512, seed=1)
    for T in (1, 4, 8, 20):
        x = tokens(T, 2048, seed=T)
        L.check(x, *L.run(x)[:3])


def test_no_bias_and_optional_routing_outputs():
    L = Layer64(256, 32, 4, 128, 128, seed=2, bias=False)
    x = tokens(5, 256, 3)
    y, ids, w, ws = L.run(x)
    L.check(x, y, ids, w)
    y2 = torch.empty_like(y)
    moe_ops.moe_fp8_layer_forward(L.handle, x, 5, y2, ws)
    assert torch.equal(y, y2)


def test_ties_go_to_the_lower_expert():
    L = Layer64(128, 64, 6, 64, 0, seed=4, bias=False)
    L.router_w.zero_()                                  # every logit equal
    x = tokens(8, 128, 1)
    y, ids, w, _ = L.run(x)
    assert (ids == torch.arange(6, device="cuda", dtype=torch.int32)).all()
    assert (w - 1 / 6).abs().max() <= 1e-7
    L.check(x, y, ids, w)
    L.router_w[40:44] = L.router_w.new_ones(128) * 0.25  # four equal rows, above or below the rest
    y, ids, w, _ = L.run(x)
    up = x.float().sum(1) > 0
    assert (ids[up][:, :4] == torch.arange(40, 44, device="cuda", dtype=torch.int32)).all()
    assert (ids[up][:, 4:] == torch.arange(2, device="cuda", dtype=torch.int32)).all()
    assert (ids[~up] == torch.arange(6, device="cuda", dtype=torch.int32)).all()


def test_one_token_alone_and_in_a_window():
    """The rows of a window equal the same tokens run alone, within the sum
    order of the experts; the routing is equal."""
    L = Layer64(1024, 128, 8, 256, 256, seed=5)
    x = tokens(8, 1024, 2)
    y, ids, w, ws = L.run(x)
    for t in range(8):
        y1, i1, w1, _ = L.run(x[t:t + 1].contiguous(), ws)
        assert torch.equal(i1[0], ids[t]) and torch.equal(w1[0], w[t])
        L.check(x[t:t + 1], y1, i1, w1)


def test_calls_repeat_byte_for_byte_and_leave_the_workspace_ready():
    L = Layer64(2048, 64, 10, 512, 512, seed=6)
    x = tokens(8, 2048, 7)
    y, ids, w, ws = L.run(x)
    big = tokens(32, 2048, 8)
    for _ in range(20):
        L.run(big, ws)
        y2, i2, w2, _ = L.run(x, ws)
        assert torch.equal(y, y2) and torch.equal(ids, i2) and torch.equal(w, w2)
    assert moe.moe_workspace_error(ws) == (0, 0)


def test_a_nan_token_keeps_to_itself():
    L = Layer64(512, 32, 4, 128, 128, seed=8)
    x = tokens(6, 512, 9)
    x[2, 100] = float("nan")
    y, ids, w, _ = L.run(x)
    assert y[2].isnan().all()
    keep = [0, 1, 3, 4, 5]
    L.check(x[keep], y[keep], ids[keep], w[keep])


@pytest.mark.parametrize("what", ["codes", "scales"])
@pytest.mark.parametrize("part", ["gu", "dn"])
def test_nan_weights_reach_only_the_tokens_of_their_expert(part, what):
    """NaN or infinity in one expert's weights: the rows of the tokens that did
    not select it keep every bit."""
    L = Layer64(512, 32, 4, 128, 128, seed=12)
    x = tokens(8, 512, 13)
    y, ids, w, ws = L.run(x)
    count = torch.bincount(ids.flatten().long(), minlength=32)
    e = int(((count > 0) & (count < 8)).nonzero()[0])
    if what == "codes":
        getattr(L, part).view(torch.uint8)[e] = 0x7F
    else:
        getattr(L, part + "s")[e] = float("inf")
    y2, i2, w2, _ = L.run(x, ws)
    assert moe.moe_workspace_error(ws) == (0, 0)
    hit = (ids == e).any(1)
    assert torch.equal(ids, i2) and torch.equal(w, w2) and torch.equal(y[~hit], y2[~hit])
    assert not torch.isfinite(y2[hit].float()).any()


def test_large_and_small_values():
    L = Layer64(512, 32, 4, 128, 128, seed=8, router_std=1e-4)
    for scale in (300.0, 1e-3):
        x = tokens(4, 512, 9, scale)
        L.check(x, *L.run(x)[:3])


def test_streams_and_graphs():
    """Two captured graphs on workspaces of their own run at the same time as
    eager calls; each gives the eager result."""
    L = Layer64(1024, 64, 6, 256, 256, seed=10)
    xs = [tokens(T, 1024, T) for T in (1, 5, 12)]
    refs = [L.run(x)[0] for x in xs]
    graphs, outs, streams = [], [], []
    for x in xs:
        ws = moe_ops.alloc_fp8_workspace(L.handle, 32)
        y, s, gr = torch.empty_like(x), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(gr, stream=s):
            moe_ops.moe_fp8_layer_forward(L.handle, x, x.shape[0], y, ws)
        graphs.append((gr, ws))
        outs.append(y)
        streams.append(s)
    torch.cuda.synchronize()
    for _ in range(5):
        for y in outs:
            y.zero_()
        torch.cuda.synchronize()
        for (gr, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for y, r in zip(outs, refs):
            assert torch.equal(y, r)
    for _, ws in graphs:
        assert moe.moe_workspace_error(ws) == (0, 0)


def test_no_tokens():
    L = Layer64(64, 8, 2, 32, 0, seed=1)
    ws = moe_ops.alloc_fp8_workspace(L.handle, 1)
    y = torch.full((1, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    x = torch.zeros_like(y)
    assert moe_ops.load().moe_fp8_layer_forward(L.handle.ref, x.data_ptr(), 0, y.data_ptr(), None,
                                                None, ws.data_ptr(), ws.numel(), None) == 0
    torch.cuda.synchronize()
    assert (y == 7).all()


def test_norm_layer_norm():
    """The run a decoder layer makes: norm, MoE layer, then the norm after it
    with gate and residual and the norm before the next block."""
    d, T = 1024, 6
    L = Layer64(d, 64, 6, 256, 256, seed=12)
    g = gen(13)
    w1, w2 = (1 + 0.1 * torch.randn(d, device="cuda", generator=g) for _ in range(2))
    gate = torch.randn(T, device="cuda", generator=g).to(torch.bfloat16)
    x = tokens(T, d, 14, 2.0)
    n = moe_ops.make_norm(d, w1, w2, True, "token", "sigmoid", branch_scale=0.5)
    h, x2, h2 = (torch.empty_like(x) for _ in range(3))
    moe_ops.moe_norm_block(n, x, None, None, T, None, h)
    y, ids, w, _ = L.run(h)
    moe_ops.moe_norm_block(n, x, y, gate, T, x2, h2)
    _, h64, _, dh = norm64(x, None, None, "none", w1, None, False, False, False, 1.0, 1.0, 1e-6)
    assert ((h.double() - h64).abs() <= BF16 * h64.abs() + dh * 1.01).all()
    L.check(h, y, ids, w)
    r64, h64, dr, dh = norm64(x, y, gate, "token", w1, w2, True, True, False, 1.0, 0.5, 1e-6)
    assert ((x2.double() - r64).abs() <= BF16 * r64.abs() + dr * 1.01).all()
    assert ((h2.double() - h64).abs() <= BF16 * h64.abs() + dh * 1.01).all()


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_clean():
    """The grid's first counter starts so low that the blocks' arrivals do not
    reach the count they wait for: every block's wait ends after the limit, the
    error word says so, and the counters are back where the next call needs them."""
    L = Layer64(256, 32, 4, 64, 64, seed=3)
    x = tokens(4, 256, 1)
    y, ids, w, ws = L.run(x)
    moe.moe_workspace_set_wait_limit(ws, 2000)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws[:256].view(torch.int32)[6] = -sms                  # the control block's first free word
    L.run(x, ws)
    torch.cuda.synchronize()
    assert moe.moe_workspace_error(ws) == (7, 1)          # timeout
    y2, ids2, w2, _ = L.run(x, ws)
    assert torch.equal(y, y2) and torch.equal(ids, ids2) and torch.equal(w, w2)
    assert moe.moe_workspace_error(ws) == (0, 0)


def test_two_threads_call_at_once():
    """Layers of different widths (different shared memory) from two threads."""
    import threading
    Ls = [Layer64(64, 8, 2, 32, 32, seed=1), Layer64(4096, 8, 2, 32, 32, seed=2)]
    xs = [tokens(3, L.d, 5) for L in Ls]
    refs = [L.run(x) for L, x in zip(Ls, xs)]
    torch.cuda.synchronize()
    bad = []

    def work(L, x, ref):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                y, _, _, ws = L.run(x, ref[3])
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, ref[0]):
                    bad.append(L.d)
    ts = [threading.Thread(target=work, args=a) for a in zip(Ls, xs, refs)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_refusals():
    L = Layer64(64, 8, 2, 32, 32, seed=1)
    ws = moe_ops.alloc_fp8_workspace(L.handle, 32)
    x = torch.zeros(33, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(moe.MoEError) as e:
        moe_ops.moe_fp8_layer_forward(L.handle, x, 33, torch.empty_like(x), ws)
    assert e.value.status == 2
    with pytest.raises(moe.MoEError) as e:
        moe_ops.moe_fp8_layer_forward(L.handle, x[:4], 4, x[:4], ws)
    assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe_ops.moe_fp8_layer_forward(L.handle, x[:4], 4, torch.empty_like(x[:4]), ws[:1024])
    assert e.value.status == 3
    with pytest.raises(ValueError):
        moe_ops.moe_fp8_layer_forward(L.handle, x[:4, :32], 4, torch.empty_like(x[:4]), ws)
    for missing in (dict(x=None), dict(y=None), dict(ws=None)):
        a = dict(x=x[:4], y=torch.empty_like(x[:4]), ws=ws)
        a.update(missing)
        with pytest.raises(ValueError):
            moe_ops.moe_fp8_layer_forward(L.handle, a["x"], 4, a["y"], a["ws"])
