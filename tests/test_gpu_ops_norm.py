"""moe_norm_block and moe_fp8_quant against their 64-bit formulas."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops
from _ops_ref import BF16, E4M3, U32, gen, nb, norm64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def inputs(T, d, kind, f32, seed=0):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)   # noqa: E731
    x = (r(T, d) * 3).to(torch.float32 if f32 else torch.bfloat16)
    y = r(T, d).to(torch.bfloat16)
    shape = dict(none=None, token=(T,), channel=(d,), full=(T, d))[kind]
    gate = None if shape is None else r(*shape).to(torch.bfloat16)
    return x, y, gate, 1 + 0.1 * r(d), 1 + 0.1 * r(d)


def check_codes(codes, scales, h, dh, d):
    """Codes and scales of 128-column blocks against h with its error bound dh."""
    T = h.shape[0]
    col = torch.arange(d, device="cuda") // 128
    top = torch.zeros(T, nb(d), dtype=torch.float64, device="cuda")
    top = top.scatter_reduce(1, col.expand(T, -1), h.abs(), "amax")
    dtop = torch.zeros_like(top).scatter_reduce(1, col.expand(T, -1), dh, "amax")
    assert ((scales.double() - top / 448).abs() <= dtop / 448 + 2 * U32 * top / 448).all()
    s = scales.double()[:, col]
    q = codes.view(torch.float8_e4m3fn).double()
    # half a step of the code, and h's own error
    tol = (E4M3 * h.abs()).maximum(2.0 ** -10 * s) + dh * (1 + E4M3) + 4 * U32 * h.abs()
    err = (q * s - h).abs()
    assert (err <= tol).all(), (err / tol.clamp_min(1e-300)).max().item()


def run(T, d, kind="none", f32=False, post=True, sigmoid=False, centred=False, weights=True,
        with_y=True, a=1.0, b=0.7071, eps=1e-6, seed=0, data=None):
    x, y, gate, pre, pw = inputs(T, d, kind, f32, seed) if data is None else data
    if not weights:
        pre = pw = None
    if not with_y:
        y = None
    n = moe_ops.make_norm(d, pre, pw, post, kind, "sigmoid" if sigmoid else "none", centred, f32,
                          a, b, eps)
    x_out, h = torch.full_like(x, float("nan")), torch.full((T, d), float("nan"), device="cuda",
                                                            dtype=torch.bfloat16)
    codes = torch.empty(T, d, device="cuda", dtype=torch.uint8)
    scales = torch.full((T, nb(d)), float("nan"), device="cuda")
    moe_ops.moe_norm_block(n, x, y, gate, T, x_out, h, codes, scales)
    r64, h64, dr, dh = norm64(x, y, gate, kind, pre, pw, post, sigmoid, centred, a, b, eps)
    half = U32 if f32 else BF16
    assert ((x_out.double() - r64).abs() <= half * r64.abs() + dr * (1 + half)).all()
    assert ((h.double() - h64).abs() <= BF16 * h64.abs() + dh * (1 + BF16)).all()
    check_codes(codes, scales, h64, dh, d)
    return x_out, h, codes, scales


@pytest.mark.parametrize("T,d", [(1, 8), (1, 2048), (3, 64), (5, 120), (7, 136), (33, 256),
                                 (4, 264), (9, 520), (2, 1000), (6, 1024), (3, 1032), (257, 2048),
                                 (2, 4104), (5, 8192), (1, 8184), (1030, 384)])
@pytest.mark.parametrize("f32", [False, True])
def test_sizes(T, d, f32):
    run(T, d, "full", f32, sigmoid=True, seed=T + d)


@pytest.mark.parametrize("kind", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("sigmoid,centred,weights", [(False, False, True), (True, True, True),
                                                     (False, True, False)])
def test_forms(kind, post, sigmoid, centred, weights):
    for d in (320, 1096):
        run(11, d, kind, False, post, sigmoid, centred, weights, seed=3)


def test_first_block_has_no_branch():
    run(6, 640, "none", with_y=False, a=1.0)
    run(6, 2048, "token", with_y=False, a=0.5)     # the gate belongs to the branch


def test_outputs_are_optional_and_agree():
    T, d = 19, 1160
    x, y, gate, pre, pw = inputs(T, d, "channel", False, 5)
    n = moe_ops.make_norm(d, pre, pw, True, "channel")
    new = lambda: (torch.empty_like(x), torch.empty_like(x),   # noqa: E731
                   torch.empty(T, d, device="cuda", dtype=torch.uint8),
                   torch.empty(T, nb(d), device="cuda"))
    full = new()
    moe_ops.moe_norm_block(n, x, y, gate, T, *full)
    for keep in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)):
        o = new()
        moe_ops.moe_norm_block(n, x, y, gate, T, o[0] if keep[0] else None, o[1] if keep[1] else None,
                               *(o[2:] if keep[2] else (None, None)))
        for i, on in ((0, keep[0]), (1, keep[1]), (2, keep[2]), (3, keep[2])):
            if on:
                assert torch.equal(o[i], full[i])


@pytest.mark.parametrize("d", [512, 2048])
@pytest.mark.parametrize("f32", [False, True])
def test_pitched_rows_and_in_place(d, f32):
    T = 13
    x, y, gate, pre, pw = inputs(T, d, "full", f32, 9)
    ref = run(T, d, "full", f32, data=(x, y, gate, pre, pw))
    n = moe_ops.make_norm(d, pre, pw, True, "full", stream_f32=f32, branch_scale=0.7071)

    def wide(t, pad):
        w = torch.full((T, d + pad), 7.0, device="cuda", dtype=t.dtype)
        w[:, :d] = t
        return w
    xw, yw, gw = wide(x, 8), wide(y, 16), wide(gate, 24)
    moe_ops.moe_norm_block(n, xw[:, :d], yw[:, :d], gw[:, :d], T, xw[:, :d], yw[:, :d])
    assert torch.equal(xw[:, :d], ref[0]) and torch.equal(yw[:, :d], ref[1])
    assert (xw[:, d:] == 7).all() and (yw[:, d:] == 7).all()      # the columns between rows


def test_rows_of_zeros_and_of_special_values():
    T, d = 6, 384
    x, y, gate, pre, pw = inputs(T, d, "none", False, 2)
    x[0], y[0] = 0, 0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    y[3, 300] = float("nan")
    x[4] = x[4].abs().clamp_max(1e-30) * 1e-8          # subnormal squares
    y[4] = 0
    n = moe_ops.make_norm(d, pre, pw, True)
    x_out, h = torch.empty_like(x), torch.empty_like(x)
    codes = torch.empty(T, d, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty(T, 3, device="cuda")
    moe_ops.moe_norm_block(n, x, y, None, T, x_out, h, codes, scales)
    assert (x_out[0] == 0).all() and (h[0] == 0).all()
    assert (codes[0].float() == 0).all() and (scales[0] == 0).all()
    assert x_out[1].isnan().sum() == 1 and h[1].isnan().all() and scales[1].isnan().all()
    assert x_out[2].isinf().sum() == 1 and h[2].isnan().sum() == 1
    assert x_out[3].isnan().all() and h[3].isnan().all()
    for t in (0, 4, 5):
        assert torch.isfinite(h[t].float()).all() and torch.isfinite(scales[t]).all()
    r64, h64, _, dh = norm64(x[5:], y[5:], None, "none", pre, pw, True, False, False, 1.0, 1.0, 1e-6)
    assert ((h[5:].double() - h64).abs() <= BF16 * h64.abs() + dh * 1.01).all()


def test_no_rows():
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    n = moe_ops.make_norm(64)
    moe_ops.moe_norm_block(n, x, None, None, 0, x_out=torch.empty_like(x))
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,d", [(1, 8), (1, 128), (7, 136), (300, 2048), (3, 16384), (2, 65528)])
def test_quant(T, d):
    x = (torch.randn(T, d, device="cuda", generator=gen(d)) * 5).to(torch.bfloat16)
    x[0, : min(d, 128)] = 0
    codes = torch.empty(T, d, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.full((T, nb(d)), float("nan"), device="cuda")
    moe_ops.moe_fp8_quant(x, codes, scales)
    check_codes(codes, scales, x.double(), torch.zeros(T, d, dtype=torch.float64, device="cuda"), d)
    # rows with a pitch give the same
    if T > 1:
        w = torch.zeros(T, d + 8, device="cuda", dtype=torch.bfloat16)
        w[:, :d] = x
        c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
        moe_ops.moe_fp8_quant(w[:, :d], c2, s2)
        assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scales)


def test_stream_and_graph():
    T, d = 40, 2048
    x, y, gate, pre, pw = inputs(T, d, "token", False, 1)
    ref = run(T, d, "token", sigmoid=True, data=(x, y, gate, pre, pw))
    n = moe_ops.make_norm(d, pre, pw, True, "token", "sigmoid", branch_scale=0.7071)
    s = torch.cuda.Stream()
    xs, o, h = torch.zeros_like(x), torch.empty_like(x), torch.empty_like(x)
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            moe_ops.moe_norm_block(n, xs, y, gate, T, o, h)
            moe_ops.moe_norm_block(n, o, None, None, T, None, h)    # depends on the first
        xs.copy_(x)
        graph.replay()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, ref[0])
    _, h64, _, dh = norm64(ref[0], None, None, "none", pre, pw, False, False, False, 1.0, 1.0, 1e-6)
    assert ((h.double() - h64).abs() <= BF16 * h64.abs() + dh * 1.01).all()


def test_refusals():
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    n = moe_ops.make_norm(64)
    with pytest.raises(ValueError):
        moe_ops.moe_norm_block(n, x.float(), None, None, 4, x_out=x)
    with pytest.raises(ValueError):
        moe_ops.moe_norm_block(n, x.cpu(), None, None, 4, x_out=x)
    with pytest.raises(ValueError):
        moe_ops.moe_norm_block(n, x, x[:, :32], None, 4, x_out=x)
    with pytest.raises(moe.MoEError):
        moe_ops.moe_norm_block(n, x, None, None, 4)
