"""Operators on tensors whose offsets pass 32 bits: the far rows, experts or groups
come out bit for bit as from a call that holds them alone."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops
from _ops_ref import Layer64, gen, nb

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    torch.cuda.empty_cache()


def rows(T, d, seed):
    x = torch.empty(T, d, device="cuda", dtype=torch.bfloat16)
    return x.normal_(generator=gen(seed))


def test_norm_rows():
    T, d, n = 270_000, 8192, 40                  # 2.2e9 elements
    x, y = rows(T, d, 1), rows(T, d, 2)
    pre = torch.randn(d, device="cuda", generator=gen(3))
    norm = moe_ops.make_norm(d, pre, pre, True, "full", "sigmoid")

    def run(x, y):
        T = x.shape[0]
        o, h = torch.empty_like(x), torch.empty_like(x)
        c = torch.empty(T, d, device="cuda", dtype=torch.uint8)
        s = torch.empty(T, nb(d), device="cuda")
        moe_ops.moe_norm_block(norm, x, y, y, T, o, h, c, s)
        return [t[-n:].clone() for t in (o, h, c, s)]
    for a, b in zip(run(x, y), run(x[-n:].clone(), y[-n:].clone())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 1024])
def test_pitches(d):
    """Three rows 2^30 + 8 elements apart, in and out."""
    buf = torch.zeros(3, (1 << 30) + 8, device="cuda", dtype=torch.bfloat16)
    x = rows(3, d, 4)
    far = buf[:, 4096:4096 + d]
    far.copy_(x)
    pre = torch.randn(d, device="cuda", generator=gen(3))
    norm = moe_ops.make_norm(d, pre)
    h = torch.empty_like(x)
    moe_ops.moe_norm_block(norm, x, None, None, 3, None, h)
    out = buf[:, 16384:16384 + d]
    moe_ops.moe_norm_block(norm, far, None, None, 3, None, out)
    assert torch.equal(out, h)
    c, s = (torch.empty(3, d, device="cuda", dtype=torch.uint8), torch.empty(3, nb(d), device="cuda"))
    c2, s2 = torch.empty_like(c), torch.empty_like(s)
    moe_ops.moe_fp8_quant(x, c, s)
    moe_ops.moe_fp8_quant(far, c2, s2)
    assert torch.equal(c, c2) and torch.equal(s, s2)


def test_quant_rows():
    T, d, n = 33_000, 65_536, 10                 # 2.2e9 elements
    x = rows(T, d, 5)
    c, s = torch.empty(T, d, device="cuda", dtype=torch.uint8), torch.empty(T, nb(d), device="cuda")
    moe_ops.moe_fp8_quant(x, c, s)
    c2, s2 = torch.empty_like(c[-n:]), torch.empty_like(s[-n:])
    moe_ops.moe_fp8_quant(x[-n:].clone(), c2, s2)
    assert torch.equal(c[-n:], c2) and torch.equal(s[-n:], s2)


def codes(shape, seed):
    """Random finite codes (uint8 below 0x7F, with signs)."""
    q = torch.randint(0, 0x7F, shape, device="cuda", dtype=torch.uint8, generator=gen(seed))
    return q.bitwise_or_(torch.randint(0, 2, shape, device="cuda", dtype=torch.uint8,
                                       generator=gen(seed + 1)).mul_(128)).view(FP8)


@pytest.mark.parametrize("M,N", [(24, 2048), (600, 2048), (4000, 2040)])
def test_groups(M, N):
    G, K, far = 1024, 2048, 4                    # 4.3e9 bytes of weights, the last groups used
    w = codes((G, N, K), 6)
    sw = torch.rand(G, nb(N), nb(K), device="cuda", generator=gen(7))
    a, sa = codes((M, K), 8), torch.rand(M, nb(K), device="cuda", generator=gen(9))
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    cut = torch.tensor([0, M // 5, M // 2, M - 1, M], dtype=torch.int32, device="cuda")
    off[-far - 1:] = cut
    c = torch.full((M, N), 7.0, device="cuda", dtype=torch.bfloat16)
    moe_ops.moe_fp8_gemm_grouped(moe_ops.make_fp8_mat(w, sw), a, sa, M, off, c)
    m = moe_ops.make_fp8_mat(w[-far:].contiguous(), sw[-far:].contiguous())
    c2 = torch.full_like(c, 8.0)
    moe_ops.moe_fp8_gemm_grouped(m, a, sa, M, cut, c2)
    assert torch.equal(c, c2) and torch.isfinite(c.float()).all()


def test_product_operands():
    """More than 2^31 codes of a, the last rows compared."""
    M, N, K = 140_000, 40, 16_384
    a, sa = codes((M, K), 10), torch.rand(M, nb(K), device="cuda", generator=gen(11))
    m = moe_ops.make_fp8_mat(codes((N, K), 12), torch.rand(nb(N), nb(K), device="cuda", generator=gen(13)))
    c = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    moe_ops.moe_fp8_gemm(m, a, sa, M, c)
    c2 = torch.empty(50, N, device="cuda", dtype=torch.bfloat16)
    moe_ops.moe_fp8_gemm(m, a[-50:].contiguous(), sa[-50:].contiguous(), 50, c2)
    assert torch.equal(c[-50:], c2)


@pytest.mark.parametrize("T", [1, 8])
def test_experts(T):
    """5.0e9 bytes of gate/up and 2.5e9 of down weights; the router takes the last
    four experts.  A layer of these four alone has the same logits, the same list and
    so the same sums."""
    d, F, E, k = 4096, 2048, 300, 4
    gu, dn = codes((E, 2, F, d), 14), codes((E, d, F), 16)
    one = lambda *s: torch.rand(s, device="cuda", generator=gen(18)) * 2.0 ** -9   # noqa: E731
    gus, dns = one(E, 2, nb(F), nb(d)), one(E, nb(d), nb(F))
    wr = torch.randn(E, d, device="cuda", generator=gen(19)) * 0.02
    bias = torch.zeros(E, device="cuda")
    bias[-k:] = 100.0
    x = rows(T, d, 20) * 2.0 ** -6

    def run(lo):
        parts = [t[lo:].contiguous() for t in (wr, bias, gu, gus, dn, dns)]
        L = moe_ops.make_fp8_layer(k, *parts)
        ws = moe_ops.alloc_fp8_workspace(L, T)
        y = torch.full_like(x, float("nan"))
        ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
        w = torch.empty(T, k, device="cuda")
        moe_ops.moe_fp8_layer_forward(L, x, T, y, ws, ids, w)
        assert moe.moe_workspace_error(ws) == (0, 0)
        return y, ids + lo, w
    for a, b in zip(run(0), run(E - k)):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()


MOST = 2**31 - 256        # rows of one call


def test_most_rows_of_norm_and_quantiser():
    """8 channels and the most rows: the first, middle and last ones as alone."""
    d = 8
    x = torch.empty(MOST, d, device="cuda", dtype=torch.bfloat16)
    x.view(-1, 256 * d)[:] = rows(256, d, 21).flatten()
    x[-1024:] = rows(1024, d, 22)
    h = torch.empty_like(x)
    c = torch.empty(MOST, d, device="cuda", dtype=torch.uint8)
    s = torch.empty(MOST, 1, device="cuda")
    norm = moe_ops.make_norm(d)
    moe_ops.moe_norm_block(norm, x, None, None, MOST, None, h, c, s)
    cuts = [slice(0, 512), slice(MOST // 2 - 256, MOST // 2 + 256), slice(MOST - 1024, MOST)]
    for cut in cuts:
        xs = x[cut].clone()
        hs, cs, ss = torch.empty_like(xs), torch.empty_like(c[cut]), torch.empty_like(s[cut])
        moe_ops.moe_norm_block(norm, xs, None, None, len(xs), None, hs, cs, ss)
        assert torch.equal(h[cut], hs) and torch.equal(c[cut], cs) and torch.equal(s[cut], ss)
    c.zero_(), s.zero_()
    moe_ops.moe_fp8_quant(x, c, s)
    for cut in cuts:
        xs = x[cut].clone()
        cs, ss = torch.empty_like(c[cut]), torch.empty_like(s[cut])
        moe_ops.moe_fp8_quant(xs, cs, ss)
        assert torch.equal(c[cut], cs) and torch.equal(s[cut], ss)


@pytest.mark.parametrize("groups", [1, 3])
def test_most_rows_of_a_product(groups):
    K, N = 16, 8
    a = torch.empty(MOST, K, device="cuda", dtype=torch.uint8)
    a.view(-1, 256 * K)[:] = codes((256, K), 23).view(torch.uint8).flatten()
    a[-1024:] = codes((1024, K), 24).view(torch.uint8)
    sa = torch.full((MOST, 1), 0.5, device="cuda")
    sa[-1024:] = torch.rand(1024, 1, device="cuda", generator=gen(25))
    w = codes((groups, N, K), 26)
    sw = torch.rand(groups, 1, 1, device="cuda", generator=gen(27))
    c = torch.full((MOST, N), 7.0, device="cuda", dtype=torch.bfloat16)
    ends = [0, MOST] if groups == 1 else [5, 1000, MOST - 700, MOST - 3]
    if groups == 1:
        moe_ops.moe_fp8_gemm(moe_ops.make_fp8_mat(w[0], sw[0]), a, sa, MOST, c)
    else:
        off = torch.tensor(ends, dtype=torch.int32, device="cuda")
        moe_ops.moe_fp8_gemm_grouped(moe_ops.make_fp8_mat(w, sw), a, sa, MOST, off, c)
    for g in range(groups):
        lo, hi = ends[g], ends[g + 1]
        for cut in (slice(lo, min(lo + 400, hi)), slice(max(lo, hi - 400), hi)):
            o = torch.empty(cut.stop - cut.start, N, device="cuda", dtype=torch.bfloat16)
            moe_ops.moe_fp8_gemm(moe_ops.make_fp8_mat(w[g], sw[g]), a[cut].contiguous(),
                                 sa[cut].contiguous(), len(o), o)
            assert torch.equal(c[cut], o)
    assert (c[:ends[0]] == 7).all() and (c[ends[-1]:] == 7).all()


def test_widest_layer():
    """The largest channels, experts' and shared widths, top-k and window at once."""
    torch.cuda.empty_cache()
    L = Layer64(4096, 64, 16, 4096, 4096, seed=31)
    L.bias[:] = torch.where(torch.arange(64, device="cuda") % 3 == 0, 30.0, 0.0)
    x = rows(32, 4096, 32)
    y, ids, w, ws = L.run(x)
    assert moe.moe_workspace_error(ws) == (0, 0)
    L.check(x, y, ids, w)
