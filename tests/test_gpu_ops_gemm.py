"""moe_fp8_gemm and moe_fp8_gemm_grouped against 64-bit products."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops
from _ops_ref import BF16, gen, nb, product64, quant_rows, rand_weights

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


def dense(M, N, K, seed=0):
    a, sa = acts(M, K, seed)
    w, sw = rand_weights((N, K), seed + 1)
    c = torch.full((M, N), float("nan"), device="cuda", dtype=torch.bfloat16)
    moe_ops.moe_fp8_gemm(moe_ops.make_fp8_mat(w, sw), a, sa, M, c)
    compare(c, *product64(a, sa, w, sw))
    return a, sa, w, sw, c


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 16, 128), (1, 17, 144), (2, 64, 2048), (4, 4096, 2048), (127, 128, 256),
    (128, 129, 128), (129, 255, 272), (333, 1000, 1936), (300, 2047, 640), (1000, 257, 1040),
    (4096, 136, 512), (2500, 4096, 1024), (40, 40, 4096), (16, 300, 16384)])
def test_dense(M, N, K):
    dense(M, N, K, seed=M + N + K)


def test_each_tile_width_is_reached():
    """One row of tiles, from a few hundred columns to more than the widest tile
    times the SMs of a B200: the launcher's cost estimate goes from the
    narrowest tile to the widest."""
    for N in (512, 148 * 32, 148 * 64, 148 * 128, 148 * 256):
        dense(100, N + 3, 272, seed=N)


def test_wide_rows_pass_32_bit_offsets():
    """Outputs beyond 2^31 elements land where they belong: the last rows of a
    product with M * N > 2^31 equal the same rows on their own."""
    M, N, K = 33000, 65536, 16
    a, sa = acts(M, K, 5)
    w, sw = rand_weights((N, K), 6)
    m = moe_ops.make_fp8_mat(w, sw)
    c = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    moe_ops.moe_fp8_gemm(m, a, sa, M, c)
    tail = torch.empty(40, N, device="cuda", dtype=torch.bfloat16)
    moe_ops.moe_fp8_gemm(m, a[-40:].contiguous(), sa[-40:].contiguous(), 40, tail)
    assert torch.equal(c[-40:], tail)
    compare(tail, *product64(a[-40:], sa[-40:], w, sw))


def grouped(counts, N, K, lead=0, tail=0, seed=0):
    G = len(counts)
    off = torch.tensor([lead] + [lead + sum(counts[: g + 1]) for g in range(G)], dtype=torch.int32,
                       device="cuda")
    M = lead + sum(counts) + tail
    a, sa = acts(M, K, seed)
    w, sw = rand_weights((G, N, K), seed + 1)
    c = torch.full((M, N), 7.0, device="cuda", dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe_ops.moe_fp8_gemm_grouped(moe_ops.make_fp8_mat(w, sw), a, sa, M, off, c, ws=ws)
    assert moe.moe_workspace_error(ws) == (0, 0)
    o = off.tolist()
    for g in range(G):
        if o[g + 1] > o[g]:
            r = slice(o[g], o[g + 1])
            compare(c[r], *product64(a[r], sa[r], w[g], sw[g]))
    assert (c[: o[0]] == 7).all() and (c[o[G]:] == 7).all()     # rows of no group
    return c


@pytest.mark.parametrize("counts,N,K,lead,tail", [
    ([5], 64, 128, 0, 0),
    ([0, 3, 0, 0, 130, 1, 0], 200, 144, 0, 0),
    ([0, 0, 0], 64, 64, 4, 9),
    ([128, 256, 1, 127], 272, 512, 3, 60),
    ([1] * 300 + [0] * 212, 256, 256, 0, 0),
    ([700, 0, 1, 300], 1000, 1040, 0, 5),
    ([17] * 64, 1024, 2048, 0, 0)])
def test_grouped(counts, N, K, lead, tail):
    grouped(counts, N, K, lead, tail, seed=len(counts))


def test_grouped_of_the_most_groups():
    grouped([1 if g % 3 == 0 else 0 for g in range(1024)], 72, 64)


def test_grouped_of_one_group_is_the_dense_product():
    a, sa, w, sw, c = dense(200, 328, 400)
    c2 = torch.empty_like(c)
    off = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    moe_ops.moe_fp8_gemm_grouped(moe_ops.make_fp8_mat(w, sw), a, sa, 200, off, c2)
    assert torch.equal(c, c2)


def test_bad_offsets_stay_inside_and_are_reported():
    """Offsets are clamped to 0..M and to non-decreasing order on the device
    before any address is formed from them."""
    M, N, K = 50, 64, 128
    a, sa = acts(M, K, 1)
    w, sw = rand_weights((3, N, K), 2)
    buf = torch.full((M + 64, N), 7.0, device="cuda", dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    m = moe_ops.make_fp8_mat(w, sw)
    for off in ([-5, 10, 20, 90], [0, 40, 20, 50]):
        buf.fill_(7.0)
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        moe_ops.moe_fp8_gemm_grouped(m, a, sa, M, o, buf[:M], ws=ws)
        st, code = moe.moe_workspace_error(ws)
        assert st == 6 and code == 2                     # device check, range
        assert (buf[M:] == 7).all()
    c = buf[:M]
    compare(c[:40], *product64(a[:40], sa[:40], w[0], sw[0]))     # 0, 40, 40, 50
    compare(c[40:], *product64(a[40:], sa[40:], w[2], sw[2]))


def test_rows_with_nan_keep_to_themselves():
    M, N, K = 70, 96, 272
    a, sa = acts(M, K, 1)
    w, sw = rand_weights((N, K), 2)
    ref, bound = product64(a, sa, w, sw)
    a, sa = a.clone(), sa.clone()
    a.view(torch.uint8)[3, 200] = 0x7F
    sa[9, 1] = float("inf")
    c = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    moe_ops.moe_fp8_gemm(moe_ops.make_fp8_mat(w, sw), a, sa, M, c)
    assert c[3].isnan().all() and not torch.isfinite(c[9].float()).any()
    keep = [m for m in range(M) if m not in (3, 9)]
    compare(c[keep], ref[keep], bound[keep])


def test_unaligned_output():
    M, N, K = 37, 64, 256
    a, sa = acts(M, K, 1)
    w, sw = rand_weights((N, K), 2)
    buf = torch.full((M * N + 8,), 7.0, device="cuda", dtype=torch.bfloat16)
    c = buf[1: 1 + M * N].view(M, N)
    moe_ops.moe_fp8_gemm(moe_ops.make_fp8_mat(w, sw), a, sa, M, c)
    compare(c, *product64(a, sa, w, sw))
    assert buf[0] == 7 and (buf[1 + M * N:] == 7).all()


def test_repeats_streams_and_graphs_agree():
    a, sa, w, sw, c = dense(513, 640, 1040)
    m = moe_ops.make_fp8_mat(w, sw)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    out = torch.empty_like(c)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            moe_ops.moe_fp8_gemm(m, a, sa, 513, out)
        for _ in range(3):
            out.fill_(0)
            graph.replay()
            s.synchronize()
            assert torch.equal(out, c)
    # two products at once on two streams
    outs = [torch.empty_like(c) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st, o in zip(streams, outs):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(8):
                moe_ops.moe_fp8_gemm(m, a, sa, 513, o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], c) and torch.equal(outs[1], c)


def test_no_rows():
    w, sw = rand_weights((16, 32), 1)
    m = moe_ops.make_fp8_mat(w, sw)
    c = torch.full((1, 16), 7.0, device="cuda", dtype=torch.bfloat16)
    moe_ops.moe_fp8_gemm(m, w[:0], sw[:0], 0, c[:0])
    assert moe_ops.load().moe_fp8_gemm(m.ref, w.data_ptr(), sw.data_ptr(), 0, c.data_ptr(), None,
                                       None) == 0
    torch.cuda.synchronize()
    assert (c == 7).all()


def test_norm_feeds_the_product():
    """The codes of the fused norm go straight into the product: the same
    output as from a separate quantiser on codes equal to them, and within the
    codes' own rounding of the product of the unquantised rows."""
    T, d, N = 50, 2048, 512
    x = torch.randn(T, d, device="cuda", generator=gen(3)).to(torch.bfloat16)
    n = moe_ops.make_norm(d)
    h = torch.empty_like(x)
    codes = torch.empty(T, d, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty(T, nb(d), device="cuda")
    moe_ops.moe_norm_block(n, x, None, None, T, None, h, codes, scales)
    w, sw = rand_weights((N, d), 4)
    c = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    moe_ops.moe_fp8_gemm(moe_ops.make_fp8_mat(w, sw), codes, scales, T, c)
    compare(c, *product64(codes, scales, w, sw))


def test_refusals():
    w, sw = rand_weights((64, 128), 1)
    m = moe_ops.make_fp8_mat(w, sw)
    a, sa = acts(4, 128, 2)
    c = torch.empty(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe_ops.moe_fp8_gemm(m, a[:, :64], sa, 4, c)
    with pytest.raises(ValueError):
        moe_ops.moe_fp8_gemm(m, a, sa[:2], 4, c)
    with pytest.raises(ValueError):
        moe_ops.moe_fp8_gemm(m, a, sa, 4, c.float())
    with pytest.raises(ValueError):
        moe_ops.moe_fp8_gemm(m, a.cpu(), sa, 4, c)
    with pytest.raises(ValueError):
        moe_ops.make_fp8_mat(w, sw[:0])
