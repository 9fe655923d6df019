"""Codes and scales of moe_fp8_quant and moe_norm_block bit for bit as the header
defines them: in fp32, scale = max|h| / 448 and code = e4m3(h / scale)."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe_ops
from _ops_ref import gen, nb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def defined(h):
    """(codes, scales) of fp32 rows.  A quotient of two fp32 numbers rounded to 64
    bits and then to fp32 is the one rounded once (53 >= 2 * 24 + 2 bits)."""
    T, d = h.shape
    p = torch.zeros(T, nb(d) * 128, device="cuda")
    p[:, :d] = h
    p = p.view(T, -1, 128)
    top = p.abs().amax(2)
    s = (top.double() / 448).float()
    q = (p.double() / s[:, :, None].double()).float()
    q = torch.where(s[:, :, None] == 0, p, q).clamp(-448, 448)      # clamp keeps NaN
    return q.to(torch.float8_e4m3fn).view(T, -1)[:, :d].contiguous(), s


def same(codes, scales, h):
    c, s = defined(h)
    assert torch.equal(scales.nan_to_num(-1, -2), s.nan_to_num(-1, -2))
    a, b = codes.view(torch.float8_e4m3fn).float(), c.float()
    bad = (a != b) & ~(a.isnan() & b.isnan())
    assert not bad.any(), (int(bad.sum()), h[bad][:4], a[bad][:4], b[bad][:4])


def quant(x):
    T, d = x.shape
    codes = torch.empty(T, d, device="cuda", dtype=torch.uint8)
    scales = torch.full((T, nb(d)), float("nan"), device="cuda")
    moe_ops.moe_fp8_quant(x, codes, scales)
    return codes, scales


@pytest.mark.parametrize("T,d", [(2000, 2048), (333, 1000), (7, 136), (1, 8)])
def test_random_rows(T, d):
    x = (torch.randn(T, d, device="cuda", generator=gen(d)) * 5).to(torch.bfloat16)
    same(*quant(x), x.float())


def test_every_value_under_every_largest():
    """Row t: a largest value with the t-th of the 128 bf16 mantissas, and below it
    the bf16 numbers of 9 binades, over as many blocks as they need: every tie
    between two codes is among them."""
    m = 1 + torch.arange(128, device="cuda") / 128
    vals = torch.cat([m * 2.0 ** -e for e in range(1, 19)])          # all below 1
    vals = torch.cat([vals, -vals])
    n = -(-vals.numel() // 127)
    vals = torch.nn.functional.pad(vals, (0, n * 127 - vals.numel())).view(n, 127)
    for scale in (1.0, 2.0 ** 40, 2.0 ** -60):
        x = torch.empty(128, n, 128, device="cuda")
        x[:, :, 0] = m[:, None]
        x[:, :, 1:] = vals
        x = (x.view(128, -1) * scale).to(torch.bfloat16)
        same(*quant(x), x.float())


def test_small_and_special_blocks():
    x = torch.randn(64, 1024, device="cuda", generator=gen(3))
    x = x * 2.0 ** -torch.arange(64, 128, device="cuda").view(64, 1)     # down to subnormals
    x[:, :128] = 0
    x = x.to(torch.bfloat16)
    x[3, 300] = float("inf")
    x[5, 400] = float("-inf")
    x[7, 500] = float("nan")
    same(*quant(x), x.float())


def test_large_blocks():
    x = torch.randn(40, 1024, device="cuda", generator=gen(4)).clamp(-1.9, 1.9)
    x = x * 2.0 ** torch.arange(88, 128, device="cuda").view(40, 1)      # up to the largest binade
    x = x.to(torch.bfloat16)
    assert torch.isfinite(x.float()).all()
    same(*quant(x), x.float())


@pytest.mark.parametrize("d", [256, 2048])
def test_codes_of_the_norm(d):
    """Rows of +-1 have a mean square of exactly 1, so that with eps = 3, and the
    branch scaled, h is 1/2 times the weights, exact powers of two times them: the
    codes are those of the weights."""
    T = 40
    g = gen(d)
    x = (torch.randint(0, 2, (T, d), device="cuda", generator=g) * 2 - 1).to(torch.bfloat16)
    w = torch.randn(d, device="cuda", generator=g) * 3
    codes = torch.empty(T, d, device="cuda", dtype=torch.uint8)
    scales = torch.empty(T, nb(d), device="cuda")
    moe_ops.moe_norm_block(moe_ops.make_norm(d, w, eps=3.0), x, None, None, T, codes=codes,
                           scales=scales)
    same(codes, scales, x.float() * 0.5 * w)
