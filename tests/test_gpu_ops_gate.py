"""The gate's sigmoid over every bf16 number."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe_ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("kind", ["token", "channel", "full"])
def test_every_gate(kind):
    """x = 0, y = 1 and an fp32 stream: x_out is the sigmoid.  The exponential is
    off by at most 2 + 1.173 |g| last bits (2^-23) and the division by 2 (their
    documented bounds), the sum below it by half of one: with the exponential's share
    e / (1 + e) below 1 for g < 0 and s (1 - s)(2 + 1.173 |g|) below 0.7, the header's
    (5 + 1.2 |g|) 2^-23 of the value and 2^-21 in all."""
    g = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    T, d = {"token": (65536, 8), "channel": (1, 8192), "full": (64, 1024)}[kind]
    parts = g.view(8, 8192) if kind == "channel" else [g if kind == "token" else g.view(T, d)]
    n = moe_ops.make_norm(d, gate=kind, gate_act="sigmoid", stream_f32=True)
    x = torch.zeros(T, d, device="cuda")
    y = torch.ones(T, d, device="cuda", dtype=torch.bfloat16)
    got = []
    for p in parts:
        o = torch.full_like(x, 7.0)
        moe_ops.moe_norm_block(n, x, y, p, T, o)
        if kind == "token":
            assert torch.equal(o.nan_to_num(9), o[:, :1].expand(T, d).nan_to_num(9))
            o = o[:, 0]
        got.append(o.flatten())
    s, g64 = torch.cat(got).double(), g.double()
    assert torch.equal(s.isnan(), g64.isnan())
    ok = ~g64.isnan()
    s, g64 = s[ok], g64[ok]
    ref = torch.sigmoid(g64)
    err = (s - ref).abs()
    assert (err <= 2.0 ** -21).all() and (s >= 0).all() and (s <= 1).all()
    near = g64.abs() <= 87
    bound = (5 + 1.2 * g64.abs()) * 2.0 ** -23 * ref
    assert (err <= bound)[near].all(), (err / bound)[near].max()
    assert (s[g64 == float("-inf")] == 0).all() and (s[g64 == float("inf")] == 1).all()
