"""moe_fp8_layer_forward where arithmetic gives the outputs exactly."""
import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe_ops.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("T", [1, 4, 8, 20])
@pytest.mark.parametrize("F,Fs", [(32, 0), (32, 32), (160, 288)])
def test_hidden_values_keep_their_low_bits(T, F, Fs):
    """Hidden values of 16 significant bits whose high bits cancel in the down
    product.  One expert of weight 1 (softmax over one logit).  Channel f of a
    token with gate input g = 2^n >= 32 has gate g, where e^-g is below half a
    step of 1 and silu(g) = g, and up = 4096 * 15 + b_f with b_f = f % 16: the two
    summands lie in blocks of columns of their own and are joined in fp32.  A row
    of the down product subtracts channel j from channel i: g (b_i - b_j), exact in
    bf16, while a hidden value rounded to fp16 would lose b altogether (its step
    there is 32 g).  A shared expert of the same form adds the same again."""
    d, dev = 256, "cuda"
    fp8 = torch.float8_e4m3fn

    def expert(F):
        gu = torch.zeros(2, F, d, device=dev)
        f = torch.arange(F, device=dev)
        b = (f % 16).float()
        gu[0, :, 0] = 1.0
        gu[1, :, 1] = 15.0
        gu[1, :, 128] = b
        dn, r = torch.zeros(d, F, device=dev), torch.arange(d, device=dev)
        i, j = (r * 7) % F, (r * 3 + 5) % F
        dn[r, i] += 1.0
        dn[r, j] -= 1.0
        kf = -(-F // 128)
        return (gu.to(fp8), torch.ones(2, kf, 2, device=dev), dn.to(fp8),
                torch.ones(2, kf, device=dev), b[i] - b[j])

    gu, gus, dn, dns, diff = expert(F)
    shared, total = (None,) * 4, diff
    if Fs:
        *shared, more = expert(Fs)
        total = total + more
    layer = moe_ops.make_fp8_layer(1, torch.zeros(1, d, device=dev), None, gu[None].contiguous(),
                                   gus[None].contiguous(), dn[None].contiguous(),
                                   dns[None].contiguous(), *shared)
    g = 2.0 ** (5 + torch.arange(T, device=dev) % 3)
    x = torch.zeros(T, d, device=dev, dtype=torch.bfloat16)
    x[:, 0], x[:, 1], x[:, 128] = g.bfloat16(), 4096.0, 1.0
    y = torch.full_like(x, float("nan"))
    ws = moe_ops.alloc_fp8_workspace(layer, T)
    moe_ops.moe_fp8_layer_forward(layer, x, T, y, ws)
    assert moe.moe_workspace_error(ws) == (0, 0)
    assert torch.equal(y.float(), g[:, None] * total)
