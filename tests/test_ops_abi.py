"""Host-side validation of the operators of include/moe_ops.h: every refusal is
decided before a GPU is touched."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from routed_expert_ffn_06_b200 import build, moe, moe_ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x7F0000000000          # 256-aligned made-up device addresses, never read on the host
OK = 0 if torch.cuda.is_available() else 8      # a valid call stops at the missing device

X, Y, G, XO, H, C, S, WS = (P + i * 0x100000 for i in range(1, 9))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe_ops.load()


def ref(s):
    return ctypes.addressof(s)


# a valid call would enqueue work on the made-up addresses where a GPU is
# present: only T = 0 or M = 0 is passed as valid
def norm(**kw):
    n = dict(d=256, flags=0, gate_kind=0, eps=1e-6, stream_scale=1.0, branch_scale=1.0)
    n.update(kw)
    return moe_ops.moe_norm(**n)


def call_norm(lib, n, x=X, y=Y, gate=None, T=0, xo=XO, h=H, c=None, s=None):
    return lib.moe_norm_block(ref(n), x, y, gate, T, xo, h, c, s, None)


def test_exports(lib):
    for n in moe_ops.EXPORTS:
        assert hasattr(lib, n)


@pytest.mark.parametrize("kw,status", [
    (dict(d=4), 2), (dict(d=12), 2), (dict(d=8200), 2), (dict(d=0), 2), (dict(flags=16), 1),
    (dict(gate_kind=4), 1), (dict(gate_kind=-1), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(stream_scale=float("inf")), 1),
    (dict(branch_scale=float("nan")), 1), (dict(x_ld=128), 1), (dict(h_ld=260), 1),
    (dict(y_ld=-256), 1), (dict(pre_w=P + 4), 4), (dict(post_w=P + 8), 4)])
def test_norm_struct(lib, kw, status):
    assert call_norm(lib, norm(**kw)) == status


def test_norm_arguments(lib):
    n = norm()
    assert call_norm(lib, n) == OK
    assert call_norm(lib, n, x=None) == 1
    assert lib.moe_norm_block(None, X, Y, None, 0, XO, H, None, None, None) == 1
    assert call_norm(lib, n, T=-1) == 1 and call_norm(lib, n, T=2**31 - 1) == 2
    assert call_norm(lib, n, xo=None, h=None) == 1                # no output
    assert call_norm(lib, n, c=C) == 1 and call_norm(lib, n, s=S) == 1
    assert call_norm(lib, n, c=C, s=S) == OK
    assert call_norm(lib, n, c=C + 4, s=S) == 4
    assert call_norm(lib, n, x=X + 8) == 4 and call_norm(lib, n, y=Y + 2) == 4
    assert call_norm(lib, n, xo=XO + 8) == 4 and call_norm(lib, n, h=H + 8) == 4
    g = norm(gate_kind=moe_ops.GATES["channel"])
    assert call_norm(lib, g) == 1                                 # gate missing
    assert call_norm(lib, g, gate=G) == OK
    assert call_norm(lib, g, gate=G + 2) == 4
    assert call_norm(lib, g, y=None) == OK                        # no branch, no gate
    assert call_norm(lib, norm(gate_kind=1), gate=G + 2) == OK    # a bf16 per token
    # in place only over rows that coincide
    assert call_norm(lib, n, xo=X) == OK and call_norm(lib, n, h=Y) == OK
    assert call_norm(lib, norm(x_ld=512), xo=X) == 1
    assert call_norm(lib, norm(y_ld=512), h=Y) == 1
    assert call_norm(lib, n, xo=Y) == 1 and call_norm(lib, n, h=X) == 1
    assert call_norm(lib, n, xo=H, h=H) == 1


def test_quant_arguments(lib):
    f = lib.moe_fp8_quant
    assert f(X, 0, 0, 128, C, S, None) == OK
    assert f(X, 136, 0, 128, C, S, None) == OK
    assert f(X, 64, 0, 128, C, S, None) == 1 and f(X, 132, 0, 128, C, S, None) == 1
    assert f(None, 0, 1, 128, C, S, None) == 1 and f(X, 0, 1, 128, None, S, None) == 1
    assert f(X, 0, -1, 128, C, S, None) == 1 and f(X, 0, 2**31 - 1, 128, C, S, None) == 2
    assert f(X, 0, 1, 132, C, S, None) == 2 and f(X, 0, 1, 65544, C, S, None) == 2
    assert f(X + 2, 0, 1, 128, C, S, None) == 4 and f(X, 0, 1, 128, C + 4, S, None) == 4


def mat(**kw):
    m = dict(n=100, k=256, groups=1, codes=C, scales=S)
    m.update(kw)
    return moe_ops.moe_fp8_mat(**m)


def test_gemm_arguments(lib):
    def f(m, a=X, sa=G, M=0, c=Y, ws=None):
        return lib.moe_fp8_gemm(ref(m), a, sa, M, c, ws, None)
    assert f(mat()) == OK and f(mat(), ws=WS) == OK
    for kw in (dict(n=0), dict(n=65537), dict(k=0), dict(k=24), dict(k=65552), dict(groups=0),
               dict(groups=1025), dict(n=65536, groups=1024 * 32)):
        assert f(mat(**kw)) == 2, kw
    assert f(mat(codes=None)) == 1 and f(mat(scales=None)) == 1
    assert f(mat(codes=C + 8)) == 4
    assert f(mat(groups=2)) == 1                                  # groups need offsets
    assert lib.moe_fp8_gemm(None, X, G, 0, Y, None, None) == 1
    assert f(mat(), a=None) == 1 and f(mat(), sa=None) == 1 and f(mat(), c=None) == 1
    assert f(mat(), M=-1) == 1 and f(mat(), M=2**31 - 1) == 2
    assert f(mat(), a=X + 8) == 4 and f(mat(), c=Y + 1) == 4 and f(mat(), ws=WS + 16) == 4
    assert f(mat(), c=Y + 2) == OK


def test_grouped_arguments(lib):
    def f(m, off=H, M=0):
        return lib.moe_fp8_gemm_grouped(ref(m), X, G, M, off, Y, None, None)
    assert f(mat(groups=7)) == OK and f(mat()) == OK
    assert f(mat(groups=7), off=None) == 1
    assert f(mat(groups=7), off=H + 2) == 4
    assert f(mat(n=65536, groups=1024)) == OK                     # the largest


def layer(**kw):
    base = dict(d_model=64, n_experts=16, ffn=32, top_k=2, shared_ffn=32)
    names = ("router_w", "gate_up", "gate_up_scales", "down", "down_scales", "shared_gate_up",
             "shared_gate_up_scales", "shared_down", "shared_down_scales")
    base.update({n: P + 0x10000000 + i * 0x100000 for i, n in enumerate(names)})
    base.update(kw)
    return moe_ops.moe_fp8_layer(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(d_model=48), 2), (dict(d_model=8192), 2), (dict(ffn=16), 2), (dict(ffn=40), 2),
    (dict(shared_ffn=-32), 2), (dict(shared_ffn=4128), 2), (dict(top_k=0), 2), (dict(top_k=17), 2),
    (dict(n_experts=1), 2), (dict(n_experts=1025), 2), (dict(router_w=None), 1),
    (dict(gate_up=None), 1), (dict(down_scales=None), 1), (dict(shared_down=None), 1),
    (dict(gate_up=P + 8), 4), (dict(shared_gate_up=P + 4), 4), (dict(router_bias=P + 2), 4)])
def test_layer_struct(lib, kw, status):
    L = layer(**kw)
    assert lib.moe_fp8_layer_forward(ref(L), X, 0, Y, None, None, WS, 1 << 30, None) == status
    assert lib.moe_fp8_layer_workspace_bytes(ref(L), 8) == 0


def test_layer_arguments(lib):
    L = layer()
    need = lib.moe_fp8_layer_workspace_bytes(ref(L), 8)
    assert need > 0 and need % 256 == 0
    assert lib.moe_fp8_layer_workspace_bytes(ref(L), -1) == 0
    assert lib.moe_fp8_layer_workspace_bytes(None, 1) == 0

    def f(x=X, T=0, y=Y, ids=None, w=None, ws=WS, n=1 << 30):
        return lib.moe_fp8_layer_forward(ref(L), x, T, y, ids, w, ws, n, None)
    assert f() == OK and f(n=need) == OK
    assert f(n=need - 1) == 3
    assert f(x=None) == 1 and f(y=None) == 1 and f(ws=None) == 1 and f(T=-1) == 1
    assert f(y=X) == 1                                            # y may not be x
    assert f(x=X + 8) == 4 and f(y=Y + 8) == 4 and f(ws=WS + 16) == 4 and f(ids=G + 2) == 4
    assert f(T=moe_ops.FP8_LAYER_MAX_T + 1) == 2
    assert lib.moe_fp8_layer_forward(None, X, 1, Y, None, None, WS, 1 << 30, None) == 1
    # without a shared expert its pointers may be missing
    L = layer(shared_ffn=0, shared_gate_up=None, shared_gate_up_scales=None, shared_down=None,
              shared_down_scales=None)
    assert f() == OK


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    w = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moe_ops.make_norm(64, pre_w=w[0])
    with pytest.raises(ValueError):
        moe_ops.make_norm(64, gate="row")
    with pytest.raises(ValueError):
        moe_ops.make_fp8_mat(w, w)
    with pytest.raises(ValueError):
        moe_ops.moe_fp8_quant(w.bfloat16(), w, w)
    for f in (moe_ops._need, lambda *a: moe_ops._rows(*a, {})):
        with pytest.raises(ValueError, match="expected a tensor"):
            f(None, "x", (torch.bfloat16,), (4, 64), -1)
    with pytest.raises(ValueError):
        moe_ops.make_fp8_mat(w.to(torch.float8_e4m3fn), None)


def test_binding_takes_pitched_rows_and_refuses_overlapping_ones():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    bf16, host, seen = (torch.bfloat16,), -1, {}
    assert moe_ops._rows(x[:, :32], "x", bf16, (4, 32), host, seen) == x.data_ptr()
    assert seen == {"x_ld": 64}
    for t in (x[:1].expand(4, 64), x.view(-1).as_strided((4, 64), (32, 1)), x.t()):
        with pytest.raises(ValueError):
            moe_ops._rows(t, "x", bf16, tuple(t.shape), host, {})


def test_header_compiles_as_c99_and_ctypes_mirrors_the_structs(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    structs = [moe_ops.moe_norm, moe_ops.moe_fp8_mat, moe_ops.moe_fp8_layer]
    src = ["#include <stddef.h>", "#include <stdio.h>", '#include "moe_ops.h"', "int main(void) {",
           '  printf("%d\\n", MOE_FP8_LAYER_MAX_T);']
    for s in structs:
        src.append(f'  printf("%zu\\n", sizeof({s.__name__}));')
        src += [f'  printf("%zu\\n", offsetof({s.__name__}, {f}));' for f, _ in s._fields_]
    src += ["  return 0;", "}"]
    c, exe = tmp_path / "layout.c", tmp_path / "layout"
    c.write_text("\n".join(src) + "\n")
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    out = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    want = [moe_ops.FP8_LAYER_MAX_T]
    for s in structs:
        want += [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]
    assert out == want


def test_status_is_raised(lib):
    with pytest.raises(moe.MoEError) as e:
        moe._check(call_norm(lib, norm(d=4)), "moe_norm_block")
    assert e.value.status == 2
