"""ctypes binding of the C ABI in ``include/moe_ops.h``: the operators around
and beside the routed block (fused norms, e4m3 block-scaled products, the MoE
layer with e4m3 experts).

As in :mod:`.moe`, functions keep the C names, tensors are torch tensors, the
stream is torch's current stream unless one is passed, and nothing falls back
to another implementation.  Tensors have to lie on the current CUDA device,
with the types and shapes the header gives; the checks here raise
``ValueError``, the library's own raise ``MoEError``.

e4m3 codes are ``torch.float8_e4m3fn`` (or ``uint8`` holding the same bits).
A handle (``make_norm``, ``make_fp8_mat``, ``make_fp8_layer``) holds the
struct the C call reads and keeps the weight tensors alive.
"""
from __future__ import annotations

import ctypes

import torch

from . import moe
from .moe import MoEError, _check, _ptr, _stream

NORM_F_POST = 1
NORM_F_ZERO_CENTRED = 2
NORM_F_STREAM_F32 = 4
NORM_F_SIGMOID = 8

GATES = {"none": 0, "token": 1, "channel": 2, "full": 3}

FP8_LAYER_MAX_T = 32

EXPORTS = ["moe_norm_block", "moe_fp8_quant", "moe_fp8_gemm", "moe_fp8_gemm_grouped",
           "moe_fp8_layer_workspace_bytes", "moe_fp8_layer_forward"]


class moe_norm(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("flags", ctypes.c_uint32), ("gate_kind", ctypes.c_int32),
                ("eps", ctypes.c_float), ("stream_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("pre_w", ctypes.c_void_p),
                ("post_w", ctypes.c_void_p), ("x_ld", ctypes.c_int64), ("y_ld", ctypes.c_int64),
                ("gate_ld", ctypes.c_int64), ("x_out_ld", ctypes.c_int64),
                ("h_ld", ctypes.c_int64)]


class moe_fp8_mat(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("k", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class moe_fp8_layer(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("shared_ffn", ctypes.c_int32),
                ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("gate_up", ctypes.c_void_p), ("gate_up_scales", ctypes.c_void_p),
                ("down", ctypes.c_void_p), ("down_scales", ctypes.c_void_p),
                ("shared_gate_up", ctypes.c_void_p), ("shared_gate_up_scales", ctypes.c_void_p),
                ("shared_down", ctypes.c_void_p), ("shared_down_scales", ctypes.c_void_p)]


_lib = None


def load() -> ctypes.CDLL:
    """libmoe.so with the signatures of moe_ops.h (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    L = moe.load()
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    st = ctypes.c_int
    for name, args in [
            ("moe_norm_block", [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp]),
            ("moe_fp8_quant", [vp, i64, i32, i32, vp, vp, vp]),
            ("moe_fp8_gemm", [vp, vp, vp, i32, vp, vp, vp]),
            ("moe_fp8_gemm_grouped", [vp, vp, vp, i32, vp, vp, vp, vp]),
            ("moe_fp8_layer_forward", [vp, vp, i32, vp, vp, vp, vp, sz, vp])]:
        f = getattr(L, name)
        f.restype, f.argtypes = st, args
    L.moe_fp8_layer_workspace_bytes.restype = sz
    L.moe_fp8_layer_workspace_bytes.argtypes = [vp, i32]
    _lib = L
    return L


_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _need(t, name, dtypes, shape=None, rows_only=False):
    """Check one tensor: on the current device, of one of dtypes, of the shape
    given, dense (or, with rows_only, rows dense and any row pitch)."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: on {t.device}, not on the current CUDA device")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if rows_only:
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: rows are not dense")
    elif not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")


def _blocks(n: int) -> int:
    return -(-n // 128)


class _Handle:
    """A C struct, its address, and the tensors it points to."""

    def __init__(self, struct, *keep):
        self.struct = struct
        self.ref = ctypes.addressof(struct)
        self.keep = keep


# ------------------------------------------------------------------- norms
def make_norm(d: int, pre_w=None, post_w=None, post: bool = False, gate: str = "none",
              gate_act: str = "none", zero_centred: bool = False, stream_f32: bool = False,
              stream_scale: float = 1.0, branch_scale: float = 1.0, eps: float = 1e-6) -> _Handle:
    """Weights and constants of the norms between two blocks (moe_norm).
    pre_w, post_w: fp32 [d] or None (factor 1); gate: "none", "token",
    "channel" or "full"; gate_act: "none" or "sigmoid"."""
    if gate not in GATES or gate_act not in ("none", "sigmoid"):
        raise ValueError(f"gate {gate!r} / {gate_act!r}")
    for name, w in (("pre_w", pre_w), ("post_w", post_w)):
        if w is not None:
            _need(w, name, _F32, (d,))
    flags = ((NORM_F_POST if post else 0) | (NORM_F_ZERO_CENTRED if zero_centred else 0)
             | (NORM_F_STREAM_F32 if stream_f32 else 0)
             | (NORM_F_SIGMOID if gate_act == "sigmoid" else 0))
    return _Handle(moe_norm(d, flags, GATES[gate], eps, stream_scale, branch_scale, _ptr(pre_w),
                            _ptr(post_w)), pre_w, post_w)


def moe_norm_block(n: _Handle, x, y, gate, T: int, x_out=None, h=None, codes=None, scales=None,
                   stream=None) -> None:
    """The norms after one block and before the next (include/moe_ops.h).  x,
    y, gate ("full"), x_out, h: [T, d] with dense rows and any row pitch the
    library takes; y may be None."""
    s, ref = n.struct, n.ref
    d, kind = s.d, s.gate_kind
    sdt = _F32 if s.flags & NORM_F_STREAM_F32 else _BF16
    pitched = {}
    for name, t, dt in (("x", x, sdt), ("y", y, _BF16), ("gate", gate if kind == 3 else None, _BF16),
                        ("x_out", x_out, sdt), ("h", h, _BF16)):
        if t is not None:
            _need(t, name, dt, (T, d), True)
            if T > 1 and t.stride(0) != d:
                pitched[name + "_ld"] = t.stride(0)
    if pitched:   # the handle itself is never written: calls may share it
        s = moe_norm.from_buffer_copy(s)
        for name, v in pitched.items():
            setattr(s, name, v)
        ref = ctypes.addressof(s)
    if gate is not None and kind in (1, 2):
        _need(gate, "gate", _BF16, (T,) if kind == 1 else (d,))
    if codes is not None:
        _need(codes, "codes", _E4M3, (T, d))
    if scales is not None:
        _need(scales, "scales", _F32, (T, _blocks(d)))
    if T == 0:   # an empty tensor has no address to pass
        return
    _check(load().moe_norm_block(ref, _ptr(x), _ptr(y), _ptr(gate), T, _ptr(x_out), _ptr(h),
                                 _ptr(codes), _ptr(scales), _stream(stream)), "moe_norm_block")


# ---------------------------------------------------------------- products
def make_fp8_mat(codes, scales) -> _Handle:
    """A weight matrix [N, K], or one per group [G, N, K], with its block
    scales [(G,) ceil(N/128), ceil(K/128)]."""
    if codes.dim() not in (2, 3):
        raise ValueError("codes: [N, K] or [G, N, K]")
    lead, (N, K) = tuple(codes.shape[:-2]), codes.shape[-2:]
    _need(codes, "codes", _E4M3)
    _need(scales, "scales", _F32, lead + (_blocks(N), _blocks(K)))
    return _Handle(moe_fp8_mat(N, K, lead[0] if lead else 1, _ptr(codes), _ptr(scales)), codes,
                   scales)


def moe_fp8_quant(x, codes, scales, stream=None) -> None:
    """bf16 rows [T, d] to e4m3 codes [T, d] and scales [T, ceil(d/128)]."""
    if x.dim() != 2:
        raise ValueError("x: [T, d]")
    T, d = x.shape
    _need(x, "x", _BF16, rows_only=True)
    _need(codes, "codes", _E4M3, (T, d))
    _need(scales, "scales", _F32, (T, _blocks(d)))
    if T == 0:
        return
    _check(load().moe_fp8_quant(_ptr(x), x.stride(0) if T > 1 else 0, T, d, _ptr(codes),
                                _ptr(scales), _stream(stream)), "moe_fp8_quant")


def _products(w, a, a_scales, M, c):
    s = w.struct
    _need(a, "a", _E4M3, (M, s.k))
    _need(a_scales, "a_scales", _F32, (M, _blocks(s.k)))
    _need(c, "c", _BF16, (M, s.n))


def moe_fp8_gemm(w: _Handle, a, a_scales, M: int, c, ws=None, stream=None) -> None:
    """c = (a * a_scales) (w * w_scales)^T in bf16 (include/moe_ops.h)."""
    _products(w, a, a_scales, M, c)
    if M == 0:
        return
    _check(load().moe_fp8_gemm(w.ref, _ptr(a), _ptr(a_scales), M, _ptr(c), _ptr(ws),
                               _stream(stream)), "moe_fp8_gemm")


def moe_fp8_gemm_grouped(w: _Handle, a, a_scales, M: int, offsets, c, ws=None, stream=None) -> None:
    """The same with group g's matrix for rows offsets[g] <= m < offsets[g+1]."""
    _products(w, a, a_scales, M, c)
    _need(offsets, "offsets", _I32, (w.struct.groups + 1,))
    if M == 0:
        return
    _check(load().moe_fp8_gemm_grouped(w.ref, _ptr(a), _ptr(a_scales), M, _ptr(offsets), _ptr(c),
                                       _ptr(ws), _stream(stream)), "moe_fp8_gemm_grouped")


# ------------------------------------------------------------------- layer
def make_fp8_layer(top_k: int, router_w, router_bias, gate_up, gate_up_scales, down, down_scales,
                   shared_gate_up=None, shared_gate_up_scales=None, shared_down=None,
                   shared_down_scales=None) -> _Handle:
    """A MoE layer with e4m3 experts: router_w fp32 [E, d], router_bias fp32
    [E] or None, gate_up e4m3 [E, 2, F, d] (gate rows, then up rows), down
    [E, d, F], the shared expert [2, Fs, d] and [d, Fs] or None, each with its
    scales per 128 x 128 block."""
    E, d = router_w.shape
    F = gate_up.shape[-2]
    Fs = 0 if shared_gate_up is None else shared_gate_up.shape[-2]
    kd, kf, ks = _blocks(d), _blocks(F), _blocks(Fs)
    _need(router_w, "router_w", _F32)
    if router_bias is not None:
        _need(router_bias, "router_bias", _F32, (E,))
    _need(gate_up, "gate_up", _E4M3, (E, 2, F, d))
    _need(gate_up_scales, "gate_up_scales", _F32, (E, 2, kf, kd))
    _need(down, "down", _E4M3, (E, d, F))
    _need(down_scales, "down_scales", _F32, (E, kd, kf))
    if Fs:
        _need(shared_gate_up, "shared_gate_up", _E4M3, (2, Fs, d))
        _need(shared_gate_up_scales, "shared_gate_up_scales", _F32, (2, ks, kd))
        _need(shared_down, "shared_down", _E4M3, (d, Fs))
        _need(shared_down_scales, "shared_down_scales", _F32, (kd, ks))
    keep = (router_w, router_bias, gate_up, gate_up_scales, down, down_scales, shared_gate_up,
            shared_gate_up_scales, shared_down, shared_down_scales)
    return _Handle(moe_fp8_layer(d, E, F, top_k, Fs, *map(_ptr, keep)), *keep)


def moe_fp8_layer_workspace_bytes(layer: _Handle, max_tokens: int) -> int:
    return load().moe_fp8_layer_workspace_bytes(layer.ref, int(max_tokens))


def alloc_fp8_workspace(layer: _Handle, max_tokens: int, device=None) -> torch.Tensor:
    n = moe_fp8_layer_workspace_bytes(layer, max_tokens)
    if n == 0:
        raise MoEError(1, "moe_fp8_layer_workspace_bytes")
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    moe.moe_workspace_init(ws)
    return ws


def moe_fp8_layer_forward(layer: _Handle, x, T: int, y, ws, ids=None, w=None, stream=None) -> None:
    """The whole layer for up to FP8_LAYER_MAX_T tokens (include/moe_ops.h)."""
    s = layer.struct
    _need(x, "x", _BF16, (T, s.d_model))
    _need(y, "y", _BF16, (T, s.d_model))
    if ids is not None:
        _need(ids, "ids", _I32, (T, s.top_k))
    if w is not None:
        _need(w, "w", _F32, (T, s.top_k))
    if T == 0:
        return
    _check(load().moe_fp8_layer_forward(layer.ref, _ptr(x), T, _ptr(y), _ptr(ids), _ptr(w),
                                        _ptr(ws), ws.numel(), _stream(stream)),
           "moe_fp8_layer_forward")
