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
from .moe import MoEError, _check, _ptr

# The current device and a device's current stream as plain integers: torch's
# public calls build objects on the way (3 us for a stream, as long as a launch).
_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

NORM_F_POST = 1
NORM_F_ZERO_CENTRED = 2
NORM_F_STREAM_F32 = 4
NORM_F_SIGMOID = 8

GATES = {"none": 0, "token": 1, "channel": 2, "full": 3}

FP8_LAYER_MAX_T = 32

EXPORTS = ["moe_norm_block", "moe_fp8_quant", "moe_fp8_gemm", "moe_fp8_gemm_grouped",
           "moe_fp8_gemm_plan", "moe_fp8_layer_workspace_bytes", "moe_fp8_layer_forward"]


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
            ("moe_fp8_gemm_plan", [vp, i32, i32, vp]),
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


def _stream(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _need(t, name, dtypes, shape, dev):
    """Check one tensor: on the current device `dev`, of one of dtypes, of the
    shape given, dense.  Returns its address."""
    try:
        if t.dtype in dtypes and t.get_device() == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise ValueError(f"{name}: {type(t).__name__}, expected a tensor") from None
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, not on the current CUDA device")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name}: not contiguous")


def _shape(t, name, form, *ranks):
    """Shape of a tensor that has one of these numbers of dimensions."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: {type(t).__name__}, expected a tensor")
    if t.dim() not in ranks:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {form}")
    return t.shape


def _rows(t, name, dtypes, shape, dev, pitched):
    """The same for rows that are dense themselves but may have any pitch, which
    is noted in the dict `pitched` where it is not the row's length."""
    try:
        if t.dtype in dtypes and t.get_device() == dev and t.shape == shape:
            if t.is_contiguous():
                return t.data_ptr()
            if shape[1] == 1 or t.stride(1) == 1:
                if shape[0] > 1:
                    # a pitch of 0 (an expanded row) would mean dense rows to the library
                    if t.stride(0) < shape[1]:
                        raise ValueError(f"{name}: rows overlap")
                    pitched[name + "_ld"] = t.stride(0)
                return t.data_ptr()
            raise ValueError(f"{name}: rows are not dense")
    except AttributeError:
        pass   # no tensor: said below
    return _need(t, name, dtypes, shape, dev)


def _current():
    """The current CUDA device, -2 (no tensor's) where there is none."""
    return _device() if torch.cuda.is_initialized() else -2


def _blocks(n: int) -> int:
    return -(-n // 128)


class _Handle:
    """A C struct, its address, the tensors it points to and their device (None
    without any)."""

    def __init__(self, struct, *keep):
        self.struct = struct
        self.ref = ctypes.addressof(struct)
        self.keep = keep
        self.dev = next((t.get_device() for t in keep if t is not None), None)

    def here(self, dev):
        if self.dev is not None and self.dev != dev:
            raise ValueError(f"weights on cuda:{self.dev}, not on the current CUDA device")


CONTROL_BYTES = 256     # a workspace's control block, which holds the error word


def _workspace(ws, dev):
    """Address of a workspace: dense bytes on the current device, a control block
    of them at least."""
    if ws is None:
        return None
    p = _need(ws, "ws", (torch.uint8,), getattr(ws, "shape", None), dev)
    if ws.numel() < CONTROL_BYTES:
        raise ValueError(f"ws: {ws.numel()} bytes, expected at least {CONTROL_BYTES}")
    return p


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
            _need(w, name, _F32, (d,), _current())
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
    s, ref, dev = n.struct, n.ref, _current()
    n.here(dev)
    d, kind = s.d, s.gate_kind
    sdt, rows = _F32 if s.flags & NORM_F_STREAM_F32 else _BF16, (T, d)
    pitched = {}
    px = _rows(x, "x", sdt, rows, dev, pitched)
    py = None if y is None else _rows(y, "y", _BF16, rows, dev, pitched)
    pg = None
    if gate is not None and kind:
        pg = _rows(gate, "gate", _BF16, rows, dev, pitched) if kind == 3 else \
            _need(gate, "gate", _BF16, (T,) if kind == 1 else (d,), dev)
    po = None if x_out is None else _rows(x_out, "x_out", sdt, rows, dev, pitched)
    ph = None if h is None else _rows(h, "h", _BF16, rows, dev, pitched)
    pc = None if codes is None else _need(codes, "codes", _E4M3, rows, dev)
    ps = None if scales is None else _need(scales, "scales", _F32, (T, (d + 127) // 128), dev)
    if T == 0:   # an empty tensor has no address to pass
        return
    if pitched:  # the handle itself is never written: calls may share it
        s = moe_norm.from_buffer_copy(s)
        for name, v in pitched.items():
            setattr(s, name, v)
        ref = ctypes.addressof(s)
    st = (_lib or load()).moe_norm_block(ref, px, py, pg, T, po, ph, pc, ps, _stream(stream, dev))
    if st:
        raise MoEError(st, "moe_norm_block")


# ---------------------------------------------------------------- products
def make_fp8_mat(codes, scales) -> _Handle:
    """A weight matrix [N, K], or one per group [G, N, K], with its block
    scales [(G,) ceil(N/128), ceil(K/128)]."""
    shape, dev = _shape(codes, "codes", "[N, K] or [G, N, K]", 2, 3), _current()
    lead, (N, K) = tuple(shape[:-2]), shape[-2:]
    _need(codes, "codes", _E4M3, shape, dev)
    _need(scales, "scales", _F32, lead + (_blocks(N), _blocks(K)), dev)
    return _Handle(moe_fp8_mat(N, K, lead[0] if lead else 1, _ptr(codes), _ptr(scales)), codes,
                   scales)


def moe_fp8_quant(x, codes, scales, stream=None) -> None:
    """bf16 rows [T, d] to e4m3 codes [T, d] and scales [T, ceil(d/128)]."""
    (T, d), dev = _shape(x, "x", "[T, d]", 2), _current()
    pitched = {}
    px = _rows(x, "x", _BF16, x.shape, dev, pitched)
    pc = _need(codes, "codes", _E4M3, (T, d), dev)
    ps = _need(scales, "scales", _F32, (T, _blocks(d)), dev)
    if T == 0:
        return
    _check(load().moe_fp8_quant(px, pitched.get("x_ld", 0), T, d, pc, ps,
                                _stream(stream, dev)), "moe_fp8_quant")


def _products(w, a, a_scales, M, c, dev):
    w.here(dev)
    s = w.struct
    k = s.k
    return (_need(a, "a", _E4M3, (M, k), dev),
            _need(a_scales, "a_scales", _F32, (M, (k + 127) // 128), dev),
            _need(c, "c", _BF16, (M, s.n), dev))


def moe_fp8_gemm(w: _Handle, a, a_scales, M: int, c, ws=None, stream=None) -> None:
    """c = (a * a_scales) (w * w_scales)^T in bf16 (include/moe_ops.h)."""
    dev = _current()
    pa, psa, pc = _products(w, a, a_scales, M, c, dev)
    if M == 0:
        return
    _check(load().moe_fp8_gemm(w.ref, pa, psa, M, pc, _workspace(ws, dev),
                               _stream(stream, dev)), "moe_fp8_gemm")


def moe_fp8_gemm_grouped(w: _Handle, a, a_scales, M: int, offsets, c, ws=None, stream=None) -> None:
    """The same with group g's matrix for rows offsets[g] <= m < offsets[g+1]."""
    dev = _current()
    pa, psa, pc = _products(w, a, a_scales, M, c, dev)
    po = _need(offsets, "offsets", _I32, (w.struct.groups + 1,), dev)
    if M == 0:
        return
    _check(load().moe_fp8_gemm_grouped(w.ref, pa, psa, M, po, pc, _workspace(ws, dev),
                                       _stream(stream, dev)),
           "moe_fp8_gemm_grouped")


def moe_fp8_gemm_plan(w: _Handle, M: int, grouped: bool = False):
    """The kernel a product takes: (tile columns, rows of a staged, ring stages)."""
    plan = (ctypes.c_int32 * 3)()
    _check(load().moe_fp8_gemm_plan(w.ref, M, int(grouped), plan), "moe_fp8_gemm_plan")
    return tuple(plan)


# ------------------------------------------------------------------- layer
def make_fp8_layer(top_k: int, router_w, router_bias, gate_up, gate_up_scales, down, down_scales,
                   shared_gate_up=None, shared_gate_up_scales=None, shared_down=None,
                   shared_down_scales=None) -> _Handle:
    """A MoE layer with e4m3 experts: router_w fp32 [E, d], router_bias fp32
    [E] or None, gate_up e4m3 [E, 2, F, d] (gate rows, then up rows), down
    [E, d, F], the shared expert [2, Fs, d] and [d, Fs] or None, each with its
    scales per 128 x 128 block."""
    E, d = _shape(router_w, "router_w", "[E, d]", 2)
    F = _shape(gate_up, "gate_up", "[E, 2, F, d]", 4)[-2]
    Fs = 0 if shared_gate_up is None else _shape(shared_gate_up, "shared_gate_up", "[2, Fs, d]", 3)[-2]
    kd, kf, ks, dev = _blocks(d), _blocks(F), _blocks(Fs), _current()
    _need(router_w, "router_w", _F32, (E, d), dev)
    if router_bias is not None:
        _need(router_bias, "router_bias", _F32, (E,), dev)
    _need(gate_up, "gate_up", _E4M3, (E, 2, F, d), dev)
    _need(gate_up_scales, "gate_up_scales", _F32, (E, 2, kf, kd), dev)
    _need(down, "down", _E4M3, (E, d, F), dev)
    _need(down_scales, "down_scales", _F32, (E, kd, kf), dev)
    if Fs:
        _need(shared_gate_up, "shared_gate_up", _E4M3, (2, Fs, d), dev)
        _need(shared_gate_up_scales, "shared_gate_up_scales", _F32, (2, ks, kd), dev)
        _need(shared_down, "shared_down", _E4M3, (d, Fs), dev)
        _need(shared_down_scales, "shared_down_scales", _F32, (kd, ks), dev)
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
    s, dev = layer.struct, _current()
    layer.here(dev)
    px = _need(x, "x", _BF16, (T, s.d_model), dev)
    py = _need(y, "y", _BF16, (T, s.d_model), dev)
    pi = None if ids is None else _need(ids, "ids", _I32, (T, s.top_k), dev)
    pw = None if w is None else _need(w, "w", _F32, (T, s.top_k), dev)
    if ws is None:
        raise ValueError("ws: the layer needs a workspace")
    if T == 0:
        return
    _check(load().moe_fp8_layer_forward(layer.ref, px, T, py, pi, pw, _workspace(ws, dev),
                                        ws.numel(), _stream(stream, dev)), "moe_fp8_layer_forward")
