"""Projections around a mixer and rows in 8 bits (binding of ``replayssm_linear``,
``replayssm_quantize_mx``, ``replayssm_gated_norm_mx`` and ``replayssm_add_norm_mx``).

Rows in 8 bits are a pair ``(codes, scales)`` of dense device tensors: codes
[rows, dim] ``torch.float8_e4m3fn`` and scales [rows, dim / 32]
``torch.float8_e8m0fnu``, one power of two per 32 consecutive elements (OCP MX).
The norms write such pairs, ``quantize_mx`` makes them of weights once, and
``linear`` takes them as operands and can return one.
"""
from __future__ import annotations

import ctypes

import torch

from . import BF16, F32, FP8_E4M3, NONE, ReplaySSMError, _check, _need, lib
from .mixer import _TYPES, _empty, _pitch, _raw_stream

__all__ = ["linear", "quantize_mx", "gated_norm_mx", "add_norm_mx"]

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_BLOCK = 32   # elements that share a scale
_ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "relu2": 3}
_OUT_TYPES = {torch.float32: F32, torch.bfloat16: BF16, _E4M3: FP8_E4M3}


class RssmLinearDesc(ctypes.Structure):
    _fields_ = [("rows", _i64)] + [(n, _i32) for n in ("n_in", "n_out", "in_dtype", "out_dtype", "res_dtype",
                                                       "activation")] + [("scale", _f32), ("products", _i32)]


class RssmLinearIO(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_pitch", _i64)] + [(n, _vp) for n in ("x_scales", "weight", "weight_scales", "bias",
                                                                     "residual", "out", "out_scales")]


_BOUND = None


def _lib():
    """The library, with the argument types of these calls set."""
    global _BOUND
    L = lib()
    if _BOUND is not L:
        L.replayssm_quantize_mx.argtypes = [_i64, _i32, _vp, _i32, _i64, _vp, _vp, _vp]
        L.replayssm_gated_norm_mx.argtypes = [_i64, _i32, _i32, _vp, _i32, _vp, _i32, _i64, _vp, _f32, _i32, _vp, _vp,
                                              _vp]
        L.replayssm_add_norm_mx.argtypes = [_i64, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _f32, _f32, _vp, _vp, _vp]
        L.replayssm_linear.argtypes = [_vp, _vp, _vp]
        for n in ("quantize_mx", "gated_norm_mx", "add_norm_mx", "linear"):
            getattr(L, "replayssm_" + n).restype = ctypes.c_int
        _BOUND = L
    return L


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device(t, name: str) -> int:
    """The device of a call's tensors, which has to be the current one (launches go there).
    (A token's calls are bound by the host: each tensor is looked at once, in ``_at``.)"""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise ReplaySSMError(f"{name}: expected a device tensor, got "
                             f"{f'{tuple(t.shape)} {t.dtype} device={t.device}' if isinstance(t, torch.Tensor) else type(t).__name__}")
    if dev != _current_device():
        raise ReplaySSMError(f"{name}: is on device {dev}, which is not the current one (torch.cuda.device)")
    return dev


def _at(t: torch.Tensor, shape: tuple, dtype, dev: int, name: str) -> int:
    """Address of a dense tensor of this shape and type on device ``dev`` (else raise)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _need(t, shape, dtype, name)
    raise ReplaySSMError(f"{name}: is on device {t.get_device()}, the call's other tensors on {dev}")


def _type(t, name: str) -> int:
    ty = _TYPES.get(t.dtype)
    if ty is None:
        raise ReplaySSMError(f"{name}: expected fp32 or bf16, got {t.dtype}")
    return ty


def _mx(pair, rows: int, dim: int, dev: int, name: str):
    """Addresses of codes and scales of MX rows (else raise)."""
    if not isinstance(pair, (tuple, list)) or len(pair) != 2:
        raise ReplaySSMError(f"{name}: expected a pair (codes, scales)")
    codes, scales = pair
    return (_at(codes, (rows, dim), _E4M3, dev, name + " codes"),
            _at(scales, (rows, dim // _BLOCK), _E8M0, dev, name + " scales"))


def _blocks(dim: int, name: str) -> None:
    if dim % _BLOCK or not dim:
        raise ReplaySSMError(f"{name}: MX rows hold a positive multiple of {_BLOCK} elements, got {dim}")


def _mx_empty(rows: int, dim: int, device, stream):
    return _empty((rows, dim), _E4M3, device, stream), _empty((rows, dim // _BLOCK), _E8M0, device, stream)


def quantize_mx(x, *, out=None, stream=None):
    """Rows to MX (replayssm_quantize_mx): x [rows,dim] fp32 or bf16, a view of
    evenly spaced rows or dense; returns (codes, scales)."""
    if x.dim() != 2:
        raise ReplaySSMError(f"x: expected [rows, dim], got {tuple(x.shape)}")
    rows, dim = x.shape
    _blocks(dim, "x")
    dev, xt = _device(x, "x"), _type(x, "x")
    pitch = dim if x.is_contiguous() else _pitch(x, (rows,), dim, x.dtype, "x")
    if out is None:
        out = _mx_empty(rows, dim, x.device, stream)
    codes, scales = _mx(out, rows, dim, dev, "out")
    rc = _lib().replayssm_quantize_mx(rows, dim, x.data_ptr(), xt, pitch, codes, scales, _raw_stream(stream, x))
    if rc:
        _check(rc)
    return out


def gated_norm_mx(y, z, weight, *, groups: int = 1, eps: float = 1e-5, norm_before_gate: bool = False, out=None,
                  stream=None):
    """``gated_norm`` with its output in MX (replayssm_gated_norm_mx); returns (codes, scales)."""
    if z.dim() != 2:
        raise ReplaySSMError(f"z: expected [rows, dim], got {tuple(z.shape)}")
    rows, dim = z.shape
    _blocks(dim, "z")
    dev, yt, zt = _device(z, "z"), _type(y, "y"), _type(z, "z")
    if y.shape[:1] != (rows,) or y.numel() != rows * dim or not y.is_contiguous() or y.get_device() != dev:
        raise ReplaySSMError(f"y: expected a dense tensor of {rows} rows of {dim} on device {dev}, got {tuple(y.shape)} "
                             f"contiguous={y.is_contiguous()} device={y.device}")
    pitch = _pitch(z, (rows,), dim, z.dtype, "z")
    w = _at(weight, (dim,), torch.float32, dev, "weight")
    if out is None:
        out = _mx_empty(rows, dim, z.device, stream)
    codes, scales = _mx(out, rows, dim, dev, "out")
    rc = _lib().replayssm_gated_norm_mx(rows, dim, groups, y.data_ptr(), yt, z.data_ptr(), zt, pitch, w, eps,
                                        1 if norm_before_gate else 0, codes, scales, _raw_stream(stream, z))
    if rc:
        _check(rc)
    return out


def add_norm_mx(x, residual, weight, *, scale: float = 1.0, post_weight=None, eps: float = 1e-5, out=None,
                residual_out=None, stream=None):
    """``add_norm`` with its output in MX (replayssm_add_norm_mx); returns
    ((codes, scales), new residual).  With ``x`` None it is the norm of the
    residual alone, which is returned as it is."""
    if residual.dim() != 2:
        raise ReplaySSMError(f"residual: expected [rows, dim], got {tuple(residual.shape)}")
    rows, dim = shape = residual.shape
    _blocks(dim, "residual")
    dev, ty = _device(residual, "residual"), residual.dtype
    rt = _type(residual, "residual")
    rp = _at(residual, shape, ty, dev, "residual")
    w = _at(weight, (dim,), torch.float32, dev, "weight")
    p = None if post_weight is None else _at(post_weight, (dim,), torch.float32, dev, "post_weight")
    if x is None:
        if residual_out is not None or post_weight is not None:
            raise ReplaySSMError("x: residual_out and post_weight go with it")
        xp, xt, op = None, F32, None
    else:
        xt = _type(x, "x")
        xp = _at(x, shape, x.dtype, dev, "x")
        if residual_out is None:
            residual_out = _empty(shape, ty, residual.device, stream)
        op = _at(residual_out, shape, ty, dev, "residual_out")
    if out is None:
        out = _mx_empty(rows, dim, residual.device, stream)
    codes, scales = _mx(out, rows, dim, dev, "out")
    rc = _lib().replayssm_add_norm_mx(rows, dim, xp, xt, rp, op, rt, w, p, scale, eps, codes, scales,
                                      _raw_stream(stream, residual))
    if rc:
        _check(rc)
    return out, residual if x is None else residual_out


def linear(x, weight, bias=None, *, activation: str | None = None, residual=None, scale: float = 1.0, out=None,
           out_dtype: torch.dtype = torch.bfloat16, fast_products: bool = False, stream=None):
    """Matrix product with its epilogue (replayssm_linear):
    ``residual + scale * act(x @ weight.T + bias)``.

    x [rows,n_in] and weight [n_out,n_in] are bf16 (x a view of evenly spaced rows
    or dense), or both MX pairs; bias [n_out] fp32; activation None, "silu",
    "gelu" or "relu2"; residual [rows,n_out] fp32 or bf16, which may be ``out``.
    Returns [rows,n_out] in ``out_dtype`` (of ``out`` when it is given): bf16, fp32,
    or ``torch.float8_e4m3fn`` for an MX pair.

    ``fast_products`` allows products of MX rows that may be off by 2^-13 of the
    largest among 16 neighbouring ones (RSSM_PRODUCTS_FAST), at up to twice the
    rate; large products that cancel may then take small ones with them."""
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ReplaySSMError(f"activation must be None, 'silu', 'gelu' or 'relu2', got {activation!r}")
    mx = isinstance(x, (tuple, list))
    if mx != isinstance(weight, (tuple, list)):
        raise ReplaySSMError("x and weight: both are MX pairs or neither")
    xs, ws = (x[0], weight[0]) if mx and x and weight else (x, weight)
    dev = _device(xs, "x")
    if xs.dim() != 2 or not isinstance(ws, torch.Tensor) or ws.dim() != 2:
        raise ReplaySSMError("x and weight: expected [rows, n_in] and [n_out, n_in]")
    rows, n_in = xs.shape
    n_out = ws.shape[0]
    if mx:
        _blocks(n_in, "x")
        xp, xsp = _mx(x, rows, n_in, dev, "x")
        wp, wsp = _mx(weight, n_out, n_in, dev, "weight")
        pitch, ty = n_in, FP8_E4M3
    else:
        if xs.dtype is torch.bfloat16 and xs.is_contiguous():
            pitch = n_in
        else:
            pitch = _pitch(xs, (rows,), n_in, torch.bfloat16, "x")
        xp, xsp, wsp, ty = xs.data_ptr(), None, None, BF16
        wp = _at(weight, (n_out, n_in), torch.bfloat16, dev, "weight")
    bp = None if bias is None else _at(bias, (n_out,), torch.float32, dev, "bias")
    rp, rt = None, NONE
    if residual is not None:
        rt = _type(residual, "residual")
        rp = _at(residual, (rows, n_out), residual.dtype, dev, "residual")
    if out is not None:
        out_dtype = _E4M3 if isinstance(out, (tuple, list)) else out.dtype
    ot = _OUT_TYPES.get(out_dtype)
    if ot is None or (ot == FP8_E4M3 and isinstance(out, torch.Tensor)):
        raise ReplaySSMError(f"out: bfloat16, float32 or an MX pair (float8_e4m3fn), got {out_dtype}")
    if ot == FP8_E4M3:
        _blocks(n_out, "out")
        if out is None:
            out = _mx_empty(rows, n_out, xs.device, stream)
        op, osp = _mx(out, rows, n_out, dev, "out")
    else:
        if out is None:
            out = _empty((rows, n_out), out_dtype, xs.device, stream)
        op, osp = _at(out, (rows, n_out), out_dtype, dev, "out"), None
    d = RssmLinearDesc(rows, n_in, n_out, ty, ot, rt, act, scale, 1 if fast_products else 0)
    io = RssmLinearIO(xp, pitch, xsp, wp, wsp, bp, rp, op, osp)
    rc = _lib().replayssm_linear(ctypes.addressof(d), ctypes.addressof(io), _raw_stream(stream, xs))
    if rc:
        _check(rc)
    return out
