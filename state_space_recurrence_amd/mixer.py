"""Mixer operators around the replayed recurrence (binding of the
``replayssm_conv_*``, ``replayssm_prefill_packed``, ``replayssm_gated_norm`` and
``replayssm_add_norm`` calls).

An SSM layer turns the rows of its input projection, ``[z | x B C | dt]``, into
the block's output: short causal convolution and dt transform -> recurrence ->
gated norm; the next block's input is the normed sum of the block's output and
the residual.  Rows of the projection are taken as strided views; nothing is
copied.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import BF16, F32, LayerState, ReplaySSMError, _check, _ctx, _need, _ptr, lib

__all__ = ["ConvState", "conv_step", "conv_verify", "conv_accept", "conv_prefill", "prefill_packed",
           "gated_norm", "add_norm"]

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_TYPES = {torch.float32: F32, torch.bfloat16: BF16}


class RssmConvDesc(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("batch", "n_slots", "n_heads", "head_dim", "d_state", "n_groups", "width",
                                    "max_draft", "in_dtype", "activation")] + [("dt_min", _f32), ("dt_max", _f32)]


class RssmConvState(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("ring", "head", "work", "weight", "bias", "dt_bias", "slot_idx")]


class RssmConvIO(ctypes.Structure):
    _fields_ = [("u", _vp), ("u_pitch", _i64), ("dt_raw", _vp), ("dt_pitch", _i64),
                ("x", _vp), ("B", _vp), ("C", _vp), ("dt", _vp)]


_CD, _CS, _CI = (ctypes.POINTER(s) for s in (RssmConvDesc, RssmConvState, RssmConvIO))
_BOUND = None


def _lib():
    """The library, with the argument types of the mixer calls set."""
    global _BOUND
    L = lib()
    if _BOUND is not L:
        L.replayssm_conv_step.argtypes = [_CD, _CS, _CI, _vp]
        L.replayssm_conv_verify.argtypes = [_CD, _CS, _i32, _CI, _vp]
        L.replayssm_conv_accept.argtypes = [_CD, _CS, _vp, _i32, _vp]
        L.replayssm_conv_prefill.argtypes = [_CD, _CS, _i64, _vp, _i32, _vp, _CI, _vp]
        L.replayssm_conv_ring_rows.argtypes = [_CD]
        L.replayssm_conv_check_desc.argtypes = [_CD]
        L.replayssm_prefill_packed.argtypes = [_vp, _vp, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                               ctypes.c_size_t, _vp]
        L.replayssm_prefill_packed_workspace.argtypes = [_vp, _i64]
        L.replayssm_prefill_packed_workspace.restype = ctypes.c_size_t
        L.replayssm_gated_norm.argtypes = [_i64, _i32, _i32, _vp, _i32, _vp, _i32, _i64, _vp, _f32, _i32, _vp, _i32,
                                           _vp]
        L.replayssm_add_norm.argtypes = [_i64, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _f32, _f32, _vp, _i32, _vp]
        for n in ("conv_step", "conv_verify", "conv_accept", "conv_prefill", "conv_check_desc", "prefill_packed",
                  "gated_norm", "add_norm"):
            getattr(L, "replayssm_" + n).restype = ctypes.c_int
        L.replayssm_conv_ring_rows.restype = _i32
        _BOUND = L
    return L


_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, t: torch.Tensor) -> int:
    """The stream of a call: the given one, or the current one of t's device.
    (A decode token's calls are bound by the host, so the paths that every
    call takes are kept short: about 4 us a call.)"""
    if stream is not None:
        return stream.cuda_stream
    if _current_raw is not None:
        return _current_raw(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _empty(shape, dtype, device, stream):
    """An output of a call on ``stream``: allocated on that stream, so that its
    memory is not handed on while the call still writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dense(t: torch.Tensor, shape: tuple, dtype, name: str) -> int:
    """Address of a dense device tensor of this shape and type (else raise)."""
    if t.shape == shape and t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _need(t, shape, dtype, name)
    return t.data_ptr()


def _pitch(t: torch.Tensor, lead: tuple, width: int, dtype, name: str) -> int:
    """Elements between consecutive tokens of a view [*lead, width] of a
    projection's rows: innermost dense, tokens evenly spaced."""
    st = t.stride()
    if t.shape != (*lead, width) or t.dtype is not dtype or not t.is_cuda:
        raise ReplaySSMError(f"{name}: expected device tensor {(*lead, width)} {dtype}, got {tuple(t.shape)} "
                             f"{t.dtype} device={t.device}")
    if len(lead) == 1:
        pitch = st[0] if lead[0] > 1 else max(st[0], width)
        even = True
    else:   # the last token axis that has a stride at all gives the pitch
        n, T = lead
        pitch = st[1] if T > 1 else (st[0] if n > 1 else max(st[1], width))
        even = n <= 1 or st[0] == T * pitch
    if (width > 1 and st[-1] != 1) or not even or pitch < width:
        raise ReplaySSMError(f"{name}: rows must be dense and evenly spaced, got strides {st}")
    return pitch


class ConvState:
    """Device state of one layer's causal convolution.

      ring [S,R,Cc] recent raw inputs;  head [S] int32 ring row of the next
      token;  work [S+1] int32;  weight [W,Cc], bias [Cc], dt_bias [H] fp32.

    ``batch`` slots; channels Cc = H*P + 2*G*N ordered x, B, C.  ``weight`` is
    given as [Cc, W] with the last tap on the current token.  A slot starts
    with an all-zero history."""

    def __init__(self, batch: int, heads: int, groups: int, weight: torch.Tensor, bias: torch.Tensor | None = None,
                 dt_bias: torch.Tensor | None = None, *, head_dim: int = 64, d_state: int = 128, max_draft: int = 1,
                 in_dtype: torch.dtype = torch.bfloat16, activation: str | None = "silu",
                 dt_limit: tuple = (0.0, math.inf), device="cuda"):
        if activation not in (None, "silu"):
            raise ReplaySSMError(f"activation must be None or 'silu', got {activation!r}")
        if in_dtype not in _TYPES:
            raise ReplaySSMError(f"in_dtype must be float32 or bfloat16, got {in_dtype}")
        self.batch, self.heads, self.groups, self.head_dim, self.d_state = batch, heads, groups, head_dim, d_state
        self.max_draft, self.in_dtype = max_draft, in_dtype
        self.channels = heads * head_dim + 2 * groups * d_state
        if weight.dim() != 2 or weight.shape[0] != self.channels:
            raise ReplaySSMError(f"weight must have shape ({self.channels}, width), got {tuple(weight.shape)}")
        for t, n, what in ((bias, self.channels, "bias"), (dt_bias, heads, "dt_bias")):
            if t is not None and tuple(t.shape) != (n,):
                raise ReplaySSMError(f"{what} must have shape ({n},), got {tuple(t.shape)}")
        self.width = weight.shape[1]
        self._desc = RssmConvDesc(batch, batch, heads, head_dim, d_state, groups, self.width, max_draft,
                                  _TYPES[in_dtype], int(activation == "silu"), dt_limit[0], dt_limit[1])
        _check(_lib().replayssm_conv_check_desc(ctypes.byref(self._desc)))
        self.ring_rows = _lib().replayssm_conv_ring_rows(ctypes.byref(self._desc))
        dev = torch.device(device)
        f32 = lambda t: None if t is None else t.to(device=dev, dtype=torch.float32).contiguous()  # noqa: E731
        self.weight, self.bias, self.dt_bias = f32(weight.t()), f32(bias), f32(dt_bias)
        self.ring = torch.zeros(batch, self.ring_rows, self.channels, dtype=in_dtype, device=dev)
        self.head = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.work = torch.zeros(batch + 1, dtype=torch.int32, device=dev)

    def tensors(self):
        return {"ring": self.ring, "head": self.head}

    def snapshot(self):
        return {k: v.clone() for k, v in self.tensors().items()}

    def restore(self, snap) -> None:
        for k, v in self.tensors().items():
            v.copy_(snap[k])

    def _call(self, rows, slots):
        if slots is not None:
            at = _dense(slots, (rows,), torch.int32, "slots")
        else:
            at = None
            if rows != self.batch:
                raise ReplaySSMError(f"a call without slots covers all {self.batch} slots, got {rows} rows")
        d = self._desc
        if rows != d.batch:
            d = RssmConvDesc.from_buffer_copy(d)
            d.batch = rows
        return d, RssmConvState(self.ring.data_ptr(), self.head.data_ptr(), self.work.data_ptr(),
                                self.weight.data_ptr(), _ptr(self.bias), _ptr(self.dt_bias), at)

    def _io(self, u, dt, lead, out, stream):
        ty = self.in_dtype
        up, dp = _pitch(u, lead, self.channels, ty, "u"), _pitch(dt, lead, self.heads, ty, "dt")
        head, group = (*lead, self.heads, self.head_dim), (*lead, self.groups, self.d_state)
        if out is None:
            out = tuple(_empty(s, ty, u.device, stream) for s in (head, group, group, (*lead, self.heads)))
        x, B, C, d = out
        return out, RssmConvIO(u.data_ptr(), up, dt.data_ptr(), dp, _dense(x, head, ty, "out x"),
                               _dense(B, group, ty, "out B"), _dense(C, group, ty, "out C"),
                               _dense(d, (*lead, self.heads), ty, "out dt"))

    def check_device_errors(self, stream=None) -> None:
        """Raise if a call on this state met a device-side range error (synchronises)."""
        from . import RssmState
        st = RssmState()
        st.work = self.work.data_ptr()
        _check(lib().replayssm_check_device_errors(ctypes.byref(st), self.batch, _raw_stream(stream, self.work)))


def conv_step(cs: ConvState, u, dt, out=None, stream=None, slots=None):
    """One decode token per row (replayssm_conv_step): u [rows,Cc] and dt
    [rows,H] raw (views of the projection's rows); returns (x, B, C, dt) as
    ``step`` takes them."""
    rows = u.shape[0]
    d, st = cs._call(rows, slots)
    out, io = cs._io(u, dt, (rows,), out, stream)
    _check(_lib().replayssm_conv_step(ctypes.byref(d), ctypes.byref(st), ctypes.byref(io), _raw_stream(stream, u)))
    return out


def conv_verify(cs: ConvState, u, dt, out=None, stream=None, slots=None):
    """T draft positions per row (replayssm_conv_verify): u [rows,T,Cc], dt
    [rows,T,H] raw; returns (x, B, C, dt) as ``verify`` takes them.  The
    history does not move before ``conv_accept``."""
    rows, T = u.shape[:2]
    d, st = cs._call(rows, slots)
    out, io = cs._io(u, dt, (rows, T), out, stream)
    _check(_lib().replayssm_conv_verify(ctypes.byref(d), ctypes.byref(st), T, ctypes.byref(io), _raw_stream(stream, u)))
    return out


def conv_accept(cs: ConvState, n_keep: torch.Tensor, T: int, stream=None, slots=None) -> None:
    """Keep the first n_keep[row] verified positions (replayssm_conv_accept)."""
    rows = n_keep.numel()
    _need(n_keep, (rows,), torch.int32, "n_keep")
    d, st = cs._call(rows, slots)
    _check(_lib().replayssm_conv_accept(ctypes.byref(d), ctypes.byref(st), n_keep.data_ptr(), T,
                                        _raw_stream(stream, n_keep)))


def _packed(cu_seqlens, fresh):
    rows = cu_seqlens.numel() - 1
    if rows < 0:
        raise ReplaySSMError("cu_seqlens: needs at least one offset")
    _need(cu_seqlens, (rows + 1,), torch.int32, "cu_seqlens")
    if fresh is not None:
        _need(fresh, (rows,), torch.int32, "fresh")
    return rows


def conv_prefill(cs: ConvState, u, dt, cu_seqlens, *, from_zero: bool = False, fresh=None, out=None, stream=None,
                 slots=None):
    """Packed prompts (replayssm_conv_prefill): u [total,Cc], dt [total,H] raw,
    cu_seqlens [rows+1] int32 device offsets; returns (x, B, C, dt) as
    ``prefill_packed`` takes them.  Rows continue their slot's history, or start
    from zeros (``from_zero``, or per row where ``fresh`` [rows] int32 is set)."""
    rows, total = _packed(cu_seqlens, fresh), u.shape[0]
    d, st = cs._call(rows, slots)
    out, io = cs._io(u, dt, (total,), out, stream)
    _check(_lib().replayssm_conv_prefill(ctypes.byref(d), ctypes.byref(st), total, cu_seqlens.data_ptr(),
                                         int(from_zero), _ptr(fresh), ctypes.byref(io), _raw_stream(stream, u)))
    return out


def prefill_packed(ls: LayerState, x, B, C, dt, cu_seqlens, *, from_zero: bool = False, fresh=None,
                   outputs: bool = True, y=None, y_dtype: torch.dtype = torch.float32, stream=None, slots=None):
    """Packed prompts into the checkpoints (replayssm_prefill_packed): x
    [total,H,P], B/C [total,G,N], dt [total,H], cu_seqlens [rows+1] int32 device
    offsets; returns y [total,H,P] in ``y_dtype`` (fp32 or bf16; of ``y`` when it
    is given) when ``outputs``, else None.  A call allocates its scratch, as it
    does a missing ``y``, and gives it back to the allocator."""
    rows, total = _packed(cu_seqlens, fresh), x.shape[0]
    if slots is None and rows != ls.batch:
        raise ReplaySSMError(f"a call without slots covers all {ls.batch} slots, got {rows} sequences")
    if slots is not None:
        _need(slots, (rows,), torch.int32, "slots")
    d, st, _ = _ctx(ls, slots)
    _need(x, (total, ls.heads, ls.head_dim), ls.in_dtype, "x")
    _need(B, (total, ls.groups, ls.d_state), ls.in_dtype, "B")
    _need(dt, (total, ls.heads), ls.in_dtype, "dt")
    if outputs:
        _need(C, (total, ls.groups, ls.d_state), ls.in_dtype, "C")
        if y is None:
            if y_dtype not in _TYPES:
                raise ReplaySSMError(f"y_dtype must be float32 or bfloat16, got {y_dtype}")
            y = _empty((total, ls.heads, ls.head_dim), y_dtype, x.device, stream)
        elif y.dtype not in _TYPES:
            raise ReplaySSMError(f"y must be float32 or bfloat16, got {y.dtype}")
        _need(y, (total, ls.heads, ls.head_dim), y.dtype, "y")
    else:
        y = None
    L = _lib()
    need = L.replayssm_prefill_packed_workspace(ctypes.addressof(d), total)
    # Scratch of this call alone, from its own stream's memory (or a capture's): calls of one layer on two streams
    # share nothing, a captured call's stays with its graph, and no layer holds any between calls.
    ws = _empty((need,), torch.uint8, x.device, stream) if need else None
    _check(L.replayssm_prefill_packed(ctypes.addressof(d), ctypes.addressof(st), total, cu_seqlens.data_ptr(),
                                      int(from_zero), _ptr(fresh), x.data_ptr(), B.data_ptr(), _ptr(C),
                                      dt.data_ptr(), _ptr(y), F32 if y is None else _TYPES[y.dtype],
                                      _ptr(ws), need, _raw_stream(stream, x)))
    return y


def _float(t, name):
    ty = _TYPES.get(t.dtype)
    if ty is None or not t.is_cuda:
        raise ReplaySSMError(f"{name}: expected an fp32 or bf16 device tensor, got {t.dtype} device={t.device}")
    return ty


def gated_norm(y, z, weight, *, groups: int = 1, eps: float = 1e-5, norm_before_gate: bool = False, out=None,
               stream=None):
    """Gated group norm (replayssm_gated_norm): y the recurrence's outputs
    ([rows,H,P] or [rows,dim], dense), z [rows,dim] the gate (a view of the
    projection's rows), weight [dim] fp32; returns [rows,dim] in z's type."""
    if z.dim() != 2:
        raise ReplaySSMError(f"z: expected [rows, dim], got {tuple(z.shape)}")
    rows, dim = shape = z.shape
    yt, zt = _float(y, "y"), _float(z, "z")
    if y.shape[0] != rows or y.numel() != rows * dim or not y.is_contiguous():
        raise ReplaySSMError(f"y: expected a dense tensor of {rows} rows of {dim}, got {tuple(y.shape)} "
                             f"contiguous={y.is_contiguous()}")
    pitch = _pitch(z, (rows,), dim, z.dtype, "z")
    w = _dense(weight, (dim,), torch.float32, "weight")
    if out is None:
        out = _empty(shape, z.dtype, z.device, stream)
    ot = _float(out, "out")
    rc = _lib().replayssm_gated_norm(rows, dim, groups, y.data_ptr(), yt, z.data_ptr(), zt, pitch, w, eps,
                                     1 if norm_before_gate else 0, _dense(out, shape, out.dtype, "out"), ot,
                                     _raw_stream(stream, z))
    if rc:
        _check(rc)
    return out


def add_norm(x, residual, weight, *, scale: float = 1.0, post_weight=None, eps: float = 1e-5, out=None,
             residual_out=None, stream=None):
    """Residual add and norms around a block (replayssm_add_norm): x [rows,dim]
    the block's output (normed with ``post_weight`` when given), residual
    [rows,dim]; returns (normed input of the next block in x's type, new
    residual).  ``residual_out`` may be ``residual``."""
    if x.dim() != 2:
        raise ReplaySSMError(f"x: expected [rows, dim], got {tuple(x.shape)}")
    rows, dim = shape = x.shape
    xt, rt = _float(x, "x"), _float(residual, "residual")
    xp, rp = _dense(x, shape, x.dtype, "x"), _dense(residual, shape, residual.dtype, "residual")
    w = _dense(weight, (dim,), torch.float32, "weight")
    p = None if post_weight is None else _dense(post_weight, (dim,), torch.float32, "post_weight")
    if residual_out is None:
        residual_out = _empty(shape, residual.dtype, x.device, stream)
    if out is None:
        out = _empty(shape, x.dtype, x.device, stream)
    ot = _float(out, "out")
    rc = _lib().replayssm_add_norm(rows, dim, xp, xt, rp, _dense(residual_out, shape, residual.dtype, "residual_out"),
                                   rt, w, p, scale, eps, _dense(out, shape, out.dtype, "out"), ot,
                                   _raw_stream(stream, x))
    if rc:
        _check(rc)
    return out, residual_out
