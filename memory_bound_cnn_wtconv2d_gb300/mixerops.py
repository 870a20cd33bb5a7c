"""Thin ctypes binding of include/wtconv_mixer.h: a gated channel mixer's operators.

Root-mean-square norm with the residual's addition (forward, 8-bit output,
backward), the gated product of two pointwise matrices (forward, on 8-bit
operands, backward), and the global norm of many gradients with clipping.  As
in ``blockops``: argument checks and marshalling only, the C names, work on
the current torch stream unless ``stream`` is given, outputs and workspaces may
be passed in, a mismatch raises ``ValueError`` before anything is launched, and
there is no CPU fallback.  What a call allocates belongs to the stream that it
works on.
"""
from __future__ import annotations

import array
import ctypes
import math

import torch

from . import blockops as _b
from . import wtconv as _c

OP_GATED_FWD, OP_GATED_BWD, OP_GATED_Q8 = 0, 1, 2
E4M3 = torch.float8_e4m3fn

# entry points declared in include/wtconv_mixer.h
EXPORTS = ("wtconv_rms_norm_fwd", "wtconv_rms_norm_q8", "wtconv_quantize_rows", "wtconv_rms_workspace_size",
           "wtconv_rms_norm_bwd", "wtconv_gated_workspace_size", "wtconv_gated_fwd", "wtconv_gated_q8",
           "wtconv_gated_bwd", "wtconv_test_dh_timeout", "wtconv_clip_workspace_size", "wtconv_grad_norm",
           "wtconv_clip_grads")


class RmsDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_longlong), ("C", ctypes.c_int), ("dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("x_stride", ctypes.c_longlong), ("r_stride", ctypes.c_longlong), ("d_stride", ctypes.c_longlong)]


class GatedDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_longlong), ("C", ctypes.c_int), ("H", ctypes.c_int), ("dtype", ctypes.c_int),
                ("act", ctypes.c_int), ("x_stride", ctypes.c_longlong), ("gate_stride", ctypes.c_longlong),
                ("up_stride", ctypes.c_longlong), ("dh_stride", ctypes.c_longlong), ("align", ctypes.c_int)]


class Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_longlong), ("dtype", ctypes.c_int)]


_LIB = None


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        L = _c.lib()
        vp, sz, f, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float, ctypes.c_int
        rd, gd, td = ctypes.POINTER(RmsDesc), ctypes.POINTER(GatedDesc), ctypes.POINTER(Tensor)
        for name, res, args in (
                ("wtconv_rms_norm_fwd", i, [rd, vp, vp, vp, vp, vp, vp, vp]),
                ("wtconv_rms_norm_q8", i, [rd, vp, vp, vp, vp, vp, vp, vp]),
                ("wtconv_quantize_rows", i, [rd, vp, vp, vp, vp]),
                ("wtconv_rms_workspace_size", sz, [rd]),
                ("wtconv_rms_norm_bwd", i, [rd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
                ("wtconv_gated_workspace_size", sz, [gd, i]),
                ("wtconv_gated_fwd", i, [gd, vp, vp, vp, vp, vp, sz, vp]),
                ("wtconv_gated_q8", i, [gd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
                ("wtconv_gated_bwd", i, [gd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
                ("wtconv_test_dh_timeout", None, [i]),
                ("wtconv_clip_workspace_size", sz, [i]),
                ("wtconv_grad_norm", i, [td, i, vp, vp, sz, vp]),
                ("wtconv_clip_grads", i, [td, i, f, f, vp, vp, sz, vp])):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _LIB = L
    return _LIB


def _row_stride(t, name):
    """Distance of the rows of t [..., C], whose leading axes must be walkable with
    one stride; 0 where there is no second row."""
    if not (isinstance(t, torch.Tensor) and _c._on_cuda(t)):
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError(f"{name} must be rows [..., C], got {tuple(shape)}")
    C = shape[-1]
    if t.is_contiguous() or t.numel() == 0:
        return C
    st = t.stride()
    if C > 1 and st[-1] != 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous (stride {st[-1]})")
    row = expect = None
    for size, stride in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if size == 1:
            continue
        if row is None:
            row = stride
        elif stride != expect:
            raise ValueError(f"{name}: the rows must lie one stride apart, got strides {tuple(st)}")
        expect = stride * size
    if row is None:
        return C
    if row < C:
        raise ValueError(f"{name}: rows must not overlap (stride {row}, {C} channels)")
    return row


def _typed(t, name):
    if t.dtype not in _c.DTYPE_CODES:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")


def _like(t, name, x):
    if not isinstance(t, torch.Tensor) or t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError(f"{name} must be {tuple(x.shape)} {x.dtype} on {x.device}, got "
                         f"{(tuple(t.shape), t.dtype, t.device) if isinstance(t, torch.Tensor) else t!r}")


# What a call needs to know of its layout, built once for each: checking and
# describing one costs more than launching it.  Bounded, as in ``blockops``.
_LAYOUTS = {}


def _cached(key, make):
    try:
        lay = _LAYOUTS.get(key)
    except TypeError:  # options that no call takes: the checks say which
        return make()
    if lay is None:
        lay = make()
        if len(_LAYOUTS) >= _b._MAX_LAYOUTS:
            _LAYOUTS.clear()
        _LAYOUTS[key] = lay
    return lay


class _RmsLayout:
    __slots__ = ("desc", "ref", "M", "C", "device", "rows", "ws")

    def __init__(self, x, r, dy, eps, names):
        stride = _row_stride(x, names[0])
        _typed(x, names[0])
        rs = ds = 0
        if r is not None:
            _like(r, names[1], x)
            rs = _row_stride(r, names[1])
        if dy is not None:
            _like(dy, "dy", x)
            ds = _row_stride(dy, "dy")
        if not (math.isfinite(eps) and eps >= 0):
            raise ValueError(f"eps must be finite and not negative, got {eps!r}")
        self.C = x.shape[-1]
        self.rows = x.shape[:-1]
        self.M = math.prod(self.rows)
        self.device = x.device
        self.desc = RmsDesc(self.M, self.C, _c.DTYPE_CODES[x.dtype], eps, stride, rs, ds)
        self.ref = ctypes.byref(self.desc)
        self.ws = 0
        if dy is not None:
            with _b._on(x.device):  # the size follows the device
                self.ws = lib().wtconv_rms_workspace_size(self.ref)


def _rms_layout(x, r, dy, eps, names):
    eps = float(eps)  # a tensor would be found again by its identity, whatever it holds by then

    def make():
        return _RmsLayout(x, r, dy, eps, names)
    try:
        key = (x.shape, x.stride(), x.dtype, x.device, eps, names, None if r is None else (r.shape, r.stride(), r.dtype, r.device),
               None if dy is None else (dy.shape, dy.stride(), dy.dtype, dy.device))
    except AttributeError:  # not tensors: the checks say which
        return make()
    return _cached(key, make)


def _check_out(t, name, shape, dtype, device):
    if t is not None and not (isinstance(t, torch.Tensor) and t.shape == torch.Size(shape) and t.dtype == dtype
                              and t.device == device and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on {device}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def wtconv_rms_norm_fwd(x, weight=None, residual=None, eps=1e-6, y=None, total=None, rstd=None, stream=None):
    """t = x + residual, y = t / sqrt(mean(t^2) + eps) * weight over the channels of
    each row of x [..., C].

    Returns (y, total, rstd): y and total like x (total is t, rounded; x itself
    without a residual), rstd float32 [...], which the backward reads.  weight
    is float32 [C] or None.  x and residual may be slices of wider tensors as
    long as a row's channels are contiguous and the rows lie one stride apart."""
    lay = _rms_layout(x, residual, None, eps, ("x", "residual"))
    device = lay.device
    _b._float32(weight, "weight", lay.C, device)
    if y is not None or total is not None or rstd is not None:
        _check_out(y, "y", x.shape, x.dtype, device)
        if total is not None and residual is None:
            raise ValueError("total is x itself without a residual")
        _check_out(total, "total", x.shape, x.dtype, device)
        _check_out(rstd, "rstd", lay.rows, torch.float32, device)
        _b._disjoint([("y", y), ("total", total), ("rstd", rstd)], [("x", x), ("residual", residual), ("weight", weight)])
        _b._written(y, total, rstd)
    with _b._on(device, stream):
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=device)
        if total is None and residual is not None:
            total = torch.empty(x.shape, dtype=x.dtype, device=device)
        if rstd is None:
            rstd = torch.empty(lay.rows, dtype=torch.float32, device=device)
        status = lib().wtconv_rms_norm_fwd(lay.ref, x.data_ptr(), _ptr(residual), _ptr(weight), y.data_ptr(),
                                           _ptr(total), rstd.data_ptr(), _b._stream_of(device))
        if status:
            _c._check(status)
    return y, (x if residual is None else total), rstd


def _q8(call, x, weight, residual, eps, q, scale, total, stream):
    lay = _rms_layout(x, residual, None, eps, ("x", "residual"))
    device = lay.device
    _b._float32(weight, "weight", lay.C, device)
    if q is not None or scale is not None or total is not None:
        _check_out(q, "q", x.shape, E4M3, device)
        _check_out(scale, "scale", lay.rows, torch.float32, device)
        if total is not None and residual is None:
            raise ValueError("total is x itself without a residual")
        _check_out(total, "total", x.shape, x.dtype, device)
        _b._disjoint([("q", q), ("scale", scale), ("total", total)], [("x", x), ("residual", residual), ("weight", weight)])
        _b._written(q, scale, total)
    with _b._on(device, stream):
        if q is None:
            q = torch.empty(x.shape, dtype=E4M3, device=device)
        if scale is None:
            scale = torch.empty(lay.rows, dtype=torch.float32, device=device)
        if total is None and residual is not None:
            total = torch.empty(x.shape, dtype=x.dtype, device=device)
        status = call(lay.ref, q, scale, total, _b._stream_of(device))
        if status:
            _c._check(status)
    return q, scale, (x if residual is None else total)


def wtconv_rms_norm_q8(x, weight=None, residual=None, eps=1e-6, q=None, scale=None, total=None, stream=None):
    """The norm of ``wtconv_rms_norm_fwd`` with y in 8 bits: (q, scale, total), q
    float8_e4m3fn like x, scale float32 [...], y about q * scale."""
    return _q8(lambda ref, q, scale, total, s: lib().wtconv_rms_norm_q8(
        ref, x.data_ptr(), _ptr(residual), _ptr(weight), q.data_ptr(), scale.data_ptr(), _ptr(total), s),
        x, weight, residual, eps, q, scale, total, stream)


def wtconv_quantize_rows(x, q=None, scale=None, stream=None):
    """Rows of x [..., C] in 8 bits: (q, scale), x about q * scale[..., None]."""
    return _q8(lambda ref, q, scale, total, s: lib().wtconv_quantize_rows(ref, x.data_ptr(), q.data_ptr(), scale.data_ptr(), s),
               x, None, None, 0.0, q, scale, None, stream)[:2]


def wtconv_rms_norm_bwd(dy, total, rstd, weight=None, dtotal=None, dx=None, dweight=None, workspace=None, stream=None,
                        need_dweight=True):
    """Gradients of ``wtconv_rms_norm_fwd``: (dx, dweight).  dx is the gradient of x
    and of the residual alike, with dtotal (the gradient that reaches the sum by
    itself) added; dweight float32 [C] (of a None weight too), or None without
    need_dweight."""
    lay = _rms_layout(total, dtotal, dy, 0.0, ("total", "dtotal"))
    device, C = lay.device, lay.C
    _b._float32(weight, "weight", C, device)
    if rstd is None:
        raise ValueError("rstd is required")
    _b._float32(rstd, "rstd", lay.M, device)
    if dx is not None or dweight is not None or workspace is not None:
        _check_out(dx, "dx", total.shape, total.dtype, device)
        _check_out(dweight, "dweight", (C,), torch.float32, device)
        _b._disjoint([("dx", dx), ("dweight", dweight), ("workspace", workspace)],
                     [("dy", dy), ("total", total), ("dtotal", dtotal), ("rstd", rstd), ("weight", weight)])
        _b._written(dx, dweight)
    with _b._on(device, stream):
        if dx is None:
            dx = torch.empty(total.shape, dtype=total.dtype, device=device)
        if dweight is None and need_dweight:
            dweight = torch.empty(C, dtype=torch.float32, device=device)
        ws, n = _b._scratch(lay.ws if dweight is not None else 0, device, workspace)
        status = lib().wtconv_rms_norm_bwd(lay.ref, dy.data_ptr(), total.data_ptr(), _ptr(dtotal), rstd.data_ptr(),
                                           _ptr(weight), dx.data_ptr(), _ptr(dweight), _ptr(ws), n,
                                           _b._stream_of(device))
        if status:
            _c._check(status)
    return dx, dweight


class _GatedLayout:
    __slots__ = ("desc", "ref", "M", "C", "H", "device", "dtype", "h_shape", "ws")

    def __init__(self, x, gate, up, dh, activation, op, dtype, aligned):
        xs = _row_stride(x, "x")
        C = x.shape[-1]
        device = x.device
        if op == OP_GATED_Q8:
            if x.dtype != E4M3:
                raise ValueError(f"x must be {E4M3}, got {x.dtype}")
            if dtype not in _c.DTYPE_CODES:
                raise ValueError(f"dtype must be float32, float16 or bfloat16, got {dtype!r}")
        else:
            _typed(x, "x")
            dtype = x.dtype
        strides = []
        for t, name in ((gate, "gate"), (up, "up")):
            if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[1] != C or t.shape[0] < 1:
                raise ValueError(f"{name} must be a matrix [H, {C}]")
            if t.dtype != x.dtype or t.device != device:
                raise ValueError(f"{name} must be {x.dtype} on {device}, got {t.dtype} on {t.device}")
            strides.append(_row_stride(t, name))
        if gate.shape != up.shape:
            raise ValueError(f"gate and up must have one shape, got {tuple(gate.shape)} and {tuple(up.shape)}")
        if activation not in _b.ACT_CODES:
            raise ValueError(f"activation must be one of none, silu, gelu, got {activation!r}")
        self.M, self.C, self.H = math.prod(x.shape[:-1]), C, gate.shape[0]
        self.h_shape = (*x.shape[:-1], self.H)
        self.device, self.dtype = device, dtype
        ds = 0
        if dh is not None:
            if not isinstance(dh, torch.Tensor) or dh.shape != torch.Size(self.h_shape) or dh.dtype != x.dtype or dh.device != device:
                raise ValueError(f"dh must be {tuple(self.h_shape)} {x.dtype} on {device}")
            ds = _row_stride(dh, "dh")
        if op == OP_GATED_Q8 and (C % 16 or any(s % 16 for s in (xs, *strides))):
            raise ValueError(f"8-bit operands: the {C} channels and the rows' strides must be multiples of 16")
        self.desc = GatedDesc(self.M, C, self.H, _c.DTYPE_CODES[dtype], _b.ACT_CODES[activation], xs, *strides, ds,
                              16 if aligned else 0)
        self.ref = ctypes.byref(self.desc)
        with _b._on(device):  # the size follows the device
            self.ws = lib().wtconv_gated_workspace_size(self.ref, op)


def _gated_layout(x, gate, up, dh, activation, op, dtype=None):
    def make():
        return _GatedLayout(x, gate, up, dh, activation, op, dtype, aligned)
    aligned = False
    try:
        aligned = (x.data_ptr() | gate.data_ptr() | up.data_ptr()) % 16 == 0
        key = (aligned, x.shape, x.stride(), x.dtype, x.device, gate.shape, gate.stride(), gate.dtype, gate.device, up.shape,
               up.stride(), up.dtype, up.device, activation, op, dtype,
               None if dh is None else (dh.shape, dh.stride(), dh.dtype, dh.device))
    except AttributeError:  # not tensors: the checks say which
        return make()
    return _cached(key, make)


def wtconv_gated_fwd(x, gate, up, activation="silu", h=None, workspace=None, stream=None):
    """h = act(x gate^T) * (x up^T) for rows x [..., C] and matrices gate, up [H, C] of
    one type; h [..., H] contiguous.  activation is "none", "silu" or "gelu"."""
    lay = _gated_layout(x, gate, up, None, activation, OP_GATED_FWD)
    device = lay.device
    if h is not None or workspace is not None:
        _check_out(h, "h", lay.h_shape, lay.dtype, device)
        _b._disjoint([("h", h), ("workspace", workspace)], [("x", x), ("gate", gate), ("up", up)])
        _b._written(h)
    with _b._on(device, stream):
        if h is None:
            h = torch.empty(lay.h_shape, dtype=lay.dtype, device=device)
        ws, n = _b._scratch(lay.ws, device, workspace)
        status = lib().wtconv_gated_fwd(lay.ref, x.data_ptr(), gate.data_ptr(), up.data_ptr(), h.data_ptr(), _ptr(ws), n,
                                        _b._stream_of(device))
        if status:
            _c._check(status)
    return h


def wtconv_gated_q8(x, x_scale, gate, gate_scale, up, up_scale, activation="silu", dtype=torch.bfloat16, h=None,
                    workspace=None, stream=None):
    """``wtconv_gated_fwd`` on 8-bit operands (float8_e4m3fn): x [..., C] with x_scale
    [...], gate and up [H, C] with a scale for each row; the scales are float32.
    h in `dtype`.  C is a multiple of 16."""
    lay = _gated_layout(x, gate, up, None, activation, OP_GATED_Q8, dtype)
    device = lay.device
    for t, name, n in ((x_scale, "x_scale", lay.M), (gate_scale, "gate_scale", lay.H), (up_scale, "up_scale", lay.H)):
        if t is None:
            raise ValueError(f"{name} is required")
        _b._float32(t, name, n, device)
    if h is not None or workspace is not None:
        _check_out(h, "h", lay.h_shape, lay.dtype, device)
        _b._disjoint([("h", h), ("workspace", workspace)], [("x", x), ("gate", gate), ("up", up), ("x_scale", x_scale),
                                                            ("gate_scale", gate_scale), ("up_scale", up_scale)])
        _b._written(h)
    with _b._on(device, stream):
        if h is None:
            h = torch.empty(lay.h_shape, dtype=lay.dtype, device=device)
        ws, n = _b._scratch(lay.ws, device, workspace)
        status = lib().wtconv_gated_q8(lay.ref, x.data_ptr(), x_scale.data_ptr(), gate.data_ptr(), gate_scale.data_ptr(),
                                       up.data_ptr(), up_scale.data_ptr(), h.data_ptr(), _ptr(ws), n,
                                       _b._stream_of(device))
        if status:
            _c._check(status)
    return h


def wtconv_gated_bwd(dh, x, gate, up, activation="silu", dx=None, dgate=None, dup=None, workspace=None, stream=None,
                     need_dx=True, need_dweights=True):
    """Gradients of ``wtconv_gated_fwd``: (dx, dgate, dup), each contiguous and of x's
    type; None in the place of what need_dx or need_dweights leaves out.  x's
    products with the matrices are made again, nothing else is kept of the
    forward."""
    lay = _gated_layout(x, gate, up, dh, activation, OP_GATED_BWD)
    device = lay.device
    if (dgate is None) != (dup is None):
        raise ValueError("dgate and dup are given together or not at all")
    if dx is not None or dgate is not None or workspace is not None:
        _check_out(dx, "dx", x.shape, x.dtype, device)
        _check_out(dgate, "dgate", gate.shape, x.dtype, device)
        _check_out(dup, "dup", up.shape, x.dtype, device)
        _b._disjoint([("dx", dx), ("dgate", dgate), ("dup", dup), ("workspace", workspace)],
                     [("dh", dh), ("x", x), ("gate", gate), ("up", up)])
        _b._written(dx, dgate, dup)
    with _b._on(device, stream):
        if dx is None and need_dx:
            dx = torch.empty(x.shape, dtype=x.dtype, device=device)
        if dgate is None and need_dweights:
            dgate = torch.empty(gate.shape, dtype=x.dtype, device=device)
            dup = torch.empty(up.shape, dtype=x.dtype, device=device)
        ws, n = _b._scratch(lay.ws, device, workspace)
        status = lib().wtconv_gated_bwd(lay.ref, dh.data_ptr(), x.data_ptr(), gate.data_ptr(), up.data_ptr(), _ptr(dx),
                                        _ptr(dgate), _ptr(dup), _ptr(ws), n, _b._stream_of(device))
        if status:
            _c._check(status)
    return dx, dgate, dup


def wtconv_test_dh_timeout(enable: bool) -> None:
    """Test support: while on, a backward's waits for its first copies of dh run out
    (see include/wtconv_mixer.h); off restores normal operation."""
    lib().wtconv_test_dh_timeout(1 if enable else 0)


def _dense(t):
    """Whether the elements fill one stretch of memory, in any order of axes."""
    if t.is_contiguous():
        return True
    expect = 1
    for stride, size in sorted((st, n) for n, st in zip(t.shape, t.stride()) if n != 1):
        if stride != expect:
            return False
        expect *= size
    return True


def _list(tensors, name="tensors"):
    """The tensors, their entries for the library (three 64-bit words each), and their
    device."""
    ts = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
    if not ts:
        raise ValueError(f"{name}: no tensors")
    codes, words = _c.DTYPE_CODES, []
    try:  # a list is as long as a model has parameters: few calls for each
        device = ts[0].device
        index = ts[0].get_device()
        fine = index >= 0
        for t in ts:
            fine = fine and t.get_device() == index and (t.is_contiguous() or _dense(t))
            words += (t.data_ptr(), t.numel(), codes[t.dtype])
    except (AttributeError, KeyError, RuntimeError):  # sparse tensors have no address
        fine = False
    if not fine:
        for t in ts:
            if not (isinstance(t, torch.Tensor) and _c._on_cuda(t)) or t.layout is not torch.strided:
                raise ValueError(f"{name} must be dense CUDA tensors")
            if t.dtype not in codes:
                raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
            if t.device != ts[0].device:
                raise ValueError(f"{name}: one device for all, got {ts[0].device} and {t.device}")
            if not _dense(t):
                raise ValueError(f"{name}: the elements of a tensor must fill one stretch of memory, got strides {t.stride()}")
        raise ValueError(f"{name} must be dense CUDA tensors")
    return ts, (Tensor * len(ts)).from_buffer(array.array("q", words)), device


def wtconv_grad_norm(tensors, norm=None, workspace=None, stream=None):
    """The root of the sum of squares of all elements of a list of tensors (of any
    of the three types, mixed if need be): a float32 tensor of no axes, on the
    GPU."""
    ts, entries, device = _list(tensors)
    need = lib().wtconv_clip_workspace_size(len(ts))
    if norm is not None or workspace is not None:
        _check_out(norm, "norm", (), torch.float32, device)
        _b._disjoint([("norm", norm), ("workspace", workspace)], [(f"tensor {i}", t) for i, t in enumerate(ts)])
        _b._written(norm)
    with _b._on(device, stream):
        if norm is None:
            norm = torch.empty((), dtype=torch.float32, device=device)
        ws, n = _b._scratch(need, device, workspace)
        status = lib().wtconv_grad_norm(entries, len(ts), norm.data_ptr(), ws.data_ptr(), n, _b._stream_of(device))
        if status:
            _c._check(status)
    return norm


def wtconv_clip_grads(tensors, max_norm, eps=1e-6, norm=None, workspace=None, stream=None):
    """Multiplies every tensor of a list in place by min(1, max_norm / (norm + eps)),
    with the norm of ``wtconv_grad_norm``, which it returns."""
    ts, entries, device = _list(tensors)
    if not (max_norm >= 0 and math.isfinite(eps) and eps >= 0):
        raise ValueError("max_norm and eps must not be negative, eps finite")
    need = lib().wtconv_clip_workspace_size(len(ts))
    if norm is not None or workspace is not None:
        _check_out(norm, "norm", (), torch.float32, device)
        _b._disjoint([("norm", norm), ("workspace", workspace)], [(f"tensor {i}", t) for i, t in enumerate(ts)])
        _b._written(norm)
    with _b._on(device, stream):
        if norm is None:
            norm = torch.empty((), dtype=torch.float32, device=device)
        ws, n = _b._scratch(need, device, workspace)
        status = lib().wtconv_clip_grads(entries, len(ts), max_norm, eps, norm.data_ptr(), ws.data_ptr(), n,
                                         _b._stream_of(device))
        if status == _c.WTCONV_ERR_INVALID_ARG:  # what is left of that: tensors that overlap
            raise ValueError(_c.lib().wtconv_last_error().decode())
        if status:
            _c._check(status)
    _b._written(*ts)
    return norm
