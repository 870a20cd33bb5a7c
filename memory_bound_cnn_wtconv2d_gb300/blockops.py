"""Thin ctypes binding of include/wtconv_block.h: the operators around the layer.

Group norm with an activation on channels-last activations (forward and
backward), Newton-Schulz orthogonalisation, and the optimiser step built on
it.  As in ``wtconv``: argument checks and marshalling only, the C names, work
on the current torch stream unless ``stream`` is given, outputs and workspaces
may be passed in, a mismatch raises ``ValueError`` before anything is
launched, and there is no CPU fallback.  What a call allocates belongs to the
stream that it works on.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import wtconv as _c

ACT_CODES = {None: 0, "none": 0, "silu": 1, "gelu": 2}
OP_GN_FWD, OP_GN_BWD = 0, 1
NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)
NS_MAX_COUNT = 64

# entry points declared in include/wtconv_block.h
EXPORTS = ("wtconv_gn_workspace_size", "wtconv_gn_act_fwd", "wtconv_gn_act_bwd", "wtconv_ns_workspace_size",
           "wtconv_orthogonalize", "wtconv_muon_step", "wtconv_block_device_faults",
           "wtconv_block_device_faults_async")


class GnDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_longlong), ("S", ctypes.c_longlong), ("C", ctypes.c_int), ("G", ctypes.c_int),
                ("dtype", ctypes.c_int), ("act", ctypes.c_int), ("eps", ctypes.c_float),
                ("x_sample_stride", ctypes.c_longlong), ("x_row_stride", ctypes.c_longlong),
                ("dy_sample_stride", ctypes.c_longlong), ("dy_row_stride", ctypes.c_longlong)]


class NsDesc(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int), ("m", ctypes.c_int), ("n", ctypes.c_int), ("dtype", ctypes.c_int),
                ("steps", ctypes.c_int), ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("eps", ctypes.c_float)]


_LIB = None


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        L = _c.lib()
        vp, sz, ll, f, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_float, ctypes.c_int
        gd, nd = ctypes.POINTER(GnDesc), ctypes.POINTER(NsDesc)
        for name, res, args in (
                ("wtconv_gn_workspace_size", sz, [gd, i]),
                ("wtconv_gn_act_fwd", i, [gd, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
                ("wtconv_gn_act_bwd", i, [gd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
                ("wtconv_ns_workspace_size", sz, [nd]),
                ("wtconv_orthogonalize", i, [nd, vp, ll, vp, ll, vp, sz, vp]),
                ("wtconv_muon_step", i, [nd, vp, ll, vp, ll, vp, ll, f, i, f, f, vp, sz, vp]),
                ("wtconv_block_device_faults", ctypes.c_uint, []),
                ("wtconv_block_device_faults_async", i, [vp, vp])):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _LIB = L
    return _LIB


class _Here:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(device, stream=None):
    """Makes `device`, and a given stream, current for a call, so that what it
    allocates belongs to the stream that uses it; nothing to do for the current
    ones."""
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            handle = int(stream)
            stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    return _HERE if device.index is None or torch.cuda.current_device() == device.index else _c._device_ctx(device)


def _float32(t, name, numel, device):
    if t is None:
        return
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.float32 and _c._on_cuda(t) and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    if t.numel() != numel or t.device != device:
        raise ValueError(f"{name} must hold {numel} elements on {device}, got {t.numel()} on {t.device}")


def _rows(t, name):
    """(sample stride, row stride) of a channels-last activation [N, ..., C]: the
    axes between the first and the last must be walkable with one stride."""
    if not (isinstance(t, torch.Tensor) and _c._on_cuda(t)):
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() < 2:
        raise ValueError(f"{name} must be channels-last [N, ..., C]")
    if t.dtype not in _c.DTYPE_CODES:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    shape, st = t.shape, t.stride()
    C = shape[-1]
    S = math.prod(shape[1:-1])
    if t.is_contiguous() or t.numel() == 0:
        return S * C, C
    if C > 1 and st[-1] != 1:
        raise ValueError(f"{name}: the channels of a pixel must be contiguous (stride {st[-1]})")
    row = expect = None
    for size, stride in zip(reversed(shape[1:-1]), reversed(st[1:-1])):
        if size == 1:
            continue
        if row is None:
            row = stride
        elif stride != expect:
            raise ValueError(f"{name}: the pixels of a sample must lie one stride apart, got strides {tuple(st)}")
        expect = stride * size
    return st[0], C if row is None else row


class _GnLayout:
    """What a call needs to know of its layout: built once for each."""

    __slots__ = ("desc", "ref", "N", "C", "G", "device", "index", "ws", "contiguous")

    def __init__(self, x, dy, num_groups, eps, activation):
        xs = _rows(x, "x")
        ds = (0, 0)
        if dy is not None:
            ds = _rows(dy, "dy")
            if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != x.device:
                raise ValueError(f"dy must be {tuple(x.shape)} {x.dtype} on {x.device}, "
                                 f"got {tuple(dy.shape)} {dy.dtype} on {dy.device}")
        if activation not in ACT_CODES:
            raise ValueError(f"activation must be one of none, silu, gelu, got {activation!r}")
        shape = x.shape
        C = shape[-1]
        if not (isinstance(num_groups, int) and num_groups >= 1 and C >= 1 and C % num_groups == 0):
            raise ValueError(f"num_groups = {num_groups} must be a positive divisor of the {C} channels")
        self.desc = GnDesc(shape[0], math.prod(shape[1:-1]), C, num_groups, _c.DTYPE_CODES[x.dtype],
                           ACT_CODES[activation], eps, xs[0], xs[1], ds[0], ds[1])
        self.ref = ctypes.byref(self.desc)
        self.N, self.C, self.G = shape[0], C, num_groups
        self.device, self.index = x.device, x.device.index
        self.contiguous = x.is_contiguous()
        with _on(x.device):  # the size follows the device
            self.ws = lib().wtconv_gn_workspace_size(self.ref, OP_GN_FWD if dy is None else OP_GN_BWD)


# Layouts by shapes, strides, types, devices and options: a step calls the
# same few again and again, and checking and describing one costs more than
# launching it.  Bounded, for processes that meet many shapes.
_MAX_LAYOUTS = 1024
_LAYOUTS = {}


def _gn_layout(x, dy, num_groups, eps, activation):
    eps = float(eps)  # a tensor would be found again by its identity, whatever it holds by then
    try:
        # with the type: 4.0 and 4 are equal, but only one of them is taken
        key = (x.shape, x.stride(), x.dtype, x.device, num_groups, type(num_groups), eps, activation,
               None if dy is None else (dy.shape, dy.stride(), dy.dtype, dy.device))
        lay = _LAYOUTS.get(key)
    except (AttributeError, TypeError):  # not tensors, or options no call takes: the checks say which
        key = lay = None
    if lay is None:
        lay = _GnLayout(x, dy, num_groups, eps, activation)
        if len(_LAYOUTS) >= _MAX_LAYOUTS:
            _LAYOUTS.clear()
        if key is not None:
            _LAYOUTS[key] = lay
    return lay


_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device):
    """The handle of the device's current stream."""
    return _RAW_STREAM(device.index) if _RAW_STREAM is not None else torch.cuda.current_stream(device).cuda_stream


def _span(t):
    """First and last byte + 1 that a (possibly strided) tensor reaches."""
    p = t.data_ptr()
    if t.is_contiguous():
        return p, p + t.numel() * t.element_size()
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return p, p + (last + 1) * t.element_size()


def _disjoint(outs, ins):
    o = [(n, _span(t)) for n, t in outs if t is not None and t.numel()]
    every = o + [(n, _span(t)) for n, t in ins if t is not None and t.numel()]
    for i, (n, (a0, a1)) in enumerate(o):
        for m, (b0, b1) in every[i + 1:]:
            if a0 < b1 and b0 < a1:
                raise ValueError(f"{n} overlaps {m}: outputs may not share memory with inputs or other outputs")


def _given(t, name, like, contiguous=True):
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(like.shape)} {like.dtype} tensor on {like.device}")
    return t


def _written(*tensors):
    """Tells autograd that a call has written the caller's tensors: a graph that
    saved one of them before must not be used any more."""
    torch.autograd.graph.increment_version([t for t in tensors if t is not None])


def wtconv_gn_act_fwd(x, num_groups, weight=None, bias=None, eps=1e-5, activation="none", y=None, mean=None,
                      rstd=None, workspace=None, stream=None):
    """y = act(group_norm(x) * weight + bias) on channels-last x [N, ..., C].

    Returns (y, mean, rstd): y contiguous like x, the statistics float32
    [N, num_groups], which the backward reads.  weight and bias are float32
    [C] or None; activation is "none", "silu" or "gelu".  x may be a slice of
    a wider tensor as long as a pixel's channels are contiguous and the pixels
    of a sample lie one stride apart.
    """
    lay = _gn_layout(x, None, num_groups, eps, activation)
    device, C = lay.device, lay.C
    _float32(weight, "weight", C, device)
    _float32(bias, "bias", C, device)
    if y is not None or mean is not None or rstd is not None or workspace is not None:
        if y is not None:
            _given(y, "y", x)
        _float32(mean, "mean", lay.N * lay.G, device)
        _float32(rstd, "rstd", lay.N * lay.G, device)
        _disjoint([("y", y), ("mean", mean), ("rstd", rstd), ("workspace", workspace)],
                  [("x", x), ("weight", weight), ("bias", bias)])
        _written(y, mean, rstd)
    with _on(device, stream):
        if y is None:
            y = torch.empty_like(x) if lay.contiguous else torch.empty(x.shape, dtype=x.dtype, device=device)
        if mean is None:
            mean = torch.empty((lay.N, lay.G), dtype=torch.float32, device=device)
        if rstd is None:
            rstd = torch.empty((lay.N, lay.G), dtype=torch.float32, device=device)
        ws, n = _scratch(lay.ws, device, workspace)
        status = lib().wtconv_gn_act_fwd(
            lay.ref, x.data_ptr(), None if weight is None else weight.data_ptr(),
            None if bias is None else bias.data_ptr(), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
            None if ws is None else ws.data_ptr(), n, _stream_of(device))
        if status:
            _c._check(status)
    return y, mean, rstd


def wtconv_gn_act_bwd(dy, x, mean, rstd, num_groups, weight=None, bias=None, activation="none", dx=None,
                      dweight=None, dbias=None, workspace=None, stream=None, need_dweight=True, need_dbias=True):
    """Gradients of ``wtconv_gn_act_fwd``: (dx, dweight, dbias), dx contiguous in
    x's type, the parameter gradients float32 [C] (of a None weight or bias
    too: what ones and zeros in their place would get).  Without need_dweight
    or need_dbias None in its place; without both, the sums over the batch are
    not made."""
    lay = _gn_layout(x, dy, num_groups, 0.0, activation)
    device, C = lay.device, lay.C
    _float32(weight, "weight", C, device)
    _float32(bias, "bias", C, device)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd are required")
    _float32(mean, "mean", lay.N * lay.G, device)
    _float32(rstd, "rstd", lay.N * lay.G, device)
    if dx is not None or dweight is not None or dbias is not None or workspace is not None:
        if dx is not None:
            _given(dx, "dx", x)
        _float32(dweight, "dweight", C, device)
        _float32(dbias, "dbias", C, device)
        _disjoint([("dx", dx), ("dweight", dweight), ("dbias", dbias), ("workspace", workspace)],
                  [("dy", dy), ("x", x), ("mean", mean), ("rstd", rstd), ("weight", weight), ("bias", bias)])
        _written(dx, dweight, dbias)
    with _on(device, stream):
        if dx is None:
            dx = torch.empty_like(x) if lay.contiguous else torch.empty(x.shape, dtype=x.dtype, device=device)
        if dweight is None and need_dweight:
            dweight = torch.empty(C, dtype=torch.float32, device=device)
        if dbias is None and need_dbias:
            dbias = torch.empty(C, dtype=torch.float32, device=device)
        ws, n = _scratch(lay.ws, device, workspace)
        status = lib().wtconv_gn_act_bwd(
            lay.ref, dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
            None if weight is None else weight.data_ptr(), None if bias is None else bias.data_ptr(), dx.data_ptr(),
            None if dweight is None else dweight.data_ptr(), None if dbias is None else dbias.data_ptr(),
            None if ws is None else ws.data_ptr(), n, _stream_of(device))
        if status:
            _c._check(status)
    return dx, dweight, dbias


def _scratch(need, device, workspace):
    """The caller's workspace, else a new one of the size the call needs."""
    if workspace is not None:
        return workspace, _c._workspace_bytes(workspace, device)
    return (torch.empty(need, dtype=torch.uint8, device=device), need) if need else (None, 0)


class _Stack:
    """Equally shaped matrices: one tensor [..., m, n] or a list of [m, n] tensors."""

    __slots__ = ("pointers", "ld", "count", "m", "n", "dtype", "device", "tensors")

    def __init__(self, t, name, like=None, dtype=None):
        ts = [t] if isinstance(t, torch.Tensor) else list(t)
        if not ts:
            raise ValueError(f"{name}: no matrices")
        first = ts[0]
        ptrs, ld = [], None
        for q in ts:
            if not (isinstance(q, torch.Tensor) and _c._on_cuda(q)):
                raise ValueError(f"{name} must be CUDA tensors")
            shape = q.shape
            if len(shape) < 2:
                raise ValueError(f"{name} must be matrices [..., m, n], got {tuple(shape)}")
            m, n = shape[-2:]
            if q is first:
                self.m, self.n, self.dtype, self.device = m, n, q.dtype, q.device
            elif m != self.m or n != self.n or q.dtype != self.dtype or q.device != self.device:
                raise ValueError(f"{name}: one shape, type and device for all matrices")
            strides = q.stride()
            sm, sn = strides[-2:]
            if n > 1 and sn != 1:
                raise ValueError(f"{name}: the elements of a row must be contiguous (stride {sn})")
            sm = n if m <= 1 else sm
            if sm < n or (ld is not None and sm != ld):
                raise ValueError(f"{name}: rows must not overlap, and lie the same distance apart in all matrices")
            ld = sm
            if len(shape) == 2:
                ptrs.append(q.data_ptr())
            else:
                e, offsets = q.element_size(), [0]
                for size, stride in zip(shape[:-2], strides[:-2]):
                    offsets = [o + i * stride for o in offsets for i in range(size)]
                p = q.data_ptr()
                ptrs += [p + o * e for o in offsets]
        self.tensors = ts
        self.pointers, self.ld, self.count = ptrs, max(ld, 1), len(ptrs)
        if dtype is not None and self.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {self.dtype}")
        if self.dtype not in _c.DTYPE_CODES:
            raise ValueError(f"{name} must be float32, float16 or bfloat16, got {self.dtype}")
        if like is not None and (self.count, self.m, self.n, self.device) != (like.count, like.m, like.n, like.device):
            raise ValueError(f"{name} must be {like.count} x [{like.m}, {like.n}] on {like.device}, "
                             f"got {self.count} x [{self.m}, {self.n}] on {self.device}")

    def spans(self):
        return [_span(t) for t in self.tensors if t.numel()]

    def chunk(self, i, k):
        return (ctypes.c_void_p * k)(*self.pointers[i:i + k])

    def separate(self, name):
        """Raises where two of the matrices, which a call writes, overlap."""
        e = self.tensors[0].element_size()
        size = ((self.m - 1) * self.ld + self.n) * e if self.m and self.n else 0
        p = sorted(self.pointers)
        for i, a in enumerate(p):
            for b in p[i + 1:]:  # every one that begins before this one ends, not the next alone
                if b - a >= size:
                    break
                column = (b - a) // e % self.ld  # side by side in wider rows: apart when neither reaches the other
                if column < self.n or column + self.n > self.ld:
                    raise ValueError(f"{name}: the matrices overlap")


def _disjoint_stacks(w, g, b, workspace):
    """No matrix that a step writes may share memory with another tensor of the call."""
    spans = [(lo, hi, n, t) for n, st in (("weight", w), ("grad", g), ("buffer", b)) for t, (lo, hi) in
             enumerate(st.spans())]
    if workspace is not None:
        spans.append((*_span(workspace), "workspace", 0))
    spans.sort()
    reach = {}
    for lo, hi, name, _ in spans:
        for other, end in reach.items():
            if other != name and lo < end:
                raise ValueError(f"{name} overlaps {other}: outputs may not share memory with inputs or other outputs")
        reach[name] = max(hi, reach.get(name, 0))


# Descriptors and workspace sizes by shape and options.
_NS_DESCS = {}


def _ns_desc(s, count, steps, coefficients, eps):
    eps = float(eps)
    try:
        coefficients = tuple(float(v) for v in coefficients)
        key = (count, s.m, s.n, s.dtype, s.device, steps, type(steps), coefficients, eps)
        got = _NS_DESCS.get(key)
    except TypeError:
        key = got = None
    if got is None:
        if not (isinstance(steps, int) and 0 <= steps <= 64):
            raise ValueError(f"steps must be an int in [0, 64], got {steps!r}")
        if len(coefficients) != 3 or not all(math.isfinite(v) and abs(v) <= 16 for v in coefficients):
            raise ValueError(f"coefficients must be three numbers of at most 16 in size, got {coefficients!r}")
        desc = NsDesc(count, s.m, s.n, _c.DTYPE_CODES[s.dtype], steps, *coefficients, eps)
        ref = ctypes.byref(desc)
        got = (ref, lib().wtconv_ns_workspace_size(ref))
        if len(_NS_DESCS) >= _MAX_LAYOUTS:
            _NS_DESCS.clear()
        if key is not None:
            _NS_DESCS[key] = got
    return got


def wtconv_orthogonalize(g, steps=5, coefficients=NS_COEFFICIENTS, eps=1e-7, out=None, workspace=None, stream=None):
    """Newton-Schulz orthogonalisation of a stack of matrices g [..., m, n]:
    X = g / (|g|_F + eps), then `steps` times X <- a X + (b A + c A A) X with
    A = X X^T, in the orientation with the shorter side first.  Returns a
    contiguous tensor of g's shape and type (or `out`)."""
    s = _Stack(g, "g")
    if not isinstance(g, torch.Tensor):
        raise ValueError("g must be a tensor [..., m, n]")
    if out is not None:
        if out.shape != g.shape or out.dtype != g.dtype or out.device != g.device:
            raise ValueError(f"out must be {tuple(g.shape)} {g.dtype} on {g.device}")
        _disjoint([("out", out), ("workspace", workspace)], [("g", g)])
    elif workspace is not None:
        _disjoint([("workspace", workspace)], [("g", g)])
    with _on(s.device, stream):
        fresh = out is None
        if fresh:
            out = torch.empty(g.shape, dtype=g.dtype, device=g.device)
        o = _Stack(out, "out", like=s)
        if not fresh:
            o.separate("out")
        for i in range(0, s.count, NS_MAX_COUNT):
            k = min(NS_MAX_COUNT, s.count - i)
            ref, need = _ns_desc(s, k, steps, coefficients, eps)
            ws, n = _scratch(need, s.device, workspace)
            status = lib().wtconv_orthogonalize(ref, s.chunk(i, k), s.ld, o.chunk(i, k), o.ld,
                                                None if ws is None else ws.data_ptr(), n, _stream_of(s.device))
            if status:
                _c._check(status)
    if not fresh:
        _written(out)
    return out


def wtconv_muon_step(weight, grad, buffer, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=1.0, steps=5,
                     coefficients=NS_COEFFICIENTS, eps=1e-7, workspace=None, stream=None):
    """One optimiser step on equally shaped matrices, in place:

        buffer <- momentum * buffer + (1 - momentum) * grad
        u = momentum * buffer + (1 - momentum) * grad  (nesterov), else buffer
        weight <- (1 - lr * weight_decay) * weight - lr * scale * orthogonalize(u)

    weight, grad and buffer are stacks [..., m, n] or lists of [m, n] tensors;
    weight and grad of one type, buffer (the running mean of the gradients)
    float32."""
    w = _Stack(weight, "weight")
    g = _Stack(grad, "grad", like=w, dtype=w.dtype)
    b = _Stack(buffer, "buffer", like=w, dtype=torch.float32)
    if not all(math.isfinite(v) for v in (lr, momentum, weight_decay, scale)):
        raise ValueError("lr, momentum, weight_decay and scale must be finite")
    w.separate("weight")
    b.separate("buffer")
    _disjoint_stacks(w, g, b, workspace)
    with _on(w.device, stream):
        for i in range(0, w.count, NS_MAX_COUNT):
            k = min(NS_MAX_COUNT, w.count - i)
            ref, need = _ns_desc(w, k, steps, coefficients, eps)
            ws, n = _scratch(need, w.device, workspace)
            status = lib().wtconv_muon_step(
                ref, w.chunk(i, k), w.ld, g.chunk(i, k), g.ld, b.chunk(i, k), b.ld, momentum,
                int(bool(nesterov)), 1.0 - lr * weight_decay, lr * scale, None if ws is None else ws.data_ptr(), n,
                _stream_of(w.device))
            if status:
                _c._check(status)
    _written(*w.tensors, *b.tensors)
    return weight


def wtconv_block_device_faults() -> int:
    """In-kernel waits of these operators that gave up since the previous call
    (0 in normal operation); synchronises the device and resets the count."""
    return int(lib().wtconv_block_device_faults())


def wtconv_block_device_faults_async(count, device, stream=None) -> None:
    """Enqueues a copy of that count, not reset, to `count`: a pinned int32 CPU
    tensor of one element that stays alive until the copy is done.  No wait."""
    if not (isinstance(count, torch.Tensor) and count.dtype is torch.int32 and count.numel() == 1
            and count.device.type == "cpu" and count.is_pinned()):
        raise ValueError("count must be a pinned int32 CPU tensor of one element")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"device must be a CUDA device, got {device}")
    device = torch.device("cuda", torch.cuda.current_device() if device.index is None else device.index)
    with _on(device, stream):
        _c._check(lib().wtconv_block_device_faults_async(count.data_ptr(), _stream_of(device)))
